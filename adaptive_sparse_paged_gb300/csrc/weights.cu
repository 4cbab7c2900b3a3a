// weights.cu - the attention weight that every cached token receives, summed
// over query rows and over the query heads of its KV head:
//   w_out[s] = decay * w_in[s] + sum_{t >= s} exp(c q_t.k_s - lse_t).
//
// One warp per cached token holds its key row (d / 32 channels a lane) and
// walks the query rows that see it.
#include "asp_internal.cuh"

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct Params {
  const uint16_t* q;
  const int32_t* q_offsets;
  const float* q_f32;
  const int32_t* lists;
  const int32_t* lens;
  const float* lse;
  const float* w_in;
  float* w_out;
  const uint16_t* k;
  const int32_t* bt;
  const int32_t* seq_lens;
  uint32_t* err;
  int B, Hq, Hkv, max_pages, num_phys, num_tokens;
  float scale, decay;
};

template <int D, int P, bool Decode>
__global__ void __launch_bounds__(256) weights_kernel(const Params p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int seg = blockIdx.y, b = seg / p.Hkv, hk = seg % p.Hkv, g = p.Hq / p.Hkv;
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, p.err);
  const NewRows nr = new_rows(Decode ? nullptr : p.q_offsets, b, T, p.num_tokens, p.err);
  const size_t wbase = (size_t)seg * p.max_pages * P;
  for (long long s = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); s < T;
       s += (long long)gridDim.x * 8) {
    const int page = (int)(s / P);
    bool listed = true;
    if (Decode && p.lists) {
      const int N = ceil_div(T, P);
      int len = p.lens[seg];
      if (len < 0 || len > N) {
        report(p.err, ASP_DEVERR_LEN_RANGE);
        len = len < 0 ? 0 : N;
      }
      bool mine = false;
      for (int i = lane; i < len; i += 32) {
        const int e = p.lists[(size_t)seg * p.max_pages + i];
        if (e < 0 || e >= N) report(p.err, ASP_DEVERR_LIST_RANGE);
        mine |= e == page;
      }
      listed = __any_sync(kFull, mine);
    }
    float acc = 0.f;
    if (listed) {
      const int phys = p.bt[(size_t)b * p.max_pages + page];
      if (phys < 0 || phys >= p.num_phys) {
        report(p.err, ASP_DEVERR_PAGE_RANGE);
      } else {
        float k[E];
        const __nv_bfloat16* kr = reinterpret_cast<const __nv_bfloat16*>(p.k) +
                                  (((size_t)phys * p.Hkv + hk) * P + s % P) * D + lane * E;
#pragma unroll
        for (int i = 0; i < E; ++i) k[i] = __bfloat162float(kr[i]);
        for (int i = max(0, (int)(s - (T - nr.n))); i < nr.n; ++i) {
          for (int j = 0; j < g; ++j) {
            const size_t r = (size_t)(nr.row0 + i) * p.Hq + hk * g + j;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
              x += k[e] * (Decode ? p.q_f32[r * D + lane * E + e]
                                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q)[r * D + lane * E + e]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
            const float lse = p.lse[r];
            if (lse != -INFINITY) acc += expf(x * p.scale - lse);
          }
        }
      }
    }
    if (lane == 0) {
      const float before = p.w_in && s < T - nr.n ? p.decay * p.w_in[wbase + s] : 0.f;
      p.w_out[wbase + s] = before + acc;
    }
  }
}

template <int D, int P>
cudaError_t launch_t(const WeightArgs& a, bool decode, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  Params p{a.q, a.q_offsets, a.q_f32, a.lists, a.lens, a.lse, a.w_in, a.w_out, kv.k_cache,
           kv.block_table, kv.seq_lens, a.err, kv.batch, kv.num_q_heads, kv.num_kv_heads,
           kv.max_pages, kv.num_phys_pages, a.num_tokens, a.sm_scale, a.decay};
  const long long blocks = ((long long)kv.max_pages * P + 7) / 8;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536), kv.batch * kv.num_kv_heads);
  auto kernel = decode ? weights_kernel<D, P, true> : weights_kernel<D, P, false>;
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(256), 0, stream, p);
}

cudaError_t launch(const WeightArgs& a, bool decode, cudaStream_t stream) {
  const int d = a.kv->head_dim, P = a.kv->page_size;
  if (d == 128 && P == 16) return launch_t<128, 16>(a, decode, stream);
  if (d == 128 && P == 32) return launch_t<128, 32>(a, decode, stream);
  if (d == 128 && P == 64) return launch_t<128, 64>(a, decode, stream);
  if (d == 64 && P == 16) return launch_t<64, 16>(a, decode, stream);
  if (d == 64 && P == 32) return launch_t<64, 32>(a, decode, stream);
  if (d == 64 && P == 64) return launch_t<64, 64>(a, decode, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_chunk_weights(const WeightArgs& a, cudaStream_t stream) {
  return launch(a, false, stream);
}
cudaError_t launch_decode_weights(const WeightArgs& a, cudaStream_t stream) {
  return launch(a, true, stream);
}

}  // namespace asp
