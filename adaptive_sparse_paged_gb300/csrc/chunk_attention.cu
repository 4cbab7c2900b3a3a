// chunk_attention.cu - causal attention of a chunk of new tokens over the
// paged cache: out = sum_s softmax_s(c q.k_s) v_s over the slots s <= t.
//
// One warp per (row, query head) walks the request's slots with a running
// maximum and sum; each lane owns d / 32 channels.
#include "asp_internal.cuh"

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct Params {
  const uint16_t* q;
  const int32_t* q_offsets;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* bt;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;
  uint32_t* err;
  int B, Hq, Hkv, max_pages, num_phys, num_tokens;
  float scale;
};

template <int D, int P>
__global__ void __launch_bounds__(256) chunk_attention_kernel(const Params p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (unit >= (long long)p.num_tokens * p.Hq) return;
  const int row = unit / p.Hq, h = unit % p.Hq, hk = h / (p.Hq / p.Hkv);
  for (int b = 0; b < p.B; ++b) {
    const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, p.err);
    const NewRows nr = new_rows(p.q_offsets, b, T, p.num_tokens, p.err);
    if (row < nr.row0 || row >= nr.row0 + nr.n) continue;
    const int t = T - nr.n + row - nr.row0;
    float q[E], o[E], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      q[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q)[unit * D + lane * E + i]);
      o[i] = 0.f;
    }
    for (int page = 0; page <= t / P; ++page) {
      const int phys = p.bt[(size_t)b * p.max_pages + page];
      if (phys < 0 || phys >= p.num_phys) {
        report(p.err, ASP_DEVERR_PAGE_RANGE);
        continue;
      }
      const size_t base = ((size_t)phys * p.Hkv + hk) * P * D + lane * E;
      for (int s = 0; s < min(P, t + 1 - page * P); ++s) {
        const __nv_bfloat16* kr = reinterpret_cast<const __nv_bfloat16*>(p.k) + base + s * D;
        const __nv_bfloat16* vr = reinterpret_cast<const __nv_bfloat16*>(p.v) + base + s * D;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) x += q[i] * __bfloat162float(kr[i]);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(kFull, x, k);
        x *= p.scale;
        const float top = fmaxf(m, x);
        const float keep = expf(m - top), w = expf(x - top);
        sum = sum * keep + w;
        m = top;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * __bfloat162float(vr[i]);
      }
    }
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i)
      reinterpret_cast<__nv_bfloat16*>(p.out)[unit * D + lane * E + i] = __float2bfloat16(o[i] * inv);
    if (lane == 0) p.lse[unit] = sum > 0.f ? m + logf(sum) : -INFINITY;
    return;
  }
}

template <int D, int P>
cudaError_t launch_t(const ChunkAttentionArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  Params p{a.q, a.q_offsets, kv.k_cache, kv.v_cache, kv.block_table, kv.seq_lens, a.out, a.lse,
           a.err, kv.batch, kv.num_q_heads, kv.num_kv_heads, kv.max_pages, kv.num_phys_pages,
           a.num_tokens, a.sm_scale};
  cudaError_t e = set_max_dynamic_smem((const void*)chunk_attention_kernel<D, P>, 0);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)a.num_tokens * kv.num_q_heads;
  return launch_pdl(chunk_attention_kernel<D, P>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0,
                    stream, p);
}

}  // namespace

cudaError_t launch_chunk_attention(const ChunkAttentionArgs& a, cudaStream_t stream) {
  const int d = a.kv->head_dim, P = a.kv->page_size;
  if (d == 128 && P == 16) return launch_t<128, 16>(a, stream);
  if (d == 128 && P == 32) return launch_t<128, 32>(a, stream);
  if (d == 128 && P == 64) return launch_t<128, 64>(a, stream);
  if (d == 64 && P == 16) return launch_t<64, 16>(a, stream);
  if (d == 64 && P == 32) return launch_t<64, 32>(a, stream);
  if (d == 64 && P == 64) return launch_t<64, 64>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace asp
