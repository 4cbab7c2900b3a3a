// norm_rotate.cu - new tokens into the paged cache: per-head norms of queries
// and keys, position rotation, the write of K and V into their pages and the
// fold of the keys into the page summaries, in one pass over the packed rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// One work item is one page of one request: the new tokens that fall into it.
// Its CTA computes each token's cosines and sines once, in shared memory, for
// all heads; a warp takes a head and walks the item's tokens, so a key head's
// channel minima and maxima stay in registers until the page is done and the
// summary is written once, without atomics. d / 4 lanes hold a row, 8 bytes
// each; the two halves of a rotated pair meet through one shuffle.
//
// The angle: a frequency becomes a 64-bit fixed-point fraction of a turn, whose
// product with the integer position wraps exactly modulo one turn, so that
// position 2^31 is as exact as position 0 (in 32-bit floats an angle of 10^5
// radians is off by 0.004).
#include "asp_internal.cuh"

namespace asp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

struct Params {
  const uint16_t* qkv;
  const int32_t* q_offsets;
  const int32_t* positions;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const float* inv_freq;
  uint16_t* q_out;
  float* q_out_f32;
  uint16_t* k;
  uint16_t* v;
  uint16_t* summ;
  const int32_t* bt;
  const int32_t* seq_lens;
  uint32_t* err;
  int B, Hq, Hkv, max_pages, num_phys, num_tokens;
  int rot, interleaved;
  float eps;
};

// Work items are numbered so that request b's first is floor(off_b / P) + 2 b:
// n tokens touch at most floor(n / P) + 2 pages, so the ranges do not overlap,
// and an item finds its request from the offsets alone. One row per request:
// item b is request b.
template <int P>
__device__ __forceinline__ int first_item(const int32_t* q_offsets, int b, int num_tokens) {
  return min(max(q_offsets[b], 0), num_tokens) / P + 2 * b;
}

__device__ __forceinline__ float2 unpack(uint32_t x) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x));
}

template <int D, int P>
__global__ void __launch_bounds__(kThreads) norm_rotate_kernel(const Params p) {
  constexpr int kLanes = D / 4;          // lanes of one row
  constexpr int kRows = 32 / kLanes;     // rows a warp takes at once
  constexpr int kUnroll = 4;
  __shared__ float2 turn[P * (D / 2)];   // (cos, sin) of [token of the page][pair]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / kLanes, l = lane % kLanes, c0 = 4 * l;
  pdl_launch_dependents();
  pdl_wait_predecessor();

  if (p.q_offsets && blockIdx.x == 0 && blockIdx.y == 0) {  // every request's rows are checked
    for (int x = tid; x < p.B; x += kThreads)
      new_rows(p.q_offsets, x, clamp_seq_len(p.seq_lens[x], p.max_pages, P, p.err), p.num_tokens,
               p.err);
  }

  // the item's request: the last whose first item is not past it
  int b, page_of_b;
  if (p.q_offsets) {
    int before = 0;
    for (int x = 0; x < p.B; x += kThreads)
      before += __syncthreads_count(x + tid < p.B && first_item<P>(p.q_offsets, x + tid,
                                                                  p.num_tokens) <= (int)blockIdx.x);
    b = before - 1;  // offsets that do not ascend: some request of the batch
    if (b < 0) return;
    page_of_b = blockIdx.x - first_item<P>(p.q_offsets, b, p.num_tokens);
  } else {
    b = blockIdx.x;
    page_of_b = 0;
  }
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, tid == 0 ? p.err : nullptr);
  const NewRows nr = new_rows(p.q_offsets, b, T, p.num_tokens, tid == 0 ? p.err : nullptr);
  const int first = T - nr.n;                       // slot of the first new token
  const int page = first / P + page_of_b;
  const int lo = max(first, page * P), hi = min(T, (page + 1) * P);
  if (lo >= hi || page_of_b < 0) return;
  const int row0 = nr.row0 + (lo - first), cnt = hi - lo;  // packed rows of the item

  const int half = p.rot / 2;
  for (int i = tid; i < cnt * half; i += kThreads) {
    const int t = i / half, f = i % half;
    const int pos = p.positions ? p.positions[row0 + t] : lo + t;
    double turns = (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    const unsigned long long fixed = (unsigned long long)(turns * 18446744073709551616.0);
    const unsigned long long phase = fixed * (unsigned long long)(long long)pos;
    float s, c;
    sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // 2 * 2^-32 half turns
    turn[t * (D / 2) + f] = make_float2(c, s);
  }
  const int phys = p.bt[(size_t)b * p.max_pages + page];
  const bool mapped = phys >= 0 && phys < p.num_phys;
  if (!mapped && tid == 0) report(p.err, ASP_DEVERR_PAGE_RANGE);
  __syncthreads();

  const int Hall = p.Hq + 2 * p.Hkv;
  const float inv_d = 1.0f / D;
  for (int h = blockIdx.y * kWarps + warp; h < p.Hq + p.Hkv; h += gridDim.y * kWarps) {
    const bool key = h >= p.Hq;
    if (key && !mapped) continue;
    const uint16_t* wsrc = key ? p.k_weight : p.q_weight;
    float w[4] = {1.f, 1.f, 1.f, 1.f};
    if (wsrc) {
      const uint2 wb = *reinterpret_cast<const uint2*>(wsrc + c0);
      const float2 w0 = unpack(wb.x), w1 = unpack(wb.y);
      w[0] = w0.x, w[1] = w0.y, w[2] = w1.x, w[3] = w1.y;
    }
    const size_t head_block = key ? ((size_t)phys * p.Hkv + (h - p.Hq)) * P : 0;
    uint2 mn = make_uint2(0, 0), mx = mn;
    bool any = false;
    for (int t0 = 0; t0 < cnt; t0 += kRows * kUnroll) {
      uint2 x[kUnroll], vv[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int t = t0 + u * kRows + sub;
        x[u] = vv[u] = make_uint2(0, 0);
        if (t < cnt) {
          const uint16_t* row = p.qkv + ((size_t)(row0 + t) * Hall + h) * D + c0;
          x[u] = __ldg(reinterpret_cast<const uint2*>(row));
          if (key) vv[u] = __ldg(reinterpret_cast<const uint2*>(row + (size_t)p.Hkv * D));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int t = t0 + u * kRows + sub;
        const float2 x0 = unpack(x[u].x), x1 = unpack(x[u].y);
        float y[4] = {x0.x, x0.y, x1.x, x1.y};
        if (wsrc) {
          float ss = y[0] * y[0] + y[1] * y[1] + y[2] * y[2] + y[3] * y[3];
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
          const float r = rsqrtf(ss * inv_d + p.eps);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = y[i] * r * w[i];
        }
        if (p.rot > 0) {
          if (p.interleaved) {
            if (c0 < p.rot && t < cnt) {
              const float2* cs = turn + t * (D / 2) + c0 / 2;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float a = y[2 * i], bb = y[2 * i + 1];
                y[2 * i] = a * cs[i].x - bb * cs[i].y;
                y[2 * i + 1] = bb * cs[i].x + a * cs[i].y;
              }
            }
          } else {
            const int hl = p.rot / 8;  // lanes of one half of the rotated channels
            const int peer = l < hl ? l + hl : l < 2 * hl ? l - hl : l;
            float z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = __shfl_sync(kFull, y[i], peer + sub * kLanes);
            if (c0 < p.rot && t < cnt) {
              const float2* cs = turn + t * (D / 2) + (l < hl ? c0 : c0 - half);
              const float sign = l < hl ? -1.f : 1.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = y[i] * cs[i].x + sign * z[i] * cs[i].y;
            }
          }
        }
        if (t >= cnt) continue;
        const uint2 yb = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        if (!key) {
          const size_t o = ((size_t)(row0 + t) * p.Hq + h) * D + c0;
          if (p.q_out) *reinterpret_cast<uint2*>(p.q_out + o) = yb;
          if (p.q_out_f32)
            *reinterpret_cast<float4*>(p.q_out_f32 + o) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
          const size_t o = (head_block + (lo + t) % P) * D + c0;
          *reinterpret_cast<uint2*>(p.k + o) = yb;
          *reinterpret_cast<uint2*>(p.v + o) = vv[u];
          mn = any ? vmin(mn, yb) : yb;
          mx = any ? vmax(mx, yb) : yb;
          any = true;
        }
      }
    }
    if (!key) continue;
    if (kRows == 2) {  // the two half-warps took alternate rows
      const uint2 on = make_uint2(__shfl_xor_sync(kFull, mn.x, 16), __shfl_xor_sync(kFull, mn.y, 16));
      const uint2 ox = make_uint2(__shfl_xor_sync(kFull, mx.x, 16), __shfl_xor_sync(kFull, mx.y, 16));
      const bool oa = __shfl_xor_sync(kFull, (int)any, 16) != 0;
      mn = any && oa ? vmin(mn, on) : any ? mn : on;
      mx = any && oa ? vmax(mx, ox) : any ? mx : ox;
    }
    if (sub != 0) continue;
    uint16_t* s = p.summ + (((size_t)b * p.Hkv + (h - p.Hq)) * p.max_pages + page) * 2 * D + c0;
    uint2* smin = reinterpret_cast<uint2*>(s);
    uint2* smax = reinterpret_cast<uint2*>(s + D);
    const bool fresh = lo == page * P;
    *smin = fresh ? mn : vmin(*smin, mn);
    *smax = fresh ? mx : vmax(*smax, mx);
  }
}

template <int D, int P>
cudaError_t launch_t(const NormRotateArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  Params p{a.qkv, a.q_offsets, a.positions, a.q_weight, a.k_weight, a.inv_freq, a.q_out,
           a.q_out_f32, kv.k_cache, kv.v_cache, kv.summaries, kv.block_table, kv.seq_lens, a.err,
           kv.batch, kv.num_q_heads, kv.num_kv_heads, kv.max_pages, kv.num_phys_pages,
           a.num_tokens, a.rotary_dim, a.interleaved, a.eps};
  const int items = a.q_offsets ? a.num_tokens / P + 2 * kv.batch : kv.batch;
  const int heads = kv.num_q_heads + kv.num_kv_heads;
  // Few items: split their heads over several CTAs (each computes the angles
  // again) until there are about four CTAs an SM.
  const int split = min(ceil_div(heads, kWarps), max(1, 4 * a.num_sms / items));
  cudaError_t e = set_max_dynamic_smem((const void*)norm_rotate_kernel<D, P>, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_rotate_kernel<D, P>, dim3(items, split), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_norm_rotate(const NormRotateArgs& a, cudaStream_t stream) {
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
