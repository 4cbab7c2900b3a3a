// evict.cu - eviction by accumulated attention weight: per (request, KV head)
// the newest tokens and the heaviest of the others stay, in their order.
//
// select: one CTA per segment finds the weight of rank keep - recent by four
// 8-bit radix passes over the order-preserving integer image of the weights,
// then walks the slots once more, ranks what stays with a block-wide prefix
// sum and writes kept slots and weights.
//
// move: old slot kept[i] >= i, so moving rows in ascending order never
// overwrites one that is still to be read. Rows are split by channels, not by
// slots: a CTA owns 32 bytes of every K (or V) row of its segment and walks
// the slots in tiles, a tile's loads all before its stores, so that the order
// holds inside the CTA and no CTA waits for another, in place too. The K CTAs
// have each page's channels in registers and write its summary.
#include "asp_internal.cuh"

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 1024;

struct Params {
  const float* weights;
  const int32_t* src_table;
  const int32_t* dst_table;
  const int32_t* seq_lens;
  float* w_out;
  int32_t* kept;
  int32_t* new_lens;
  uint16_t* k;
  uint16_t* v;
  uint16_t* summ;
  uint32_t* err;
  int Hkv, max_pages, num_phys, keep, recent;
};

// Order-preserving image of a weight: larger weight, larger integer. Both
// zeros are equal; NaN is the largest.
__device__ __forceinline__ uint32_t ordered(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive prefix sum over the CTA's threads; `total` gets the whole sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of the call before are read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const int y = warp_sums[w];
    if (w < warp) before += y;
    total += y;
  }
  return before + x;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Params p, int P) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, seg = blockIdx.x, b = seg / p.Hkv;
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, tid == 0 ? p.err : nullptr);
  const float* w = p.weights + (size_t)seg * p.max_pages * P;
  float* wo = p.w_out + (size_t)seg * p.max_pages * P;
  int32_t* kept = p.kept + (size_t)seg * p.keep;
  if (seg % p.Hkv == 0 && tid == 0) p.new_lens[b] = min(T, p.keep);
  if (T <= p.keep) {
    for (int i = tid; i < T; i += kSelThreads) {
      kept[i] = i;
      wo[i] = w[i];
    }
    return;
  }
  const int m = T - p.recent, need0 = p.keep - p.recent;  // need0 of the first m slots stay
  uint32_t prefix = 0;
  int need = need0;
  for (int shift = 24; need0 > 0 && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kSelThreads) {
      const uint32_t u = ordered(w[i]);
      if (shift == 24 || (u >> (shift + 8)) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = 255;
      while (hist[d] < left) left -= hist[d--];
      s_prefix = prefix << 8 | d;
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // prefix: the smallest weight that stays; need: how many of that weight do
  int out = 0, ties = 0;
  for (int i0 = 0; i0 < T; i0 += kSelThreads) {
    const int i = i0 + tid;
    const float x = i < T ? w[i] : 0.f;
    const uint32_t u = ordered(x);
    const bool in = i < m && need0 > 0;
    int total;
    const int tie = block_scan(in && u == prefix, warp_sums, total);
    const bool stays = i < T && (i >= m || (in && (u > prefix || (u == prefix && ties + tie <= need))));
    ties += total;
    const int at = out + block_scan(stays, warp_sums, total) - 1;
    out += total;
    if (stays) {  // at <= i: in place, later tiles are still whole
      kept[at] = i;
      wo[at] = x;
    }
  }
}

template <int D, int P>
__global__ void __launch_bounds__(256) evict_move_kernel(const Params p) {
  constexpr int kU = 4;               // rows of one lane pair in a tile
  constexpr int kTile = 8 * 16 * kU;  // rows of a tile: a warp owns 64 in a row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x, b = seg / p.Hkv, h = seg % p.Hkv;
  const bool is_k = blockIdx.z == 0;
  const int c0 = blockIdx.y * 16 + (lane & 1) * 8;  // first of this lane's 8 channels
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, nullptr);
  const int n = min(T, p.keep);
  const int32_t* kept = p.kept + (size_t)seg * p.keep;
  const int32_t* from = p.src_table + (size_t)b * p.max_pages;
  const int32_t* to = p.dst_table + (size_t)b * p.max_pages;
  uint16_t* cache = is_k ? p.k : p.v;
  for (int t0 = 0; t0 < n; t0 += kTile) {
    uint4 x[kU];
    bool ok[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = t0 + warp * 16 * kU + u * 16 + (lane >> 1);
      ok[u] = false;
      if (i >= n) continue;
      const int s = kept[i];
      const int phys = from[s / P];
      if (phys < 0 || phys >= p.num_phys) {
        report(p.err, ASP_DEVERR_PAGE_RANGE);
        continue;
      }
      ok[u] = true;
      x[u] = *reinterpret_cast<const uint4*>(cache + (((size_t)phys * p.Hkv + h) * P + s % P) * D + c0);
    }
    __syncthreads();  // every row of the tile is read before one is written
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = t0 + warp * 16 * kU + u * 16 + (lane >> 1);
      if (i >= n || !ok[u]) continue;
      const int phys = to[i / P];
      if (phys < 0 || phys >= p.num_phys) {
        report(p.err, ASP_DEVERR_PAGE_RANGE);
        continue;
      }
      *reinterpret_cast<uint4*>(cache + (((size_t)phys * p.Hkv + h) * P + i % P) * D + c0) = x[u];
    }
    if (!is_k) continue;
    // summaries: rows 16 u .. 16 u + 15 of the warp lie in the lanes; a page is P / 16 of them
#pragma unroll
    for (int u0 = 0; u0 < kU; u0 += P / 16) {
      uint32_t mn[4], mx[4];
      bool any = false;
#pragma unroll
      for (int u = u0; u < u0 + P / 16; ++u) {
        if (!ok[u]) continue;
        const uint32_t y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mn[c] = any ? vmin(mn[c], y[c]) : y[c];
          mx[c] = any ? vmax(mx[c], y[c]) : y[c];
        }
        any = true;
      }
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) {
        const bool oa = __shfl_xor_sync(kFull, (int)any, o) != 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t a = __shfl_xor_sync(kFull, any ? mn[c] : 0u, o);
          const uint32_t z = __shfl_xor_sync(kFull, any ? mx[c] : 0u, o);
          mn[c] = any && oa ? vmin(mn[c], a) : any ? mn[c] : a;
          mx[c] = any && oa ? vmax(mx[c], z) : any ? mx[c] : z;
        }
        any |= oa;
      }
      const int page = (t0 + warp * 16 * kU + u0 * 16) / P;
      if (lane < 2 && any && page * P < n) {
        uint16_t* s = p.summ + ((size_t)seg * p.max_pages + page) * 2 * D + c0;
        *reinterpret_cast<uint4*>(s) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
        *reinterpret_cast<uint4*>(s + D) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
      }
    }
  }
}

template <int D, int P>
cudaError_t launch_t(const EvictArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  Params p{a.weights, kv.block_table, a.dst_table, kv.seq_lens, a.w_out, a.kept, a.new_lens,
           kv.k_cache, kv.v_cache, kv.summaries, a.err, kv.num_kv_heads, kv.max_pages,
           kv.num_phys_pages, a.keep, a.recent};
  const int segments = kv.batch * kv.num_kv_heads;
  cudaError_t e = set_max_dynamic_smem((const void*)evict_select_kernel, 0);
  if (e != cudaSuccess) return e;
  if ((e = set_max_dynamic_smem((const void*)evict_move_kernel<D, P>, 0)) != cudaSuccess) return e;
  e = launch_pdl(evict_select_kernel, dim3(segments), dim3(kSelThreads), 0, stream, p, P);
  if (e != cudaSuccess) return e;
  return launch_pdl(evict_move_kernel<D, P>, dim3(segments, D / 16, 2), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
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
