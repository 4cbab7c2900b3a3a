// evict.cu - eviction by accumulated attention weight: per (request, KV head)
// the newest tokens and the heaviest of the others stay, in their order.
//
// select: a cluster of one to eight CTAs per segment, each with a part of its slots in
// registers, finds the weight of rank keep - recent by four 8-bit radix passes over the
// order-preserving integer image of the weights; the CTAs add up one another's bins.
// Weights share few exponents, so most of a warp falls into one bin: every lane
// counts in a column of its own, [bin][lane], and no two lanes of a warp meet.
// One more walk ranks what stays (the slots above that weight, and of its equals
// the lowest) with a block-wide prefix sum and writes kept slots and weights.
//
// move: bound by HBM (every kept K and V row read and written once). A warp takes
// 16 rows a step, 8 bytes a lane; a page's channel minima and maxima are in the
// same registers, so the summaries cost no second read. Old slot kept[i] >= i, so
// in place rows move in ascending tiles, a tile's loads all before its stores: a
// CTA owns some channels (64 to 256 bytes) of every K or V row of a segment and
// walks its slots alone, so that the order needs no word between CTAs. Into other
// pages there is no order to keep, and the slots are split over CTAs too.
//
// Measured: 8 requests of 18-32k tokens (8 KV heads, d = 128) cut to 16k in 208 us, 5.4 TB/s
// over both kernels (selection about 20 us, of which 1.5 us look for pages that both tables have;
// the move 6.0 TB/s); 2k cut to 1k in 11 us. In place the same takes 420 us, and one request
// of 32k 126 us (53 us into other pages): too few CTAs walk the rows for the memory's latency.
#include <cooperative_groups.h>

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

constexpr int kPerThread = 4;                       // slots of a thread in one step
constexpr int kStep = kSelThreads * kPerThread;
constexpr int kHeld = 4;                            // steps whose slots stay in registers

// Exclusive prefix sum over the CTA's threads; `total` gets the whole sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t z = __shfl_up_sync(kFull, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  const uint32_t w = lane < kSelThreads / 32 ? warp_sums[lane] : 0;
  uint32_t z = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(kFull, z, o);
    if (lane >= o) z += u;
  }
  total = __shfl_sync(kFull, z, 31);
  return __shfl_sync(kFull, z - w, warp) + y - x;
}

constexpr int kLogPageSlots = 13;  // of the set of pages below: it takes the place of the bins

// Whether any page of `dst` is one of `src`'s; entries that are no page at all do not count. The
// whole CTA asks. The pages of `src` go into a set in shared memory, at most half as many at a
// time as it has slots, so that a free slot always ends a search.
__device__ __forceinline__ bool share_pages(const int32_t* src, int n_src, const int32_t* dst,
                                            int n_dst, int num_phys, int* set) {
  constexpr int kSlots = 1 << kLogPageSlots, kRound = kSlots / 2;
  auto slot_of = [](int page) { return (int)(page * 2654435769u >> (32 - kLogPageSlots)); };
  int shared = 0;
  for (int r0 = 0; r0 < n_src; r0 += kRound) {
    for (int i = threadIdx.x; i < kSlots; i += kSelThreads) set[i] = -1;
    __syncthreads();
    const int r1 = min(n_src, r0 + kRound);
    for (int i = r0 + threadIdx.x; i < r1; i += kSelThreads) {
      const int page = src[i];
      if (page < 0 || page >= num_phys) continue;
      int at = slot_of(page);
      while (true) {
        const int there = atomicCAS(&set[at], -1, page);
        if (there == -1 || there == page) break;
        at = (at + 1) & (kSlots - 1);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_dst; i += kSelThreads) {
      const int page = dst[i];
      if (page < 0 || page >= num_phys) continue;
      for (int at = slot_of(page); set[at] != -1; at = (at + 1) & (kSlots - 1))
        if (set[at] == page) {
          shared = 1;
          break;
        }
    }
    __syncthreads();
  }
  return __syncthreads_or(shared);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Params p, int P) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ int hist[256 * 32];           // [bin][lane]
  static_assert(256 * 32 == 1 << kLogPageSlots, "the set of pages lies there first");
  __shared__ int bins[2][256];             // this CTA's, read by the cluster; two passes' worth
  __shared__ int all_bins[256];
  __shared__ int counts[2];                // this CTA's slots above and equal
  __shared__ uint32_t warp_sums[2][kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_in_bin;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = blockIdx.x / C, b = seg / p.Hkv;
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, tid == 0 ? p.err : nullptr);
  const float* w = p.weights + (size_t)seg * p.max_pages * P;  // 16-byte aligned: P % 16 == 0
  float* wo = p.w_out + (size_t)seg * p.max_pages * P;
  int32_t* kept = p.kept + (size_t)seg * p.keep;
  const bool tells = seg % p.Hkv == 0 && rank == 0 && tid == 0;  // the request's new length
  if (p.src_table != p.dst_table) {
    // pages of the request's own would be written before they are read: not done
    const size_t at = (size_t)b * p.max_pages;
    const int n = min(T, p.keep);
    if (share_pages(p.src_table + at, ceil_div(T, P), p.dst_table + at, ceil_div(n, P), p.num_phys,
                    hist)) {
      if (tid == 0) report(p.err, ASP_DEVERR_PAGE_RANGE);
      if (tells) p.new_lens[b] = T;  // nothing moved: it is as long as it was
      for (int i = tid; i < n; i += kSelThreads) kept[i] = -1;
      return;
    }
  }
  if (tells) p.new_lens[b] = min(T, p.keep);
  if (T <= p.keep) {
    for (int i = rank * kSelThreads + tid; i < T; i += C * kSelThreads) {
      kept[i] = i;
      wo[i] = w[i];
    }
    return;
  }
  // four slots of this thread from i on; past `end` they are 0 and not used
  auto load4 = [&](int i, int end) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i + 3 < end) {
      x = *reinterpret_cast<const float4*>(w + i);
    } else {
      if (i < end) x.x = w[i];
      if (i + 1 < end) x.y = w[i + 1];
      if (i + 2 < end) x.z = w[i + 2];
    }
    return x;
  };
  // This CTA's slots: [s0, s1). The first steps' weights are read once, all loads in flight;
  // later ones (of parts over kHeld * kStep slots) again in every pass.
  const int span = ceil_div(T, C * kPerThread) * kPerThread;
  const int s0 = min(T, rank * span), s1 = min(T, s0 + span);
  float4 held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = load4(s0 + k * kStep + tid * kPerThread, s1);
  const int m = T - p.recent, need0 = p.keep - p.recent;  // need0 of the first m slots stay
  const int m1 = min(m, s1);
  uint32_t prefix = 0;
  int need = need0;
  if (need0 > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256 * 32; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      auto count = [&](int i0, const float4& x) {
        const int i = i0 + tid * kPerThread;
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u = ordered(y[k]);
          if (i + k < m1 && (shift == 24 || (u >> (shift + 8)) == prefix))
            atomicAdd(&hist[((u >> shift) & 255) * 32 + lane], 1);
        }
      };
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (s0 + k * kStep < m1) count(s0 + k * kStep, held[k]);
      for (int i0 = s0 + kHeld * kStep; i0 < m1; i0 += kStep)
        count(i0, load4(i0 + tid * kPerThread, s1));
      __syncthreads();
      // bin sums: a warp adds up eight bins, a lane a column
#pragma unroll
      for (int k = 0; k < 256 / (kSelThreads / 32); ++k) {
        const int bin = warp * (256 / (kSelThreads / 32)) + k;
        const int n = __reduce_add_sync(kFull, hist[bin * 32 + lane]);
        if (lane == 0) bins[(shift >> 3) & 1][bin] = n;
      }
      int* const own_bins = bins[(shift >> 3) & 1];
      if (C > 1) {
        cluster.sync();
        if (tid < 256) {
          int n = 0;
          for (int r = 0; r < C; ++r) n += cluster.map_shared_rank(own_bins, r)[tid];
          all_bins[tid] = n;
        }
      }
      __syncthreads();
      if (warp == 0) {  // the bin of rank `need` from the top; lane i holds bins 8 i .. 8 i + 7
        int n[8], mine = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) mine += n[k] = (C > 1 ? all_bins : own_bins)[lane * 8 + k];
        int above = mine;  // inclusive sum from this lane's bins to the top
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int z = __shfl_down_sync(kFull, above, o);
          if (lane + o < 32) above += z;
        }
        if (above >= need && above - mine < need) {
          int left = need - (above - mine), k = 7;
          while (n[k] < left) left -= n[k--];
          s_prefix = prefix << 8 | (uint32_t)(lane * 8 + k);
          s_need = left;
          s_in_bin = n[k];
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      if (s_in_bin == need && shift > 0) {
        // the whole bin stays: nothing below its lower edge does, whatever the lower digits
        prefix <<= shift;
        need = 0;
        break;
      }
    }
  }
  // Slots with a larger image than `prefix` stay, and the first `need` that equal it; where a
  // whole bin stays (need 0 after it), equals of its lower edge stay too.
  const bool all_equal = need0 > 0 && need == 0;
  if (all_equal) need = 0x7fffffff;
  // What the CTAs of the slots before keep: each counts its own. The barrier also says that
  // every part in registers has been read, before any slot is written in place.
  int above_before = 0, equal_before = 0;
  if (C > 1) {
    uint32_t mine = 0;  // above in the low half, equal in the high half: 16 of a thread, or
                        // as many as the steps read again give, under 2^16 together
    auto tally = [&](int i0, const float4& x) {
      const int i = i0 + tid * kPerThread;
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t u = ordered(y[k]);
        const bool in = i + k < m1 && need0 > 0;
        mine += ((i + k >= m && i + k < s1) || (in && u > prefix) ? 1u : 0u) +
                (in && u == prefix ? 0x10000u : 0u);
      }
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (s0 + k * kStep < s1) tally(s0 + k * kStep, held[k]);
    for (int i0 = s0 + kHeld * kStep; i0 < s1; i0 += kStep)
      tally(i0, load4(i0 + tid * kPerThread, s1));
    if (tid < 2) counts[tid] = 0;
    __syncthreads();
    const int over_n = __reduce_add_sync(kFull, (int)(mine & 0xffff));
    const int same_n = __reduce_add_sync(kFull, (int)(mine >> 16));
    if (lane == 0) {
      atomicAdd(&counts[0], over_n);
      atomicAdd(&counts[1], same_n);
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      const int* theirs = cluster.map_shared_rank(&counts[0], r);
      above_before += theirs[0];
      equal_before += theirs[1];
    }
    cluster.sync();  // every CTA has read the others' counts: they may end
  }
  int par = 0;
  float4 next = make_float4(0.f, 0.f, 0.f, 0.f);
  auto emit = [&](int i0, const float4& x) {
    const int i = i0 + tid * kPerThread;
    const float y[4] = {x.x, x.y, x.z, x.w};
    bool over[4], same[4];
    uint32_t cnt = 0;  // above in the low half, equal in the high half: at most 4096 each
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t u = ordered(y[k]);
      const bool in = i + k < m1 && need0 > 0;
      over[k] = (i + k >= m && i + k < s1) || (in && u > prefix);
      same[k] = in && u == prefix;
      cnt += (over[k] ? 1u : 0u) + (same[k] ? 0x10000u : 0u);
    }
    uint32_t total;
    const uint32_t pre = block_scan(cnt, warp_sums[par], total);
    int above = above_before + (int)(pre & 0xffff), equal = equal_before + (int)(pre >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (over[k] || (same[k] && equal < need)) {
        const int at = above + min(equal, need);  // at <= slot: in place, later steps are whole
        kept[at] = i + k;
        wo[at] = y[k];
      }
      above += over[k];
      equal += same[k];
    }
    above_before += (int)(total & 0xffff);
    equal_before += (int)(total >> 16);
    par ^= 1;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (s0 + k * kStep < s1) emit(s0 + k * kStep, held[k]);
  // a step's slots are read before the step before is written: it writes lower slots only
  const int more = s0 + kHeld * kStep;
  if (more < s1) next = load4(more + tid * kPerThread, s1);
  for (int i0 = more; i0 < s1; i0 += kStep) {
    const float4 x = next;
    next = load4(i0 + kStep + tid * kPerThread, s1);
    emit(i0, x);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kGroup = 16;  // rows of a warp's lane group in one step

// Lanes: kLanes of them, 8 bytes each, hold a row's slice.
template <int D, int P, int kLanes>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const Params p, int in_order) {
  constexpr int kGroups = 32 / kLanes;                 // groups of 16 rows a warp
  constexpr int kWarpRows = kGroup * kGroups;
  constexpr int kTile = kMoveThreads / 32 * kWarpRows;
  constexpr int kIdx = (kWarpRows + 31) / 32;          // rows whose places a lane looks up
  __shared__ uint2 s_mn[P > kGroup ? kMoveThreads : 1], s_mx[P > kGroup ? kMoveThreads : 1];
  __shared__ uint32_t s_have[P > kGroup ? kMoveThreads : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x, b = seg / p.Hkv, h = seg % p.Hkv;
  const bool is_k = (blockIdx.y & 1) == 0;
  const int c0 = (blockIdx.y >> 1) * (kLanes * 4) + (lane % kLanes) * 4;  // this lane's 4 channels
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, nullptr);
  const int n = min(T, p.keep);
  const int32_t* kept = p.kept + (size_t)seg * p.keep;
  const int32_t* from = p.src_table + (size_t)b * p.max_pages;
  const int32_t* to = p.dst_table + (size_t)b * p.max_pages;
  uint16_t* cache = (is_k ? p.k : p.v) + c0;
  const int tiles = ceil_div(n, kTile);
  const int t0 = (int)((long long)tiles * blockIdx.z / gridDim.z);
  const int t1 = (int)((long long)tiles * (blockIdx.z + 1) / gridDim.z);

  // cache row of slot s under a table, -1 where the table has none
  auto row_of = [&](const int32_t* table, int s) {
    const int phys = table[s / P];
    if (phys < 0 || phys >= p.num_phys) {
      report(p.err, ASP_DEVERR_PAGE_RANGE);
      return -1;
    }
    return (phys * p.Hkv + h) * P + s % P;
  };
  int src[kIdx], dst[kIdx];
  auto places = [&](int t) {
#pragma unroll
    for (int q = 0; q < kIdx; ++q) {
      const int i = t * kTile + warp * kWarpRows + q * 32 + lane;
      src[q] = dst[q] = -1;
      if (q * 32 + lane < kWarpRows && i < n) {
        const int s = kept[i];  // negative: the segment is not moved
        src[q] = s >= 0 ? row_of(from, s) : -1;
        dst[q] = row_of(to, i);
      }
    }
  };
  if (t0 < t1) places(t0);
  for (int t = t0; t < t1; ++t) {
    uint2 x[kGroup];
    int to_row[kGroup];
    uint32_t have = 0;
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int r = lane / kLanes * kGroup + u;  // the warp's row, held by lane r % 32
      int s, d;
      if constexpr (kIdx == 1) {
        s = __shfl_sync(kFull, src[0], r);
        d = __shfl_sync(kFull, dst[0], r);
      } else {
        const int s0 = __shfl_sync(kFull, src[0], r & 31), s1 = __shfl_sync(kFull, src[1], r & 31);
        const int d0 = __shfl_sync(kFull, dst[0], r & 31), d1 = __shfl_sync(kFull, dst[1], r & 31);
        s = r < 32 ? s0 : s1;
        d = r < 32 ? d0 : d1;
      }
      to_row[u] = s >= 0 ? d : -1;
      if (s >= 0) {  // loaded whether or not it has a place to go: places come later
        x[u] = __ldcg(reinterpret_cast<const uint2*>(cache + (size_t)s * D));
      }
    }
    if (t + 1 < t1) places(t + 1);
    if (in_order) __syncthreads();  // every row of the tile is read before one is written
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
      if (to_row[u] >= 0) {
        *reinterpret_cast<uint2*>(cache + (size_t)to_row[u] * D) = x[u];
        have |= 1u << u;
      }
    if (!is_k) continue;
    uint2 mn = make_uint2(kNanPair, kNanPair), mx = mn;
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
      if (have >> u & 1) {
        mn = vmin(mn, x[u]);
        mx = vmax(mx, x[u]);
      }
    const int first = t * kTile + warp * kWarpRows + lane / kLanes * kGroup;  // the group's slot
    if constexpr (P > kGroup) {
      // a page is P / 16 groups in a row: neighbouring lane groups, then warps
      s_mn[tid] = mn;
      s_mx[tid] = mx;
      s_have[tid] = have;
      __syncthreads();
      if (first % P == 0) {
#pragma unroll
        for (int k = 1; k < P / kGroup; ++k) {
          mn = vmin(mn, s_mn[tid + k * kLanes]);
          mx = vmax(mx, s_mx[tid + k * kLanes]);
          have |= s_have[tid + k * kLanes];
        }
      }
      __syncthreads();
    }
    if (first % P == 0 && first < n && have) {  // 0: no row of the page was moved
      uint16_t* s = p.summ + ((size_t)seg * p.max_pages + first / P) * 2 * D + c0;
      *reinterpret_cast<uint2*>(s) = mn;
      *reinterpret_cast<uint2*>(s + D) = mx;
    }
  }
}

template <int D, int P, int kLanes>
cudaError_t launch_move(const Params& p, const asp_paged_kv& kv, int sms, cudaStream_t stream) {
  auto kernel = evict_move_kernel<D, P, kLanes>;
  const int slices = D / (kLanes * 4) * 2, segments = kv.batch * kv.num_kv_heads;
  const bool in_order = p.src_table == p.dst_table;
  // Into other pages: enough CTAs to fill the GPU (three an SM fit) twice over.
  const int tile = kMoveThreads / 32 * kGroup * (32 / kLanes);
  const int splits =
      in_order ? 1 : max(1, min(ceil_div(p.keep, tile), ceil_div(6 * sms, slices * segments)));
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(segments, slices, splits), dim3(kMoveThreads), 0, stream, p,
                    (int)in_order);
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
  // CTAs of a segment: as many as the GPU holds at once, with more than 4096 slots each. With
  // the weights in place the whole segment has to be in registers (a CTA writes slots that
  // another reads); a table too long for that leaves the segment to one CTA. Both go by the
  // table's capacity, which the host knows, not by the lengths, which it does not.
  const long long capacity = (long long)kv.max_pages * P;
  int C = 1;
  while (C < 8 && 2 * C * segments <= a.num_sms && capacity > 8192ll * C) C *= 2;
  if (p.weights == p.w_out && capacity > (long long)C * kHeld * kStep) C = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(segments * C);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)C, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, P)) != cudaSuccess) return e;
  // Whole rows where the segments alone fill the GPU; in place with fewer of them,
  // slices of 64 bytes make up for it.
  const bool few = p.src_table == p.dst_table && segments < a.num_sms;
  if (few) return launch_move<D, P, 8>(p, kv, a.num_sms, stream);
  return launch_move<D, P, D / 4>(p, kv, a.num_sms, stream);
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
