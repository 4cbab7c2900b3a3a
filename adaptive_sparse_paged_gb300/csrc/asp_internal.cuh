// asp_internal.cuh - device primitives and workspace layout shared by the
// kernels of libasp.so (sm_103a). Nothing here is part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>
#include <utility>

#include "asp.h"

namespace asp {

// Named NVTX range over one host entry point, so a profiler that reads NVTX
// (Nsight Systems, or ncu with --nvtx and --nvtx-include) attributes the
// kernels a call launches to that call. With no tool attached, push and pop
// only test a null hook.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr int kMaxSegments = 4096;     // batch * Hkv handled by one call
constexpr int kMaxPages = 1 << 20;     // max_pages bound (int32 page-space arithmetic)
// The decode splits its page sequence by weight: a list's first page weighs
// 1 + decode_piece_cost(d, P) pages, about the K and V a CTA streams in the
// time that ending a piece stalls it (its 8 warp pipelines drift 2-4 us
// apart over a piece and all wait for the last, then merge). The measured
// step time is flat for weights of 160-384 KiB and worse at 48 or 512 KiB.
constexpr int kDecodePieceBytes = 256 * 1024;
constexpr int kMaxPieceCost = 128;
inline int decode_piece_cost(int head_dim, int page_size) {
  const int page_bytes = 4 * page_size * head_dim;  // K and V, bf16
  const int c = (kDecodePieceBytes + page_bytes / 2) / page_bytes;
  return c < kMaxPieceCost ? c : kMaxPieceCost;
}
constexpr int kMaxGroup = 8;           // query heads per KV head (padded mma width)
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // a bounded on-chip wait gives up after 2 s

// ----------------------------------------------------------------- workspace
// [ header 256 B | arrivals int32[S] | scores f32[S*max_pages] | partials |
//   chunk joins | chunk partials ]
// arrivals[s] counts the decode CTAs done with split segment s; the CTA that
// completes it merges s and puts the count back to zero.
// header word 0 is the sticky device error mask. A CTA of the chunk attention
// leaves at most two partials (its first and its last piece), of up to
// kChunkRows query rows each, and at most one join: where the pieces of the
// item that its last piece begins lie.
constexpr int kChunkRows = 256;
struct ChunkJoin {
  int b, h, item, pieces;  // pieces 0: no item begins here that other CTAs end
};
// Whether the join that CTA `cta` of `ctas` left names pieces of this call. A CTA that gives up
// a wait leaves none (pieces 0), and nothing else that may lie in the workspace is followed.
__host__ __device__ inline bool chunk_join_valid(const ChunkJoin& j, int batch, int kv_heads, int cta,
                                                 int ctas) {
  return j.pieces >= 2 && j.pieces <= ctas - cta && j.b >= 0 && j.b < batch && j.h >= 0 &&
         j.h < kv_heads && j.item >= 0;
}
struct WsLayout {
  size_t arrivals_off = 0;
  size_t scores_off = 0;
  size_t partials_off = 0;
  size_t joins_off = 0;
  size_t chunk_off = 0;
  size_t total = 0;
  int decode_grid = 0;   // CTAs of the decode kernel
  int slot_floats = 0;   // floats per partial slot: m[8], l[8], o[8][d]
};

// floats of one chunk partial: m[kChunkRows], l[kChunkRows], o[kChunkRows][d]
__host__ __device__ inline size_t chunk_slot_floats(int head_dim) {
  return size_t(kChunkRows) * (2 + head_dim);
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline WsLayout ws_layout(const asp_paged_kv& kv, int num_sms) {
  WsLayout w;
  const size_t S = size_t(kv.batch) * kv.num_kv_heads;
  w.decode_grid = num_sms;
  w.slot_floats = 2 * kMaxGroup + kMaxGroup * kv.head_dim;
  w.arrivals_off = 256;
  w.scores_off = align256(w.arrivals_off + S * sizeof(int32_t));
  w.partials_off = align256(w.scores_off + S * size_t(kv.max_pages) * sizeof(float));
  w.joins_off = align256(w.partials_off +
                         (S + size_t(w.decode_grid)) * size_t(w.slot_floats) * sizeof(float));
  w.chunk_off = align256(w.joins_off + size_t(num_sms) * sizeof(ChunkJoin));
  w.total = align256(w.chunk_off + 2 * size_t(num_sms) * chunk_slot_floats(kv.head_dim) *
                                       sizeof(float));
  return w;
}

// ------------------------------------------------------------- device errors
__device__ __forceinline__ void report(uint32_t* err, uint32_t bits) {
  if (err) atomicOr(err, bits);
}

// ------------------------------------------------------------------- helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Valid tokens of request b: seq_lens clamped to [0, max_pages*P]; a clamp
// raises ASP_DEVERR_SEQ_RANGE.
__device__ __forceinline__ int clamp_seq_len(int T, int max_pages, int P, uint32_t* err) {
  const long long cap = (long long)max_pages * P;
  if (T < 0 || (long long)T > cap) {
    report(err, ASP_DEVERR_SEQ_RANGE);
    return T < 0 ? 0 : (int)cap;
  }
  return T;
}

// Request b's rows of a packed batch of new tokens: [row0, row0 + n), the last
// n of its T cached tokens. q_offsets null: one row per request. Offsets that
// do not ascend within [0, num_tokens], or that give more rows than T, set
// ASP_DEVERR_OFFSET_RANGE and leave the request without rows, `bad` set: it is skipped.
struct NewRows {
  int row0, n;
  bool bad;
};
__device__ __forceinline__ NewRows new_rows(const int32_t* q_offsets, int b, int T, int num_tokens,
                                            uint32_t* err) {
  NewRows r{b, 1, false};
  if (q_offsets) {
    r.row0 = q_offsets[b];
    const int end = q_offsets[b + 1];
    r.n = end - r.row0;
    if (r.row0 < 0 || end < r.row0 || end > num_tokens) {
      report(err, ASP_DEVERR_OFFSET_RANGE);
      return NewRows{0, 0, true};
    }
  }
  if (r.n > T) {
    if (q_offsets) report(err, ASP_DEVERR_OFFSET_RANGE);  // an empty request has no row to skip
    return NewRows{0, 0, q_offsets != nullptr};
  }
  return r;
}

// The work items of the calls that append: a page (or block of 2^ls slots) of one request each,
// numbered so that request b's first is floor(off_b / 2^ls) + 2 b: n tokens touch at most
// floor(n / 2^ls) + 2 of them, so that the ranges of requests whose offsets ascend do not
// overlap, and an item finds its request from the offsets alone.
__device__ __forceinline__ int held_offset(const int32_t* q_offsets, int b, int num_tokens) {
  return min(max(q_offsets[b], 0), num_tokens);
}
__device__ __forceinline__ int first_item(const int32_t* q_offsets, int b, int num_tokens, int ls) {
  return (held_offset(q_offsets, b, num_tokens) >> ls) + 2 * b;
}
// The request of item `it`, found by a whole warp: the last whose first item is not past it, -1
// before the first. Only up to the first request whose offsets descend: it is skipped (new_rows),
// and behind it the ranges may overlap others, so that those requests get no items at all.
__device__ __forceinline__ int request_of_item(const int32_t* q_offsets, int B, int num_tokens,
                                               int ls, int it, int lane) {
  int end = B;  // the first request that the item lies before, or that is behind a descent
  for (int y = lane; y < B; y += 32) {
    const int off = held_offset(q_offsets, y, num_tokens);
    const int last = held_offset(q_offsets, max(y - 1, 0), num_tokens);
    const bool past = (off >> ls) + 2 * y > it, fell = off < last;
    end = min(end, past | fell ? y : B);
  }
  return __reduce_min_sync(0xffffffffu, end) - 1;
}

// ------------------------------------------------------------------ mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

__device__ __forceinline__ void mbar_fence_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Waits until the phase with the given parity has completed. Returns false
// (and the caller reports ASP_DEVERR_TIMEOUT) if that takes longer than
// kWaitLimitNs: no wait in this library can spin forever.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

// ----------------------------------------------------------- bulk / TMA copy
// 1-D bulk copy global -> shared, completing `bytes` on the mbarrier.
// Both addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_g2s(void* smem_dst, const void* gsrc, uint32_t bytes,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(gsrc), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// 2-D tiled TMA load of one box at (x, y). x is the innermost coordinate in
// elements and must be a multiple of 8 for bf16 (16-byte rule).
__device__ __forceinline__ void tma_load_2d(void* smem_dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// L2 policy for data read exactly once per call (K/V pages, page summaries):
// evict it first, so that it does not push out the small structures that the
// dependent lookups of every kernel read (lengths, lists, block table, scores).
__device__ __forceinline__ uint64_t l2_evict_first_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// bulk_g2s and tma_load_2d with an L2 cache policy.
__device__ __forceinline__ void bulk_g2s_hint(void* smem_dst, const void* gsrc, uint32_t bytes,
                                              uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(smem_dst)),
      "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_hint(void* smem_dst, const CUtensorMap* map, int x,
                                                 int y, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ----------------------------------------------------------- even splits
// Part i of n of [0, total): the first total % n parts hold one item more.
// 32-bit only (total < 2^31): 64-bit division is a called routine, and at a
// kernel's start its code fetch alone costs microseconds.
struct EvenSplit {
  int q, r;  // items per part, parts with one more
  __device__ __forceinline__ EvenSplit(int total, int n) : q(total / n), r(total % n) {}
  __device__ __forceinline__ int begin(int i) const { return i * q + min(i, r); }
  __device__ __forceinline__ int end(int i) const { return begin(i) + q + (i < r ? 1 : 0); }
  // part holding item x (x < total)
  __device__ __forceinline__ int part_of(int x) const {
    const int big = r * (q + 1);
    return x < big ? x / (q + 1) : r + (x - big) / q;
  }
};

// ------------------------------------------- programmatic dependent launch
// Every kernel of the library is launched with programmatic stream
// serialisation: the next kernel in the stream may be scheduled onto SMs as
// this one's CTAs retire, instead of after the whole grid has drained. Each
// kernel first allows its dependents to launch, then waits for its
// predecessor grid to complete and its memory to be visible before touching
// global memory; only shared-memory and mbarrier set-up come before the wait.
// Stream order is therefore unchanged. Without the launch attribute (or
// after a non-kernel node) both instructions are no-ops.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ------------------------------------------------------ bf16 channel min/max
// Exact: the min or max of two bf16 values is one of them.
__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a),
                             *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                             *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// Two bf16 NaN: what a fold starts from, as the other operand of bmin2 and bmax2 then wins, and
// what a channel that held nothing else ends as (minimum and maximum, like a bulk summary's).
constexpr uint32_t kNanPair = 0x7fff7fffu;
__device__ __forceinline__ uint2 vmin(uint2 a, uint2 b) {
  return make_uint2(bmin2(a.x, b.x), bmin2(a.y, b.y));
}
__device__ __forceinline__ uint2 vmax(uint2 a, uint2 b) {
  return make_uint2(bmax2(a.x, b.x), bmax2(a.y, b.y));
}
__device__ __forceinline__ uint32_t vmin(uint32_t a, uint32_t b) { return bmin2(a, b); }
__device__ __forceinline__ uint32_t vmax(uint32_t a, uint32_t b) { return bmax2(a, b); }


// ------------------------------------------------------ warp-level mma (bf16)
// ldmatrix of four 8x8 b16 matrices; lane i supplies the row address of
// matrix i / 8, row i % 8.
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// c += a * b for one m16n8k16 tile, bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two floats rounded to bf16 and packed, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Orders this thread's generic-proxy global writes before its later
// async-proxy (bulk copy) reads of the same memory.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Orders this thread's generic-proxy shared-memory writes before later
// async-proxy (TMA) accesses to the same buffer.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Asks L2 to fetch `bytes` (a multiple of 16) at a 16-byte aligned global
// address; nothing is returned and nothing waits on it.
__device__ __forceinline__ void prefetch_l2_bulk(const void* gsrc, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(gsrc), "r"(bytes) : "memory");
}

// Named barrier over a subset of the CTA's warps.
__device__ __forceinline__ void named_bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// -------------------------------------------------------------------- launch
// Launchers implemented in the kernel translation units. Each returns a
// cudaError_t from the launch (cudaSuccess when nothing needed launching).
struct SummarizeArgs {
  const asp_paged_kv* kv;
  int mode;
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint32_t* err;
};
cudaError_t launch_summarize(const SummarizeArgs& a, cudaStream_t stream);

struct SelectArgs {
  const asp_paged_kv* kv;
  const float* q;
  float gamma;
  int budget;
  int32_t* lists;
  int32_t* lens;
  float* scores;
  uint32_t* err;
  int num_sms;
  // optional fused append (asp_coverage_select_append): bf16 [B, Hkv, d]
  const uint16_t* k_new = nullptr;
  const uint16_t* v_new = nullptr;
};
cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream);
// The score kernel alone (a.scores: [B, Hkv, max_pages]; lists/lens unused).
cudaError_t launch_scores(const SelectArgs& a, cudaStream_t stream);
// Scoring and selection in one cluster kernel (select_cluster.cu): the
// cluster size C to use for this shape on the current device (0: the shape
// takes the two-kernel path), and the launch. Segments of kClusterSelectMinPages
// to 8192 pages qualify; a.scores is not used.
constexpr int kClusterSelectMinPages = 64;
int cluster_select_ctas(const asp_paged_kv& kv, int num_sms);
cudaError_t launch_cluster_select(const SelectArgs& a, int C, cudaStream_t stream);

struct DecodeArgs {
  const asp_paged_kv* kv;
  const float* q;
  const int32_t* lists;
  const int32_t* lens;
  float sm_scale;
  float* out;
  float* lse;
  float* partials;
  int32_t* arrivals;  // [S], zero between calls
  uint32_t* err;
  int grid;
  int slot_floats;
  const asp_q8_pages* q8 = nullptr;  // launch_q8_decode: the pages
};
cudaError_t launch_q8_decode(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);

// New tokens of a packed batch: rows q_offsets[b] .. q_offsets[b + 1] - 1 belong
// to request b and are the last of its seq_lens[b] tokens. q_offsets null: one
// row per request.
struct NormRotateArgs {
  const asp_paged_kv* kv;
  const uint16_t* qkv;
  const int32_t* q_offsets;
  int num_tokens;
  const int32_t* positions;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  float eps;
  const float* inv_freq;
  int rotary_dim;
  int interleaved;
  uint16_t* q_out;
  float* q_out_f32;
  uint32_t* err;
  int num_sms;
  const asp_q8_pages* q8;    // null: bf16 pages
  int num_axes;              // positions: [num_axes, num_tokens]
  const int32_t* pair_axis;  // null: all of axis 0
};
// bf16 pages, one axis
cudaError_t launch_norm_rotate(const NormRotateArgs& a, cudaStream_t stream);
// positions on several axes, or 8-bit pages
cudaError_t launch_append_rows(const NormRotateArgs& a, cudaStream_t stream);

struct Q8ReadArgs {
  const asp_paged_kv* kv;
  const asp_q8_pages* q8;
  uint16_t* k_out;
  uint16_t* v_out;
  const int32_t* dst_table;
  int dst_pages;
  uint32_t* err;
  int num_sms;
};
cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t stream);

struct ChunkAttentionArgs {
  const asp_paged_kv* kv;
  const uint16_t* q;
  const int32_t* q_offsets;
  int num_tokens;
  float sm_scale;
  uint16_t* out;
  float* lse;
  ChunkJoin* joins;
  float* partials;
  uint32_t* err;
  int num_sms;
  const void* own_out = nullptr;  // prefixes: each row's attention over its own tokens
  const float* own_lse = nullptr;
  int own_bf16 = 0;               // own_out is bf16, not fp32
};
cudaError_t launch_chunk_attention(const ChunkAttentionArgs& a, cudaStream_t stream);
// kv: the prefixes, a request each; q_offsets: the rows of each.
cudaError_t launch_prefix_attention(const ChunkAttentionArgs& a, cudaStream_t stream);

struct WeightArgs {
  const asp_paged_kv* kv;
  const uint16_t* q;           // chunk form
  const int32_t* q_offsets;
  int num_tokens;
  const float* q_f32;          // decode form
  const int32_t* lists;        // null: every page
  const int32_t* lens;
  const float* lse;
  float sm_scale, decay;
  const float* w_in;           // null: no weight before this call
  float* w_out;
  ChunkJoin* joins;            // chunk form
  float* partials;
  uint32_t* err;
  int num_sms;
};
cudaError_t launch_chunk_weights(const WeightArgs& a, cudaStream_t stream);
cudaError_t launch_decode_weights(const WeightArgs& a, cudaStream_t stream);

struct EvictArgs {
  const asp_paged_kv* kv;
  const float* weights;
  int keep, recent;
  const int32_t* dst_table;
  float* w_out;
  int32_t* kept;
  int32_t* new_lens;
  uint32_t* err;
  int num_sms;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

// A 2-D bf16 tensor map over [rows, inner] (row stride inner * 2 bytes) with
// boxes of [box_rows, box_inner] elements, the 128-byte swizzle and zero
// fill out of bounds (decode.cu). box_inner * 2 must be 128.
cudaError_t encode_bf16_2d_swizzled(CUtensorMap* map, const void* base, unsigned long long inner,
                                    unsigned long long rows, unsigned box_inner, unsigned box_rows);
// The same in three dimensions, innermost first; strides in bytes of the outer two.
cudaError_t encode_bf16_3d_swizzled(CUtensorMap* map, const void* base,
                                    const unsigned long long (&dims)[3],
                                    const unsigned long long (&strides)[2],
                                    const unsigned (&box)[3]);

// Per-device helpers (abi.cu).
int current_device_sm_count();
cudaError_t set_max_dynamic_smem(const void* func, int bytes);

}  // namespace asp
