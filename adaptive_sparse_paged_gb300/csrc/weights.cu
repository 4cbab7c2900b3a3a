// weights.cu - the attention weight that every cached token receives, summed
// over query rows and over the query heads of its KV head:
//   w_out[s] = decay * w_in[s] + sum_{t >= s} exp(c q_t.k_s - lse_t).
//
// The products run transposed on the tensor cores, S^T = K Q^T with 128 keys as
// rows, so that a thread owns one key: its sum over the query rows needs no
// exchange and no atomics, and comes out in a fixed order.
//
// Chunk form (chunk_weights_kernel): a persistent CTA per SM takes an equal share
// of the units (256 keys x 128 query rows, chunk_plan.cuh); two key tiles stay in
// tensor memory while the query tiles that see it stream past (from shared memory it
// would be read again for every one of them, and with the query tile's own reads and
// writes that is more than shared memory gives); with one key tile instead of two the
// query tiles' loads are what bounds the kernel (1030 cycles a tile of 128 x 128,
// whatever the products and sums take). A warpgroup sums one key tile's rows; three
// products are in tensor memory at once. The rows' lse is subtracted by the product
// itself: read from shared memory for every element it cost as much as the products. An
// item that several CTAs share leaves its partial sums in the workspace; a second, small
// kernel adds them up.
//
// Measured: 2048 rows over 32768 tokens (32 query, 8 KV heads, d = 128) in 0.38 ms, 1.40
// PFLOP/s; a product of 128 x 128 takes some 85 cycles a step where 64 are the tensor cores'
// own, the port of tensor memory being shared with the sums' reads. 733 us with keys in
// shared memory and the lse read an element at a time. At d = 64 as long (0.39 ms, 0.69
// PFLOP/s): the exponentials are as many, their pipe is 59% busy, the tensor pipe 37%.
//
// Decode form (decode_weights_kernel): one token a request, fp32 queries, page
// lists. The keys are read once and the kernel is bound by HBM, so the tiles of
// all lists form one sequence, two CTAs an SM take equal shares of it, and the
// queries (at most 8 heads of a group, each as three bf16 terms that add up to
// its 24 bits) ride along as 32 columns. Measured: 30% of the pages of 4 x 131072
// tokens in 48 us, 6.0 TB/s; all of 8 x 4096 in 10.3 us.
#include "chunk_plan.cuh"
#include "tc.cuh"

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// ================================================================ chunk form
constexpr int kThreads = 384;  // two summing warpgroups; loader, issuer, piece warp, an idle one
constexpr int kLoadWarp = 8, kMmaWarp = 9, kTaskWarp = 10;
constexpr int kKeyBufs = 3, kRowBufs = 3, kSumBufs = 3;
constexpr int kFlagRing = 16;  // tiles of rows whose flags are kept: more than are in flight
constexpr int kLseBytes = 2 * 128 * 16;  // a tile's lse as one step of the contraction
constexpr int kMaskRing = 16;
constexpr uint32_t kTmemCols = 512;    // sums (128 columns each), then key tiles (64 each)
constexpr uint32_t kKeyCol = 128 * kSumBufs;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;
};

struct ChunkShared {
  uint64_t k_full[kKeyBufs], k_empty[kKeyBufs], r_full[kRowBufs], r_empty[kRowBufs];
  uint64_t s_full[kSumBufs], s_empty[kSumBufs], k_done, drain;
  ChunkTasks tasks;
  ChunkStart start;
  long long scratch[kThreads / 32];
  uint32_t page_mask[kMaskRing];
  uint32_t row_none[kFlagRing];               // some row of the tile adds nothing:
  uint32_t row_adds[kFlagRing][kTileRows / 32];  // then these are the ones that do
  uint32_t tmem;
};

template <int D>
constexpr size_t chunk_smem() {
  return 1024 + (kKeyBufs + kRowBufs) * (size_t)Cfg<D>::kTileBytes + (1 + kRowBufs) * kLseBytes +
         sizeof(ChunkShared);
}

struct ChunkParams {
  ChunkDims c;
  const int32_t* bt;
  const float* lse;
  const float* w_in;
  float* w_out;
  ChunkJoin* joins;
  float* partials;
  uint32_t* err;
  int Hq, num_phys;
  float scale_log2, inv_scale, decay;
};

// Weight of slot s before the call: the chunk's own tokens had none.
__device__ __forceinline__ float weight_before(const float* w_in, float decay, size_t at, int s,
                                               int first_new) {
  return w_in && s < first_new ? decay * w_in[at] : 0.f;
}

template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_weights_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK, const ChunkParams p) {
  using C = Cfg<D>;
  constexpr int kPages = kTileKeys / P;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* keys = smem;
  uint8_t* rows = smem + kKeyBufs * C::kTileBytes;
  // One more step of the contraction subtracts the rows' lse: three ones in every key's
  // row against the three bf16 terms of -lse / scale in every query's.
  uint8_t* ones = rows + kRowBufs * C::kTileBytes;
  uint8_t* lses = ones + kLseBytes;  // [kRowBufs]
  ChunkShared& sh = *reinterpret_cast<ChunkShared*>(lses + kRowBufs * kLseBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kKeyBufs; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < kRowBufs; ++i) {
      mbar_init(&sh.r_full[i], 1);
      mbar_init(&sh.r_empty[i], 1);
    }
    for (int i = 0; i < kSumBufs; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 4);  // a warpgroup's warps
    }
    mbar_init(&sh.k_done, 1);
    mbar_init(&sh.drain, 1);
    chunk_tasks_init(sh.tasks, 10);  // loader, issuer, eight summing warps
    mbar_fence_init();
  }
  if (tid == kLoadWarp * 32) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
  }
  for (int i = tid; i < (1 + kRowBufs) * kLseBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(ones)[i] =
        i < 128 ? make_uint4(0x3f803f80u, 0x00003f80u, 0, 0) : make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // the tensor memory is taken: the next kernel cannot take it first
  pdl_wait_predecessor();
  const uint32_t tmem = sh.tmem;
  chunk_plan<KeyCut>(p.c, &sh.start, sh.scratch, p.err);
  const int g = p.c.g, tile_tokens = kTileRows >> p.c.lg;
  ChunkReader reader(sh.tasks);
  ChunkTask task;  // x: row tiles of the piece, the first of them

  if (warp > kMmaWarp) {
    if (tid == kTaskWarp * 32) {
      // ---------------------------------------------------------- pieces
      const bool ok = chunk_hand_out<KeyCut>(
          sh.tasks, p.c, sh.start, p.joins + blockIdx.x,
          [&](const ChunkWalk<KeyCut>& w, ChunkTask& t) {
            t.x[0] = w.r.n > 0 ? w.u1 - w.u0 : 0;
            t.x[1] = KeyCut::first_tile(w.r, p.c.lg, w.item) + w.u0;
          });
      if (!ok) report(p.err, ASP_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loader
    uint32_t kt = 0, rt = 0;  // key tiles, row tiles loaded so far
    int row_tok[4], row_at[4];  // the lane's rows in a tile: token, and place in lse
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      row_tok[i] = (lane * 4 + i) >> p.c.lg;
      row_at[i] = row_tok[i] * p.Hq + ((lane * 4 + i) & (g - 1));
    }
    bool ok = true;
    while (ok && reader.next(task)) {
      const int steps = task.x[0], tile0 = task.x[1];
      if (steps == 0) continue;
      for (int t = 0; t < 2; ++t, ++kt) {
        const uint32_t kb = kt % kKeyBufs;
        ok = ok && __all_sync(kFull, mbar_wait(&sh.k_empty[kb], ((kt / kKeyBufs) & 1) ^ 1));
        if (!ok) break;
        const int page = (2 * task.item + t) * kPages + lane;
        const bool have = lane < kPages && page < ceil_div(task.T, P);
        const int phys = have ? p.bt[(size_t)task.b * p.c.max_pages + page] : 0;
        const bool good = have && phys >= 0 && phys < p.num_phys;
        if (have && !good) report(p.err, ASP_DEVERR_PAGE_RANGE);
        const uint32_t mask = __ballot_sync(kFull, good);
        if (lane == 0) {
          sh.page_mask[kt % kMaskRing] = mask;
          const uint32_t bytes = __popc(mask) * (P * 128 * C::kHalves);
          if (bytes) mbar_arrive_expect_tx(&sh.k_full[kb], bytes);
          else mbar_arrive(&sh.k_full[kb]);
        }
        __syncwarp();
        if (good) {
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_2d(keys + kb * C::kTileBytes + hf * 16384 + lane * P * 128, &tmK, hf * 64,
                        (phys * p.c.Hkv + task.h) * P, &sh.k_full[kb]);
        }
      }
      if (!ok) break;
      // the rows' lse, four a lane, read one step ahead
      float next[4];
      const float* lse = p.lse + (size_t)task.row0 * p.Hq + task.h * g;
      auto fetch = [&](int j) {
        const int tok0 = (tile0 + j) * tile_tokens;
        const float* src = lse + (size_t)tok0 * p.Hq;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          next[i] = tok0 + row_tok[i] < task.n ? src[row_at[i]] : -INFINITY;
      };
      fetch(0);
      for (int j = 0; j < steps; ++j, ++rt) {
        const uint32_t rb = rt % kRowBufs;
        const int tok0 = (tile0 + j) * tile_tokens;
        uint4 terms[4];
        uint32_t adds = 0;  // which of the lane's four rows add anything
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = -next[i] * p.inv_scale;
          const bool none = fabsf(next[i]) == INFINITY;
          adds |= none ? 0u : 1u << i;
          const uint32_t hm = pack_bf16(v, 0.f);
          const float r1 = v - __uint_as_float(hm << 16);
          const uint32_t mid = pack_bf16(0.f, r1);
          const float r2 = r1 - __uint_as_float(mid & 0xffff0000u);
          terms[i] = none ? make_uint4(0, 0, 0, 0)
                          : make_uint4((hm & 0xffffu) | mid, pack_bf16(r2, 0.f), 0, 0);
        }
        if (j + 1 < steps) fetch(j + 1);
        ok = __all_sync(kFull, mbar_wait(&sh.r_empty[rb], ((rt / kRowBufs) & 1) ^ 1));
        if (!ok) break;
        uint4* dst = reinterpret_cast<uint4*>(lses + rb * kLseBytes) + lane * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = terms[i];
        fence_proxy_async_smem();
        const bool some_none = __any_sync(kFull, adds != 15u);
        if (some_none) {
          uint32_t word = adds << (lane % 8 * 4);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(kFull, word, o);
          if (lane % 8 == 0) sh.row_adds[rt % kFlagRing][lane / 8] = word;
        }
        __syncwarp();
        if (lane == 0) {
          sh.row_none[rt % kFlagRing] = some_none;
          mbar_arrive_expect_tx(&sh.r_full[rb], C::kTileBytes);
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(rows + rb * C::kTileBytes + hf * 16384, &tmQ, hf * 64, task.h * g,
                        task.row0 + tok0, &sh.r_full[rb]);
        }
        __syncwarp();
      }
    }
    if (!(ok && reader.ok) && lane == 0) {
      report(p.err, ASP_DEVERR_TIMEOUT);
      for (uint32_t t = kt > kKeyBufs ? kt - kKeyBufs : 0; t < kt; ++t)  // copies in flight end
        mbar_wait(&sh.k_full[t % kKeyBufs], (t / kKeyBufs) & 1);
      for (uint32_t t = rt > kRowBufs ? rt - kRowBufs : 0; t < rt; ++t)
        mbar_wait(&sh.r_full[t % kRowBufs], (t / kRowBufs) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kDesc = mma_desc(kTileKeys, kTileRows, false);
    const uint32_t k0 = uniform(smem_u32(keys)), r0 = uniform(smem_u32(rows));
    const uint32_t tm = uniform(tmem), l0 = uniform(smem_u32(lses));
    const uint64_t one = smem_desc_plain(uniform(smem_u32(ones)), kLseBytes / 2);
    uint32_t kt = 0, rt = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(kFull, mbar_wait(bar, parity)) != 0;
    };
    while (ok && uniform(reader.next(task))) {
      const int steps = uniform(task.x[0]);
      if (steps == 0) continue;
      // the products with the keys before are done
      ok = wait(&sh.k_done, ((kt >> 1) & 1) ^ 1);
      const uint32_t a = tm + kKeyCol;
      for (int t = 0; t < 2 && ok; ++t, ++kt) {
        const uint32_t kb = kt % kKeyBufs;
        ok = wait(&sh.k_full[kb], (kt / kKeyBufs) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t k_tile = smem_desc(k0 + kb * C::kTileBytes, 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tmem_copy(a + 64 * t + 8 * k, k_tile + (((k / 4) * 16384 + (k % 4) * 32) >> 4));
          mma_commit(&sh.k_empty[kb]);
        }
      }
      for (int j = 0; ok && j < steps; ++j, ++rt) {
        const uint32_t rb = rt % kRowBufs;
        ok = wait(&sh.r_full[rb], (rt / kRowBufs) & 1);
        const uint64_t b = smem_desc(r0 + rb * C::kTileBytes, 16);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t x = 2 * rt + t, sb = x % kSumBufs;
          ok = ok && wait(&sh.s_empty[sb], ((x / kSumBufs) & 1) ^ 1);
          if (!ok) continue;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ts(tm + sb * 128, a + 64 * t + 8 * k,
                     b + (((k / 4) * 16384 + (k % 4) * 32) >> 4), kDesc, k > 0);
            mma_ss(tm + sb * 128, one, smem_desc_plain(l0 + rb * kLseBytes, kLseBytes / 2), kDesc,
                   1);
            mma_commit(&sh.s_full[sb]);
            if (t == 1) mma_commit(&sh.r_empty[rb]);
          }
        }
      }
      if (elect_one()) mma_commit(&sh.k_done);
    }
    if (!(ok && reader.ok) && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
    if (elect_one()) mma_commit(&sh.drain);  // no arrival is still on its way when the CTA ends
    mbar_wait(&sh.drain, 0);
  } else {
    // ------------------------------------------------------------ sums
    const int t = warp >> 2, row = tid & 127;  // the warpgroup's key tile, the thread's key in it
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const float c = p.scale_log2;
    uint32_t kt = 0, rt = 0;
    bool ok = true;
    while (ok && reader.next(task)) {
      const int slot = task.item * kItemKeys + t * kTileKeys + row;
      const int steps = task.x[0], tile0 = task.x[1];
      const int first_new = task.T - task.n;
      float sum = 0.f;
      if (steps > 0) {
        for (int j = 0; j < steps; ++j, ++rt) {
          const uint32_t x = 2 * rt + t, sb = x % kSumBufs;
          ok = __all_sync(kFull, mbar_wait(&sh.s_full[sb], (x / kSumBufs) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t s_at = tmem + lanes + sb * 128;
          auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_empty[sb]);
          };
          // rows from `lo` on see this key
          const int lo = (slot - first_new - (tile0 + j) * tile_tokens) * g;
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          const bool none = sh.row_none[rt % kFlagRing] != 0;
          if (__any_sync(kFull, lo > 0) || none) {
            // few tiles: a short loop, whose code is fetched faster than straight code
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int from = lo - 32 * i;
              uint32_t see = from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
              if (none) see &= sh.row_adds[rt % kFlagRing][i];
              uint32_t x[32];
              tmem_ld32(s_at + 32 * i, x);
              tmem_wait_ld(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = ex2(__uint_as_float(x[e]) * c);
                part[e & 3] += see >> e & 1 ? y : 0.f;
              }
            }
            release();
          } else {
            uint32_t s[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_wait_ld(s[i]);
            release();
            const float2 c2 = make_float2(c, c);
            float2 two[4] = {};
            // 16 exponentials at a time; the ones before are summed while they run
            auto exponentials = [&](int q) {
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                uint32_t* x = &s[q / 2][(q & 1) * 16 + e];
                const float2 y =
                    mul2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2);
                x[0] = __float_as_uint(ex2(y.x));
                x[1] = __float_as_uint(ex2(y.y));
              }
            };
            exponentials(0);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              if (q < 7) exponentials(q + 1);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const uint32_t* x = &s[q / 2][(q & 1) * 16 + e];
                two[(e / 2) & 3] = add2(two[(e / 2) & 3], make_float2(__uint_as_float(x[0]),
                                                                      __uint_as_float(x[1])));
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) part[i] = two[i].x + two[i].y;
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
        }
        if (!ok) break;
        if (!((sh.page_mask[(kt + t) % kMaskRing] >> (row / P)) & 1)) sum = 0.f;
        kt += 2;
      }
      if (!task.whole) {
        p.partials[(size_t)(2 * blockIdx.x + (task.u0 == 0 ? 1 : 0)) * kItemKeys + t * kTileKeys +
                   row] = sum;
      } else if (slot < task.T) {
        const size_t at = ((size_t)task.b * p.c.Hkv + task.h) * p.c.max_pages * P + slot;
        p.w_out[at] = weight_before(p.w_in, p.decay, at, slot, first_new) + sum;
      }
    }
    if (!(ok && reader.ok) && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

// Adds up the pieces of the item that CTA blockIdx.x began, in CTA order.
__global__ void __launch_bounds__(kItemKeys) weights_join_kernel(const ChunkParams p) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  ChunkJoin jn;
  ChunkRequest r;
  if (!chunk_join<KeyCut>(p.c, p.joins, p.err, jn, r)) return;
  const int row = threadIdx.x, slot = jn.item * kItemKeys + row;
  if (slot >= r.T) return;
  float sum = p.partials[(size_t)(2 * blockIdx.x + 1) * kItemKeys + row];
  for (int k = 1; k < jn.pieces; ++k)
    sum += p.partials[(size_t)(2 * (blockIdx.x + k)) * kItemKeys + row];
  const size_t at = ((size_t)jn.b * p.c.Hkv + jn.h) * p.c.max_pages * p.c.P + slot;
  p.w_out[at] = weight_before(p.w_in, p.decay, at, slot, r.T - r.n) + sum;
}

template <int D, int P>
cudaError_t launch_chunk_t(const WeightArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  const int g = kv.num_q_heads / kv.num_kv_heads;
  const unsigned long long cache_rows =
      (unsigned long long)kv.num_phys_pages * kv.num_kv_heads * P;
  CUtensorMap tq, tk;
  // a call without rows reads none: its map only has to be valid
  const int n = a.num_tokens > 0 ? a.num_tokens : 1;
  const void* q = a.num_tokens > 0 ? (const void*)a.q : (const void*)kv.k_cache;
  cudaError_t e =
      encode_bf16_3d_swizzled(&tq, q, {D, (unsigned long long)kv.num_q_heads, (unsigned long long)n},
                              {2 * D, 2ull * D * kv.num_q_heads},
                              {64, (unsigned)g, (unsigned)(kTileRows / g)});
  if (e != cudaSuccess) return e;
  if ((e = encode_bf16_2d_swizzled(&tk, kv.k_cache, D, cache_rows, 64, P)) != cudaSuccess) return e;
  ChunkParams p{{a.q_offsets, kv.seq_lens, kv.batch, kv.num_kv_heads, g, chunk_log2(g), kv.max_pages, P,
                 a.num_tokens, chunk_inverse(a.num_sms)},
                kv.block_table, a.lse, a.w_in, a.w_out, a.joins, a.partials, a.err, kv.num_q_heads,
                kv.num_phys_pages, a.sm_scale * kLog2e, 1.0f / a.sm_scale, a.decay};
  constexpr size_t smem = chunk_smem<D>();
  if ((e = set_max_dynamic_smem((const void*)chunk_weights_kernel<D, P>, (int)smem)) != cudaSuccess)
    return e;
  if ((e = set_max_dynamic_smem((const void*)weights_join_kernel, 0)) != cudaSuccess) return e;
  e = launch_pdl(chunk_weights_kernel<D, P>, dim3(a.num_sms), dim3(kThreads), smem, stream, tq, tk,
                 p);
  if (e != cudaSuccess) return e;
  return launch_pdl(weights_join_kernel, dim3(a.num_sms), dim3(kItemKeys), 0, stream, p);
}

// =============================================================== decode form
constexpr int kDecThreads = 224;  // summing warpgroup; loader, issuer, query warp
constexpr int kDecLoad = 4, kDecMma = 5, kDecQuery = 6;
constexpr int kQueryRows = 24;    // 8 heads x (high, middle, low)
constexpr int kQueryCols = 32;    // the products' width, a multiple of 16: the last 8 columns
                                  // come from whatever lies behind the rows and are not read
constexpr int kMetaRing = 16;     // key tiles whose pages are kept: more than are in flight
constexpr int kDecBufs = 4;      // products in tensor memory at once
constexpr int kDecCols = kQueryCols * kDecBufs;

template <int D>
struct DecCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kQueryBytes = kHalves * kQueryRows * 128;
};

struct DecShared {
  int page[kMetaRing][kTileKeys / 16];  // logical page of each listed page of the tile
  float lse[2][kMaxGroup];              // -lse * log2(e) of the segment's heads
  uint64_t full[6], empty[6], q_full[2], q_empty[2], l_empty[2];
  uint64_t s_full[kDecBufs], s_empty[kDecBufs], drain;
  int warp_sum[kDecThreads / 32];
  int seg, tile;
  uint32_t tmem;
};
constexpr int kNoPage = -1, kNotMapped = 1 << 30;

template <int D>
constexpr size_t decode_smem() {
  using C = DecCfg<D>;
  return 1024 + C::kStages * (size_t)C::kTileBytes + 2 * (size_t)C::kQueryBytes + sizeof(DecShared);
}

struct DecodeParams {
  const float* q;
  const int32_t* lists;  // null: every page
  const int32_t* lens;
  const float* lse;
  const float* w_in;
  float* w_out;
  const int32_t* bt;
  const int32_t* seq_lens;
  uint32_t* err;
  int B, Hq, Hkv, g, max_pages, num_phys;
  float scale_log2, decay;
};

// Pages a segment's tiles run over.
template <int P>
__device__ __forceinline__ int listed_pages(const DecodeParams& p, int seg, int T, uint32_t* err) {
  const int n = ceil_div(T, P);
  if (!p.lens) return n;
  const int len = p.lens[seg];
  if (len < 0 || len > n) {
    report(err, ASP_DEVERR_LEN_RANGE);
    return len < 0 ? 0 : n;
  }
  return len;
}

// A CTA's tiles: segment by segment, each role walks them for itself.
template <int P>
struct DecodeWalk {
  static constexpr int kPages = kTileKeys / P;
  const DecodeParams& p;
  int left, seg, tile, T, pages, tiles;
  __device__ __forceinline__ DecodeWalk(const DecodeParams& prm, int count, int s, int t)
      : p(prm), left(count), seg(s), tile(t) {
    if (left > 0) load();
  }
  __device__ __forceinline__ void load() {
    T = clamp_seq_len(p.seq_lens[seg / p.Hkv], p.max_pages, P, nullptr);
    pages = listed_pages<P>(p, seg, T, nullptr);
    tiles = ceil_div(pages, kPages);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  // Tiles of the current segment that are this CTA's.
  __device__ __forceinline__ int run() const { return min(left, tiles - tile); }
  __device__ __forceinline__ void next_segment() {
    left -= run();
    tile = 0;
    if (left <= 0) return;
    do {  // the share ends in a later segment that has tiles
      if (++seg >= p.B * p.Hkv) {
        left = 0;
        return;
      }
      load();
    } while (tiles == 0);
  }
};

template <int D, int P>
__global__ void __launch_bounds__(kDecThreads, 2)
    decode_weights_kernel(const __grid_constant__ CUtensorMap tmK, const DecodeParams p) {
  using C = DecCfg<D>;
  constexpr int kPages = kTileKeys / P;      // listed pages of a tile
  constexpr int kBatch = 32 / kPages;        // tiles whose pages a warp looks up at once
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* queries = smem;  // before the ring: the products read 1 KiB past the rows
  uint8_t* ring = smem + 2 * C::kQueryBytes;
  DecShared& sh = *reinterpret_cast<DecShared*>(ring + C::kStages * C::kTileBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.l_empty[i], 128);
    }
    for (int i = 0; i < kDecBufs; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 128);
    }
    mbar_init(&sh.drain, 1);
    mbar_fence_init();
  }
  if (warp == kDecMma) tmem_alloc(&sh.tmem, kDecCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // the tensor memory is taken: the next kernel cannot take it first
  pdl_wait_predecessor();
  const uint32_t tmem = sh.tmem;

  // ---- plan: tiles of all segments, an equal share for this CTA
  const int S = p.B * p.Hkv;
  const int per = ceil_div(S, kDecThreads), s0 = min(S, tid * per), s1 = min(S, s0 + per);
  uint32_t* err0 = blockIdx.x == 0 ? p.err : nullptr;
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int T = clamp_seq_len(p.seq_lens[s / p.Hkv], p.max_pages, P, err0);
    mine += ceil_div(listed_pages<P>(p, s, T, err0), kPages);
  }
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh.warp_sum[warp] = x;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kDecThreads / 32; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  before += x - mine;
  const EvenSplit split(total, gridDim.x);
  const int first = split.begin(blockIdx.x), count = split.end(blockIdx.x) - first;
  if (count > 0 && first >= before && first < before + mine) {
    int at = before;
    for (int s = s0; s < s1; ++s) {
      const int T = clamp_seq_len(p.seq_lens[s / p.Hkv], p.max_pages, P, nullptr);
      const int n = ceil_div(listed_pages<P>(p, s, T, nullptr), kPages);
      if (first < at + n) {
        sh.seg = s;
        sh.tile = first - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  DecodeWalk<P> walk(p, count, sh.seg, sh.tile);

  if (warp == kDecLoad) {
    // ------------------------------------------------------------ loader
    if (lane == 0) prefetch_tensormap(&tmK);
    const uint64_t policy = l2_evict_first_policy();
    uint32_t kt = 0;
    bool ok = true;
    for (; ok && walk.more(); walk.next_segment()) {
      const int b = walk.seg / p.Hkv, h = walk.seg % p.Hkv, N = ceil_div(walk.T, P);
      const int32_t* list = p.lists ? p.lists + (size_t)walk.seg * p.max_pages : nullptr;
      const int32_t* bt = p.bt + (size_t)b * p.max_pages;
      const int run = walk.run(), end = min(walk.pages, (walk.tile + run) * kPages);
      // lane i looks up the list entries at + i, two batches ahead; their physical
      // pages, one batch ahead
      auto entry = [&](int i) {
        if (i >= end) return kNoPage;
        if (!list) return i;
        const int e = list[i];
        if (e >= 0 && e < N) return e;
        report(p.err, ASP_DEVERR_LIST_RANGE);
        return kNoPage;
      };
      auto physical = [&](int e) { return e == kNoPage ? -1 : bt[e]; };
      int at = walk.tile * kPages;
      int e_now = entry(at + lane), e_next = entry(at + 32 + lane);
      int ph_now = physical(e_now);
      for (int j = 0; j < run; ++j, ++kt) {
        if (j > 0 && j % kBatch == 0) {
          at += 32;
          e_now = e_next;
          ph_now = physical(e_now);
          e_next = entry(at + 32 + lane);
        }
        const int src = (j % kBatch) * kPages + (lane < kPages ? lane : 0);
        const int e = __shfl_sync(kFull, e_now, src), phys = __shfl_sync(kFull, ph_now, src);
        const bool have = lane < kPages && e != kNoPage;
        const bool good = have && phys >= 0 && phys < p.num_phys;
        if (have && !good) report(p.err, ASP_DEVERR_PAGE_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(kFull, good)) * (P * 128 * C::kHalves);
        const uint32_t st = kt % C::kStages;
        ok = __all_sync(kFull, mbar_wait(&sh.empty[st], ((kt / C::kStages) & 1) ^ 1));
        if (!ok) break;
        if (lane < kPages) sh.page[kt % kMetaRing][lane] = have && !good ? e | kNotMapped : e;
        __syncwarp();
        if (lane == 0) {
          if (bytes) mbar_arrive_expect_tx(&sh.full[st], bytes);
          else mbar_arrive(&sh.full[st]);
        }
        __syncwarp();
        if (good) {
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_2d_hint(ring + st * C::kTileBytes + hf * 16384 + lane * P * 128, &tmK, hf * 64,
                             (phys * p.Hkv + h) * P, &sh.full[st], policy);
        }
      }
    }
    if (!ok && lane == 0) {
      report(p.err, ASP_DEVERR_TIMEOUT);
      for (uint32_t t = kt > C::kStages ? kt - C::kStages : 0; t < kt; ++t)  // copies in flight end
        mbar_wait(&sh.full[t % C::kStages], (t / C::kStages) & 1);
    }
  } else if (warp == kDecQuery) {
    // ------------------------------------------------------------ queries
    // rows j, 8 + j, 16 + j: head j's query in three bf16 terms; rows of no head are 0
    uint32_t seg = 0;
    bool ok = true;
    for (; ok && walk.more(); walk.next_segment(), ++seg) {
      const int b = walk.seg / p.Hkv, h = walk.seg % p.Hkv, buf = seg & 1;
      const size_t q_row = (size_t)b * p.Hq + h * p.g;
      const uint32_t parity = ((seg >> 1) & 1) ^ 1;
      ok = __all_sync(kFull, mbar_wait(&sh.q_empty[buf], parity) &&
                                 mbar_wait(&sh.l_empty[buf], parity));
      if (!ok) break;
      if (lane < kMaxGroup) {
        const float l = lane < p.g ? p.lse[q_row + lane] : -INFINITY;
        sh.lse[buf][lane] = l == -INFINITY ? -INFINITY : -l * kLog2e;
      }
      uint8_t* tile = queries + buf * C::kQueryBytes;
      for (int i = lane; i < kMaxGroup * D / 8; i += 32) {  // 8 channels of one head
        const int j = i / (D / 8), ch = i % (D / 8);
        float f[8] = {};
        if (j < p.g) {
          const float4* src = reinterpret_cast<const float4*>(p.q + (q_row + j) * D + ch * 8);
          const float4 a = src[0], bb = src[1];
          f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
          f[4] = bb.x, f[5] = bb.y, f[6] = bb.z, f[7] = bb.w;
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const int r = part * 8 + j;
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[k] = pack_bf16(f[2 * k], f[2 * k + 1]);
            const float2 back = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&y[k]));
            f[2 * k] -= back.x;
            f[2 * k + 1] -= back.y;
          }
          *reinterpret_cast<uint4*>(tile + (ch / 8) * (kQueryRows * 128) + r * 128 +
                                    (((ch % 8) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[buf]);
    }
    if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
  } else if (warp == kDecMma) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kDesc = mma_desc(kTileKeys, kQueryCols, false);
    const uint32_t r0 = uniform(smem_u32(ring)), q0 = uniform(smem_u32(queries));
    const uint32_t tm = uniform(tmem);
    uint32_t kt = 0, seg = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(kFull, mbar_wait(bar, parity)) != 0;
    };
    for (; ok && uniform(walk.more()); walk.next_segment(), ++seg) {
      const int buf = seg & 1, run = uniform(walk.run());
      ok = wait(&sh.q_full[buf], (seg >> 1) & 1);
      for (int j = 0; ok && j < run; ++j, ++kt) {
        const uint32_t st = kt % C::kStages, sb = kt % kDecBufs;
        ok = wait(&sh.s_empty[sb], ((kt / kDecBufs) & 1) ^ 1) &&
             wait(&sh.full[st], (kt / C::kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = smem_desc(r0 + st * C::kTileBytes, 16);
        const uint64_t b = smem_desc(q0 + buf * C::kQueryBytes, 16);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tm + sb * kQueryCols, a + (((k / 4) * 16384 + (k % 4) * 32) >> 4),
                   b + (((k / 4) * (kQueryRows * 128) + (k % 4) * 32) >> 4), kDesc, k > 0);
          mma_commit(&sh.s_full[sb]);
          mma_commit(&sh.empty[st]);
        }
      }
      if (elect_one()) mma_commit(&sh.q_empty[buf]);
    }
    if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
    if (elect_one()) mma_commit(&sh.drain);  // no arrival is still on its way when the CTA ends
    mbar_wait(&sh.drain, 0);
  } else {
    // ------------------------------------------------------------ sums
    const uint32_t lanes = (uint32_t)warp << 21;
    const float c = p.scale_log2;
    uint32_t kt = 0, seg = 0;
    bool ok = true;
    for (; ok && walk.more(); walk.next_segment(), ++seg) {
      const int buf = seg & 1, run = walk.run();
      const size_t base = (size_t)walk.seg * p.max_pages * P;
      float nl[kMaxGroup];
      for (int j = 0; j < run; ++j, ++kt) {
        const uint32_t sb = kt % kDecBufs;
        ok = __all_sync(kFull, mbar_wait(&sh.s_full[sb], (kt / kDecBufs) & 1));
        if (!ok) break;
        const int e = sh.page[kt % kMetaRing][tid / P];
        const int slot = (e & ~kNotMapped) * P + tid % P;
        const bool mine = e != kNoPage && slot < walk.T;
        // lists: the weight carried over is there already
        float before = 0.f;
        if (mine)
          before = p.lists ? p.w_out[base + slot]
                           : weight_before(p.w_in, p.decay, base + slot, slot, walk.T - 1);
        if (j == 0) {
#pragma unroll
          for (int i = 0; i < kMaxGroup; ++i) nl[i] = sh.lse[buf][i];
        }
        __syncwarp();
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32(tmem + lanes + sb * kQueryCols, s);
        tmem_wait_ld(s);
        tc_fence_before();
        mbar_arrive(&sh.s_empty[sb]);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxGroup; ++i) {
          const float dot = __uint_as_float(s[i]) +
                            (__uint_as_float(s[8 + i]) + __uint_as_float(s[16 + i]));
          if (nl[i] != -INFINITY) sum += ex2(fmaf(dot, c, nl[i]));
        }
        if (mine) p.w_out[base + slot] = before + (e & kNotMapped ? 0.f : sum);
      }
      if (ok) mbar_arrive(&sh.l_empty[buf]);
    }
    if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == kDecMma) tmem_free(tmem, kDecCols);
}

// w_out = decay * w_in over every slot of every segment (0 for the decoded
// token), before the listed pages' weights are added.
__global__ void __launch_bounds__(256) carry_weights_kernel(const DecodeParams p, int P) {
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int seg = blockIdx.y, b = seg / p.Hkv;
  const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, nullptr);
  const size_t base = (size_t)seg * p.max_pages * P;
  for (int s = 4 * (blockIdx.x * 256 + threadIdx.x); s < T; s += 4 * 256 * gridDim.x) {
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.w_in) w = *reinterpret_cast<const float4*>(p.w_in + base + s);
    const float y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s + i < T) p.w_out[base + s + i] = s + i < T - 1 ? p.decay * y[i] : 0.f;
  }
}

template <int D, int P>
cudaError_t launch_decode_t(const WeightArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  const unsigned long long cache_rows =
      (unsigned long long)kv.num_phys_pages * kv.num_kv_heads * P;
  DecodeParams p{a.q_f32, a.lists, a.lens, a.lse, a.w_in, a.w_out, kv.block_table, kv.seq_lens,
                 a.err, kv.batch, kv.num_q_heads, kv.num_kv_heads,
                 kv.num_q_heads / kv.num_kv_heads, kv.max_pages, kv.num_phys_pages,
                 a.sm_scale * kLog2e, a.decay};
  cudaError_t e;
  if (a.lists) {
    if ((e = set_max_dynamic_smem((const void*)carry_weights_kernel, 0)) != cudaSuccess) return e;
    const int blocks = ceil_div(kv.max_pages * P, 1024);  // < 2^26 slots
    const dim3 grid(min(blocks, 1024), kv.batch * kv.num_kv_heads);
    if ((e = launch_pdl(carry_weights_kernel, grid, dim3(256), 0, stream, p, P)) != cudaSuccess)
      return e;
  }
  CUtensorMap tk;
  if ((e = encode_bf16_2d_swizzled(&tk, kv.k_cache, D, cache_rows, 64, P)) != cudaSuccess) return e;
  constexpr size_t smem = decode_smem<D>();
  if ((e = set_max_dynamic_smem((const void*)decode_weights_kernel<D, P>, (int)smem)) != cudaSuccess)
    return e;
  return launch_pdl(decode_weights_kernel<D, P>, dim3(2 * a.num_sms), dim3(kDecThreads), smem, stream,
                    tk, p);
}

}  // namespace

cudaError_t launch_chunk_weights(const WeightArgs& a, cudaStream_t stream) {
  const int d = a.kv->head_dim, P = a.kv->page_size;
  if (d == 128 && P == 16) return launch_chunk_t<128, 16>(a, stream);
  if (d == 128 && P == 32) return launch_chunk_t<128, 32>(a, stream);
  if (d == 128 && P == 64) return launch_chunk_t<128, 64>(a, stream);
  if (d == 64 && P == 16) return launch_chunk_t<64, 16>(a, stream);
  if (d == 64 && P == 32) return launch_chunk_t<64, 32>(a, stream);
  if (d == 64 && P == 64) return launch_chunk_t<64, 64>(a, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_weights(const WeightArgs& a, cudaStream_t stream) {
  const int d = a.kv->head_dim, P = a.kv->page_size;
  if (d == 128 && P == 16) return launch_decode_t<128, 16>(a, stream);
  if (d == 128 && P == 32) return launch_decode_t<128, 32>(a, stream);
  if (d == 128 && P == 64) return launch_decode_t<128, 64>(a, stream);
  if (d == 64 && P == 16) return launch_decode_t<64, 16>(a, stream);
  if (d == 64 && P == 32) return launch_decode_t<64, 32>(a, stream);
  if (d == 64 && P == 64) return launch_decode_t<64, 64>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace asp
