// chunk_attention.cu - causal attention of a chunk of new tokens over the
// paged cache: out = sum_s softmax_s(c q.k_s) v_s over the slots s <= t.
//
// One persistent CTA per SM takes an equal share of the call's units (256 query
// rows against 128 keys, chunk_plan.cuh). Per unit, on the tensor cores:
//   S = Q K^T   two tiles of [128 rows x 128 keys], fp32 in tensor memory
//   P = exp2(c S - m) rounded to bf16, back into tensor memory over S
//   O += P V    [128 rows x d], fp32 in tensor memory
// Roles: one warp loads (TMA, page by page, into a ring of 128-key tiles), one
// thread issues the products, and one warpgroup per tile of rows owns its
// softmax: a thread holds a whole row, so maxima and sums need no exchange. The
// two tiles alternate: while one is in its softmax the other's products run.
// Query heads of one KV head share its keys: rows are (token, head of the group).
//
// Measured (d = 128, 32 query and 8 KV heads, bf16; cuBLAS on the same GPU does 1.87
// PFLOP/s in bursts, 1.67 for seconds): 2048 rows over 32768 tokens in 0.67 ms, 1.58
// PFLOP/s, and 0.77 ms in a long loop, where the GPU's power limit takes the clock from
// 1.9 to 1.7 GHz; prompts of 8k in 0.59 ms, 1.41 PFLOP/s; five rows a request over
// 8 x 65536 tokens (64 heads, pages of 64) in 0.27 ms, 6.4 TB/s. A unit takes 2750 cycles,
// the products alone 2048 (ncu: tensor pipe 71% active); the rest is the tensor memory's
// port, which the softmax's reads and writes share with the products, and some 150 cycles a
// tile between a probability's arrival and its product. What brought it there:
//   - operands in uniform registers (the issuing warp stays together): 906 -> 738 us
//   - a V page in one TMA box of both halves (the boxes, not the bytes, bound the loads of
//     16-token pages), P handed over in halves: 738 -> 694
//   - one thread walks the plan, code that runs once an item kept short: 694 -> 675, and
//     694 -> 600 for the 8k prompts, whose items are short
// At d = 64 a unit has half the products and the same softmax: 564 us, 0.95 PFLOP/s, with the
// tensor pipe 41%, the exponentials' 41% and the issue slots 47% busy. No one unit is full; a
// tile's chain of waits, loads and exponentials is what the products stand still for.
// Tried and dropped: the first half's exponentials against the old maximum while the new
// one is found (675 -> 710, more instructions); one lane polling barriers (675 -> 825).
//
// The running maximum m moves only when a tile's maximum is more than 2^8 above
// it: until then the exponentials stay below 2^8, the products need no
// correction, and O stays in tensor memory untouched. Sums are of the unrounded
// exponentials in fp32.
//
// An item whose units lie in several CTAs leaves (m, l, O) partials; a second,
// small kernel joins them in order. Two launches, no atomics, no CTA waits for
// another; the result does not depend on timing.
#include "chunk_plan.cuh"
#include "tc.cuh"

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// Two softmax warpgroups; loader, issuer, the warp that hands out pieces and an idle
// one make up the third. 384 threads start with 168 registers; a row of 128 logits wants more,
// so the third warpgroup gives up 96 a thread and the others take 48:
// 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsRest = 72;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kTaskWarp = 10;
constexpr float kMoveLog2 = 8.0f;     // the maximum moves when it grows by more than 2^8
constexpr int kPageMasks = 8;         // units whose page masks are kept at once
constexpr uint32_t kTmemCols = 512;   // S of two tiles (128 each), O of two tiles (128 each)

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;  // 128 rows x d bf16, swizzled halves
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr size_t kSmem = 1024 + (2 + kStages) * (size_t)kTileBytes + 1024;
};

struct Shared {
  uint64_t q_full, q_empty, drain;
  uint64_t full[8], empty[8];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];
  ChunkTasks tasks;
  ChunkStart start;
  long long scratch[kThreads / 32];
  uint32_t page_mask[kPageMasks];
  uint32_t tmem;
};
static_assert(sizeof(Shared) <= 1024, "the tail of the dynamic shared memory");

struct Params {
  ChunkDims c;
  const int32_t* bt;
  uint16_t* out;
  float* lse;
  ChunkJoin* joins;
  float* partials;
  uint32_t* err;
  int Hq, num_phys;
  float scale, scale_log2;
};

template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg<D>;
  constexpr int kPages = kTileKeys / P;  // pages of a key tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_tiles = smem;                         // [2][halves][128 rows x 128 B]
  // K: [stages][halves][128 keys x 128 B], V: [stages][pages][halves][P keys x 128 B]
  uint8_t* ring = smem + 2 * C::kTileBytes;
  Shared& sh = *reinterpret_cast<Shared*>(ring + C::kStages * C::kTileBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], 4);  // the tile's warps
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
    }
    chunk_tasks_init(sh.tasks, 10);  // loader, issuer, eight softmax warps
    mbar_fence_init();
  }
  if (tid == kLoadWarp * 32) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now may the next kernel start: its CTAs find this one's tensor memory taken.
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const uint32_t tmem = sh.tmem;
  chunk_plan<RowCut>(p.c, &sh.start, sh.scratch, p.err);
  const int g = p.c.g, tile_tokens = kTileRows >> p.c.lg;
  ChunkReader reader(sh.tasks);
  ChunkTask task;  // x: units of its two tiles of rows, its first token, its end

  if (warp > kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (tid == kTaskWarp * 32) {
      // ---------------------------------------------------------- pieces
      const bool ok = chunk_hand_out<RowCut>(
          sh.tasks, p.c, sh.start, p.joins + blockIdx.x,
          [&](const ChunkWalk<RowCut>& w, ChunkTask& t) {
            t.x[2] = w.item * 2 * tile_tokens;
            t.x[3] = min(w.r.n, t.x[2] + 2 * tile_tokens);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int end = min(t.x[3], t.x[2] + (i + 1) * tile_tokens);
              t.x[i] = end > t.x[2] + i * tile_tokens
                           ? max(0, min(w.u1, RowCut::units_to(w.r, end - 1)) - w.u0)
                           : 0;
            }
          });
      if (!ok) report(p.err, ASP_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loader
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    uint32_t tile = 0;   // K and V tiles loaded so far
    uint32_t piece = 0;
    bool ok = true;
    uint32_t masks = 0;
    for (; ok && reader.next(task); ++piece) {
      const int n = max(task.x[0], task.x[1]);
      const bool two = task.x[3] - task.x[2] > tile_tokens;
      ok = __all_sync(kFull, mbar_wait(&sh.q_empty, (piece & 1) ^ 1));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full, (two ? 2 : 1) * C::kTileBytes);
        for (int t = 0; t < (two ? 2 : 1); ++t)
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(q_tiles + t * C::kTileBytes + hf * 16384, &tmQ, hf * 64, task.h * g,
                        task.row0 + task.x[2] + t * tile_tokens, &sh.q_full);
      }
      const int n_pages = ceil_div(task.T, P);
      const int32_t* bt = p.bt + (size_t)task.b * p.c.max_pages;
      // the tile's physical pages, read one tile ahead
      auto look_up = [&](int j) {
        const int page = (task.u0 + j) * kPages + lane;
        return lane < kPages && page < n_pages ? bt[page] : 0;
      };
      int next = look_up(0);
      for (int j = 0; j < n; ++j) {
        const bool have = lane < kPages && (task.u0 + j) * kPages + lane < n_pages;
        const int phys = next;
        next = look_up(j + 1);
        const bool good = have && phys >= 0 && phys < p.num_phys;
        if (have && !good) report(p.err, ASP_DEVERR_PAGE_RANGE);
        const uint32_t mask = __ballot_sync(kFull, good);
        const int y = (phys * p.c.Hkv + task.h) * P;
        for (int kv = 0; kv < 2; ++kv, ++tile) {
          const int st = tile % C::kStages;
          ok = __all_sync(kFull, mbar_wait(&sh.empty[st], ((tile / C::kStages) & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) {
            if (kv == 0) sh.page_mask[masks % kPageMasks] = mask;
            const uint32_t bytes = __popc(mask) * (P * 128 * C::kHalves);
            if (bytes) mbar_arrive_expect_tx(&sh.full[st], bytes);
            else mbar_arrive(&sh.full[st]);
          }
          __syncwarp();
          uint8_t* dst = ring + st * C::kTileBytes;
          if (good && kv == 0) {
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
              tma_load_2d(dst + hf * 16384 + lane * P * 128, &tmK, hf * 64, y, &sh.full[st]);
          } else if (good) {
            tma_load_3d(dst + lane * C::kHalves * P * 128, &tmV, 0, y, 0, &sh.full[st]);
          }
        }
        if (!ok) break;
        ++masks;
      }
    }
    if (!(ok && reader.ok) && lane == 0) {
      report(p.err, ASP_DEVERR_TIMEOUT);
      // copies in flight end before the CTA does
      for (uint32_t t = tile > C::kStages ? tile - C::kStages : 0; t < tile; ++t)
        mbar_wait(&sh.full[t % C::kStages], (t / C::kStages) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    constexpr uint32_t kDescS = mma_desc(128, kTileKeys, false);
    constexpr uint32_t kDescO = mma_desc(128, D, true);
    const uint32_t q0 = uniform(smem_u32(q_tiles)), r0 = uniform(smem_u32(ring));
    const uint32_t tm = uniform(tmem);
    uint32_t tile = 0, piece = 0, np[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(kFull, mbar_wait(bar, parity)) != 0;
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) mma_commit(bar);
    };
    auto product_s = [&](int t, uint32_t st) {
      const uint64_t a = smem_desc(q0 + t * C::kTileBytes, 16);
      const uint64_t b = smem_desc(r0 + st * C::kTileBytes, 16);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k / 4) * 16384 + (k % 4) * 32) >> 4;
          mma_ss(tm + t * 128, a + off, b + off, kDescS, k > 0);
        }
        mma_commit(&sh.s_full[t]);
      }
    };
    // keys 64 hf .. 64 hf + 63 of the tile
    auto product_o = [&](int t, uint32_t st, int hf, bool add) {
      const uint64_t b = smem_desc(r0 + st * C::kTileBytes, P * 128);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < kTileKeys / 32; ++i) {
          const int k = hf * (kTileKeys / 32) + i;
          const uint32_t off = k * 16 / P * (C::kHalves * P * 128) + k * 16 % P * 128;
          mma_ts(tm + 256 + t * 128, tm + t * 128 + k * 8, b + (off >> 4), kDescO, add || i > 0);
        }
      }
    };
    for (; ok && uniform(reader.next(task)); ++piece) {
      const int nt[2] = {uniform(task.x[0]), uniform(task.x[1])};
      const int n = max(nt[0], nt[1]);
      uint32_t st = tile % C::kStages;
      ok = wait(&sh.q_full, piece & 1) && wait(&sh.full[st], (tile / C::kStages) & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (nt[t] > 0) product_s(t, st);
      commit(&sh.empty[st]);
      if (n == 1) commit(&sh.q_empty);
      for (int j = 0; j < n; ++j, tile += 2) {
        const uint32_t sv = (tile + 1) % C::kStages, sk = (tile + 2) % C::kStages;
        ok = wait(&sh.full[sv], ((tile + 1) / C::kStages) & 1);
        bool k_there = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || j >= nt[t]) continue;
          ok = wait(&sh.p_half[t], np[t] & 1);
          if (!ok) continue;
          tc_fence_after();
          product_o(t, sv, 0, j > 0);
          ok = wait(&sh.p_full[t], np[t] & 1);
          ++np[t];
          if (ok && j + 1 < n && !k_there)
            k_there = ok = wait(&sh.full[sk], ((tile + 2) / C::kStages) & 1);
          if (!ok) continue;
          tc_fence_after();
          product_o(t, sv, 1, true);
          if (j + 1 < nt[t]) product_s(t, sk);
          else commit(&sh.o_full[t]);
        }
        if (!ok) break;
        commit(&sh.empty[sv]);
        if (j + 1 < n) commit(&sh.empty[sk]);
        if (j + 2 == n) commit(&sh.q_empty);
      }
    }
    if (!(ok && reader.ok) && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
    commit(&sh.drain);  // no arrival is still on its way when the CTA ends
    mbar_wait(&sh.drain, 0);
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's lanes of tensor memory
    const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + 256 + t * 128 + lanes;
    const float c = p.scale_log2;
    uint32_t phase_s = 0, phase_o = 0, units_seen = 0;
    bool ok = true;
    const int row_tok = row >> p.c.lg, row_head = row & (g - 1);
    while (ok && reader.next(task)) {
      const int n = t == 0 ? task.x[0] : task.x[1];
      const int tok = task.x[2] + t * tile_tokens + row_tok;
      // rows past the item's last take any slot that keeps them off the masked path
      const bool mine = tok < task.x[3];
      const int pos = mine ? task.T - task.n + tok : task.T - 1;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int key0 = (task.u0 + j) * kTileKeys;
        ok = __all_sync(kFull, mbar_wait(&sh.s_full[t], phase_s & 1));
        if (!ok) break;
        ++phase_s;
        tc_fence_after();
        const uint32_t pages = sh.page_mask[(units_seen + j) % kPageMasks];
        // keys past the request's tokens, or of a page that is not there
        const bool holes = pages != (1u << kPages) - 1;
        if (__any_sync(kFull, pos < key0 + kTileKeys - 1) || holes) {
          // Masked keys become -inf in tensor memory, 32 at a time: few units need it, and
          // a short loop costs them less than long straight code would (it is fetched anew).
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int lim = pos - key0 - 32 * i;  // the last key of the 32 that the row sees
            uint32_t see = lim >= 31 ? ~0u : lim < 0 ? 0u : (2u << lim) - 1;
            if (P == 16)
              see &= (pages >> (2 * i) & 1 ? 0xffffu : 0u) |
                     (pages >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
            else
              see &= pages >> (32 * i / P) & 1 ? ~0u : 0u;
            if (__all_sync(kFull, see == ~0u)) continue;
            uint32_t x[32];
            tmem_ld32(s_at + 32 * i, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see >> e & 1)) x[e] = 0xff800000u;  // -inf
            tmem_st32(s_at + 32 * i, x);
          }
          tmem_wait_st();
          if (holes || key0 + kTileKeys > task.T) {
            // their V rows may hold anything: zero times it has to stay zero
            const uint32_t tv = 2 * (units_seen + j) + 1;
            ok = __all_sync(kFull, mbar_wait(&sh.full[tv % C::kStages], (tv / C::kStages) & 1));
            if (!ok) break;
            if (key0 + row >= task.T || !((pages >> (row / P)) & 1)) {
              uint8_t* v = ring + (tv % C::kStages) * C::kTileBytes +
                           row / P * (C::kHalves * P * 128) + row % P * 128;
#pragma unroll 1
              for (int e = 0; e < 8 * C::kHalves; ++e)
                *reinterpret_cast<uint4*>(v + (e / 8) * (P * 128) + (e % 8) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            fence_proxy_async_smem();
          }
        }
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_wait_ld(s[i]);
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2)
            mx[i] = max3(mx[i], __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (j == 0) {
          m = top;
        } else {
          const bool moves = (top - m) * c > kMoveLog2;
          if (__any_sync(kFull, moves)) {
            // the product that added to O before this S is done: s_full came after it
            const float f = moves ? ex2((m - top) * c) : 1.0f;
            if (moves) m = top;
            l *= f;
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t o[32];
              tmem_ld32(o_at + 32 * i, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_at + 32 * i, o);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // 16 exponentials at a time; the ones before are summed and packed while they run
        auto exponentials = [&](int q) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            uint32_t* x = &s[q / 2][(q & 1) * 16 + e];
            const float2 y =
                fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, mc2);
            x[0] = __float_as_uint(ex2(y.x));
            x[1] = __float_as_uint(ex2(y.y));
          }
        };
        exponentials(0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t pk[32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (4 * i + q < 7) exponentials(4 * i + q + 1);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const uint32_t* x = &s[(4 * i + q) / 2][(q & 1) * 16 + e];
              const float2 y = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
              sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], y);
              pk[q * 8 + e / 2] = pack_bf16(y.x, y.y);
            }
          }
          tmem_st32(s_at + 32 * i, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(i == 0 ? &sh.p_half[t] : &sh.p_full[t]);
          __syncwarp();
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      units_seen += max(task.x[0], task.x[1]);
      // ---- the piece's end: the whole item goes out, a part of it into the workspace
      if (n > 0) {
        ok = __all_sync(kFull, mbar_wait(&sh.o_full[t], phase_o & 1));
        if (!ok) break;
        ++phase_o;
        tc_fence_after();
      }
      const size_t at = (size_t)(task.row0 + tok) * p.Hq + task.h * g + row_head;
      if (task.whole) {
        const float inv = l > 0.f ? 1.0f / l : l;  // a NaN sum stays NaN, an empty row gives 0
        // Four lanes exchange 16-byte pieces so that a row's 64 bytes leave together: a
        // thread's own row, 16 bytes a store, would touch a cache line for every lane.
        const int base = lane & ~3, q = lane & 3;
        uint16_t* dst[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t there = __shfl_sync(
              kFull, mine ? reinterpret_cast<uint64_t>(p.out + at * D) : 0ull, base + k);
          dst[k] = reinterpret_cast<uint16_t*>(there);
        }
#pragma unroll 1
        for (int i = 0; i < D / 32 && n > 0; ++i) {
          uint32_t o[32], y[4][4];  // y[piece][word]
          tmem_ld32(o_at + 32 * i, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[e / 4][e % 4] = pack_bf16(__uint_as_float(o[2 * e]) * inv,
                                        __uint_as_float(o[2 * e + 1]) * inv);
          // 4 x 4 transpose: lane q then holds piece q of rows base .. base + 3
#pragma unroll
          for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int step = 1; step < 4; step <<= 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k & step) continue;
                const bool up = q & step;
                const uint32_t give = up ? y[k][w] : y[k | step][w];
                const uint32_t got = __shfl_xor_sync(kFull, give, step);
                if (up) y[k][w] = got; else y[k | step][w] = got;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (dst[k])
              *reinterpret_cast<uint4*>(dst[k] + 32 * i + 8 * q) =
                  make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
          __syncwarp();
        }
        if (mine) p.lse[at] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
      } else {
        // [m | l | O as D / 4 columns of four, each kChunkRows rows]
        const int slot = 2 * blockIdx.x + (task.u0 == 0 ? 1 : 0);
        const int r = t * 128 + row;
        float* part = p.partials + (size_t)slot * chunk_slot_floats(D);
        part[r] = mine ? m * c : -INFINITY;
        part[kChunkRows + r] = l;
        float4* dst = reinterpret_cast<float4*>(part + 2 * kChunkRows) + r;
#pragma unroll 1
        for (int i = 0; i < D / 32 && n > 0; ++i) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * i, o);
          tmem_wait_ld(o);
          if (mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(8 * i + e) * kChunkRows] =
                  make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                              __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
          __syncwarp();
        }
      }
      tc_fence_before();  // the next piece's first product writes O after the next P arrives
    }
    if (!(ok && reader.ok) && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

// Joins the pieces of the item that CTA blockIdx.x began, 32 of its rows a block:
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. A lane owns a row, a warp some of
// its columns, four at a time; the pieces are added in order, eight loads in flight. The
// rows leave through shared memory, so that they are written as rows.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const Params p) {
  constexpr int kInFlight = 8, kCols = D / 4 / 8;  // columns of four a warp
  constexpr int kPitch = D + 8;                    // of a row in shared memory
  __shared__ __align__(16) uint16_t tile[32 * kPitch];
  pdl_launch_dependents();
  pdl_wait_predecessor();
  ChunkJoin jn;
  ChunkRequest r;
  if (!chunk_join<RowCut>(p.c, p.joins, p.err, jn, r)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = p.c.g, row = blockIdx.y * 32 + lane;
  const int tok0 = jn.item * (kChunkRows >> p.c.lg);
  const size_t slot_floats = chunk_slot_floats(D);
  const float* first = p.partials + (size_t)(2 * blockIdx.x + 1) * slot_floats + row;
  const float* rest = p.partials + (size_t)(2 * blockIdx.x) * slot_floats + row;
  auto part = [&](int k) { return k == 0 ? first : rest + (size_t)(2 * k) * slot_floats; };
  float M = -INFINITY;
  for (int k = 0; k < jn.pieces; k += kInFlight) {
    float m[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) m[u] = k + u < jn.pieces ? *part(k + u) : -INFINITY;
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) M = fmaxf(M, m[u]);
  }
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kStep = kInFlight / kCols;
  for (int k = 0; k < jn.pieces; k += kStep) {
    float w[kStep], l[kStep];
    float4 o[kStep][kCols];
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      w[u] = -INFINITY;
      l[u] = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k + u >= jn.pieces) continue;
      const float* q = part(k + u);
      w[u] = *q;
      l[u] = q[kChunkRows];
      if (w[u] == -INFINITY) continue;  // none of its keys count for this row: no O was written
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        o[u][i] = *reinterpret_cast<const float4*>(
            q - row + 2 * kChunkRows + 4 * ((size_t)(warp * kCols + i) * kChunkRows + row));
    }
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      const float f = ex2(w[u] - ref);  // 0 where there is nothing
      L = fmaf(f, l[u], L);
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        acc[i].x = fmaf(f, o[u][i].x, acc[i].x);
        acc[i].y = fmaf(f, o[u][i].y, acc[i].y);
        acc[i].z = fmaf(f, o[u][i].z, acc[i].z);
        acc[i].w = fmaf(f, o[u][i].w, acc[i].w);
      }
    }
  }
  const float inv = L > 0.f ? 1.0f / L : L;
#pragma unroll
  for (int i = 0; i < kCols; ++i)
    *reinterpret_cast<uint2*>(tile + lane * kPitch + 4 * (warp * kCols + i)) =
        make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
  if (warp == 0 && tok0 + (row >> p.c.lg) < r.n)
    p.lse[(size_t)(r.row0 + tok0 + (row >> p.c.lg)) * p.Hq + jn.h * g + (row & (g - 1))] =
        L == 0.f ? -INFINITY : M * 0.69314718055994530942f + logf(L);
  __syncthreads();
  constexpr int kPieces = D / 8;  // of 16 bytes
  for (int i = threadIdx.x; i < 32 * kPieces; i += 256) {
    const int rr = blockIdx.y * 32 + i / kPieces;
    if (tok0 + (rr >> p.c.lg) >= r.n) break;
    const size_t at = (size_t)(r.row0 + tok0 + (rr >> p.c.lg)) * p.Hq + jn.h * g + (rr & (g - 1));
    *reinterpret_cast<uint4*>(p.out + at * D + 8 * (i % kPieces)) =
        *reinterpret_cast<const uint4*>(tile + i / kPieces * kPitch + 8 * (i % kPieces));
  }
}

template <int D, int P>
cudaError_t launch_t(const ChunkAttentionArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  const asp_paged_kv& kv = *a.kv;
  const int g = kv.num_q_heads / kv.num_kv_heads;
  const unsigned long long rows = (unsigned long long)kv.num_phys_pages * kv.num_kv_heads * P;
  CUtensorMap tq, tk, tv;
  cudaError_t e = encode_bf16_3d_swizzled(
      &tq, a.q, {D, (unsigned long long)kv.num_q_heads, (unsigned long long)a.num_tokens},
      {2 * D, 2ull * D * kv.num_q_heads}, {64, (unsigned)g, (unsigned)(kTileRows / g)});
  if (e != cudaSuccess) return e;
  if ((e = encode_bf16_2d_swizzled(&tk, kv.k_cache, D, rows, 64, P)) != cudaSuccess) return e;
  // a V page in one box: [half][P rows][64 channels]
  if ((e = encode_bf16_3d_swizzled(&tv, kv.v_cache, {64, rows, D / 64}, {2 * D, 128},
                                   {64, (unsigned)P, (unsigned)(D / 64)})) != cudaSuccess)
    return e;
  Params p{{a.q_offsets, kv.seq_lens, kv.batch, kv.num_kv_heads, g, chunk_log2(g), kv.max_pages, P, a.num_tokens,
            chunk_inverse(a.num_sms)},
           kv.block_table, a.out, a.lse, a.joins, a.partials, a.err, kv.num_q_heads,
           kv.num_phys_pages, a.sm_scale, a.sm_scale * 1.4426950408889634f};
  if ((e = set_max_dynamic_smem((const void*)chunk_attention_kernel<D, P>, (int)C::kSmem)) !=
      cudaSuccess)
    return e;
  if ((e = set_max_dynamic_smem((const void*)chunk_join_kernel<D>, 0)) != cudaSuccess) return e;
  e = launch_pdl(chunk_attention_kernel<D, P>, dim3(a.num_sms), dim3(kThreads), C::kSmem, stream, tq,
                 tk, tv, p);
  if (e != cudaSuccess) return e;
  // an item has no more rows than the call
  const long long item_rows = min((long long)a.num_tokens * g, (long long)kChunkRows);
  return launch_pdl(chunk_join_kernel<D>, dim3(a.num_sms, (unsigned)((item_rows + 31) / 32)), dim3(256),
                    0, stream, p);
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
