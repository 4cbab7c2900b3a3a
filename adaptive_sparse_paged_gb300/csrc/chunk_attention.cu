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

#include <type_traits>

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// Two softmax warpgroups; loader, issuer and two idle warps that make up the
// third. 384 threads start with 168 registers; a row of 128 logits wants more,
// so the third warpgroup gives up 96 a thread and the others take 48:
// 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsRest = 72;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr float kMoveLog2 = 8.0f;     // the maximum moves when it grows by more than 2^8
constexpr int kPageMasks = 8;         // units whose page masks are kept at once
constexpr uint32_t kTmemCols = 512;   // S of two tiles (128 each), O of two tiles (128 each)

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * 128 * 128;  // 128 rows x d bf16, swizzled halves
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr size_t kSmem = 1024 + (2 + kStages) * (size_t)kTileBytes + 512;
};

struct Shared {
  uint64_t q_full, q_empty, drain;
  uint64_t full[8], empty[8];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];
  ChunkStart start;
  long long scratch[kThreads / 32];
  uint32_t page_mask[kPageMasks];
  uint32_t tmem;
  int failed;
};
static_assert(sizeof(Shared) <= 512, "the tail of the dynamic shared memory");

// The current piece's tokens of the chunk, [tok0, last), and the units that its
// two tiles of rows need.
struct Piece {
  int tok0, last, n[2];
  __device__ __forceinline__ Piece(const ChunkWalk<RowCut>& w, int tile_tokens) {
    tok0 = w.item * 2 * tile_tokens;
    last = min(w.r.n, tok0 + 2 * tile_tokens);
    for (int t = 0; t < 2; ++t) {
      const int end = min(last, tok0 + (t + 1) * tile_tokens);
      n[t] = end > tok0 + t * tile_tokens
                 ? max(0, min(w.u1, RowCut::units_to(w.r, end - 1)) - w.u0)
                 : 0;
    }
  }
};

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
    mbar_fence_init();
    sh.failed = 0;
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
  ChunkWalk<RowCut> walk(p.c, sh.start);
  const int g = p.c.g, tile_tokens = kTileRows / g;
  auto fail = [&] {
    report(p.err, ASP_DEVERR_TIMEOUT);
    *(volatile int*)&sh.failed = 1;
  };

  if (warp > kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loader
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (lane == 0) {
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
    }
    uint32_t tile = 0;   // K and V tiles loaded so far
    uint32_t piece = 0;
    bool ok = true;
    uint32_t masks = 0;
    for (; ok && walk.more(); walk.next(), ++piece) {
      const Piece pc(walk, tile_tokens);
      const int n = max(pc.n[0], pc.n[1]);
      const bool two = pc.last - pc.tok0 > tile_tokens;
      ok = __all_sync(kFull, mbar_wait(&sh.q_empty, (piece & 1) ^ 1));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full, (two ? 2 : 1) * C::kTileBytes);
        for (int t = 0; t < (two ? 2 : 1); ++t)
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(q_tiles + t * C::kTileBytes + hf * 16384, &tmQ, hf * 64, walk.h * g,
                        walk.r.row0 + pc.tok0 + t * tile_tokens, &sh.q_full);
      }
      const int n_pages = ceil_div(walk.r.T, P);
      const int32_t* bt = p.bt + (size_t)walk.b * p.c.max_pages;
      // the tile's physical pages, read one tile ahead
      auto look_up = [&](int j) {
        const int page = (walk.u0 + j) * kPages + lane;
        return lane < kPages && page < n_pages ? bt[page] : 0;
      };
      int next = look_up(0);
      for (int j = 0; j < n; ++j) {
        const bool have = lane < kPages && (walk.u0 + j) * kPages + lane < n_pages;
        const int phys = next;
        next = look_up(j + 1);
        const bool good = have && phys >= 0 && phys < p.num_phys;
        if (have && !good) report(p.err, ASP_DEVERR_PAGE_RANGE);
        const uint32_t mask = __ballot_sync(kFull, good);
        const int y = (phys * p.c.Hkv + walk.h) * P;
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
    if (!ok && lane == 0) {
      fail();
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
    for (; ok && uniform(walk.more()); walk.next(), ++piece) {
      const Piece pc(walk, tile_tokens);
      const int nt[2] = {uniform(pc.n[0]), uniform(pc.n[1])};
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
    if (!ok && lane == 0) fail();
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
    if (tid == 0) p.joins[blockIdx.x].pieces = 0;
    for (; ok && walk.more(); walk.next()) {
      const Piece pc(walk, tile_tokens);
      const int n = pc.n[t];
      const int tok = pc.tok0 + t * tile_tokens + row / g;
      // rows past the item's last take any slot that keeps them off the masked path
      const bool mine = tok < pc.last;
      const int pos = mine ? walk.r.T - walk.r.n + tok : walk.r.T - 1;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int key0 = (walk.u0 + j) * kTileKeys;
        ok = __all_sync(kFull, mbar_wait(&sh.s_full[t], phase_s & 1));
        if (!ok) break;
        ++phase_s;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_wait_ld(s[i]);
        const uint32_t pages = sh.page_mask[(units_seen + j) % kPageMasks];
        // keys past the request's tokens, or of a page that is not there
        const bool holes = pages != (1u << kPages) - 1;
        if (__any_sync(kFull, pos < key0 + kTileKeys - 1) || holes) {
          const int lim = pos - key0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int k = 32 * i + e;
              if (k > lim || !((pages >> (k / P)) & 1)) s[i][e] = 0xff800000u;  // -inf
            }
          if (holes || key0 + kTileKeys > walk.r.T) {
            // their V rows may hold anything: zero times it has to stay zero
            const uint32_t tv = 2 * (units_seen + j) + 1;
            ok = __all_sync(kFull, mbar_wait(&sh.full[tv % C::kStages], (tv / C::kStages) & 1));
            if (!ok) break;
            if (key0 + row >= walk.r.T || !((pages >> (row / P)) & 1)) {
              uint8_t* v = ring + (tv % C::kStages) * C::kTileBytes +
                           row / P * (C::kHalves * P * 128) + row % P * 128;
#pragma unroll
              for (int e = 0; e < 8 * C::kHalves; ++e)
                *reinterpret_cast<uint4*>(v + (e / 8) * (P * 128) + (e % 8) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
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
#pragma unroll
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
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      units_seen += max(pc.n[0], pc.n[1]);
      // ---- the piece's end: the whole item goes out, a part of it into the workspace
      const bool whole = walk.whole();
      if (n > 0) {
        ok = __all_sync(kFull, mbar_wait(&sh.o_full[t], phase_o & 1));
        if (!ok) break;
        ++phase_o;
        tc_fence_after();
      }
      const int head = walk.h * g + row % g;
      if (whole) {
        const size_t at = (size_t)(walk.r.row0 + tok) * p.Hq + head;
        const float inv = l > 0.f ? 1.0f / l : l;  // a NaN sum stays NaN, an empty row gives 0
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          if (n == 0) break;
          uint32_t o[32];
          tmem_ld32(o_at + 32 * i, o);
          tmem_wait_ld(o);
          if (mine) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + 32 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = pack_bf16(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                 __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
              dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        }
        if (mine) p.lse[at] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
      } else {
        const int slot = 2 * blockIdx.x + (walk.u0 == 0 ? 1 : 0);
        float* part = p.partials + (size_t)slot * chunk_slot_floats(D);
        const int r = t * 128 + row;
        if (mine) {
          part[r] = m * c;
          part[kChunkRows + r] = l;
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          if (n == 0) break;
          uint32_t o[32];
          tmem_ld32(o_at + 32 * i, o);
          tmem_wait_ld(o);
          if (mine) {
            float4* dst = reinterpret_cast<float4*>(part + 2 * kChunkRows + (size_t)r * D + 32 * i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
        if (tid == 0 && walk.u0 == 0) {
          const int end = sh.start.shares.taker(walk.at + walk.units - 1, blockIdx.x);
          p.joins[blockIdx.x] = ChunkJoin{walk.b, walk.h, walk.item, end - (int)blockIdx.x + 1};
        }
      }
      tc_fence_before();  // the next piece's first product writes O after the next P arrives
    }
    if (!ok && lane == 0) fail();
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

// Joins the pieces of the item that CTA blockIdx.x began, a warp a row:
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. A lane holds one piece's
// maximum and sum; the pieces' O rows are added in order, eight loads in flight.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const Params p) {
  constexpr int E = D / 32, kInFlight = 8;
  using V = typename std::conditional<E == 4, float4, float2>::type;
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const ChunkJoin jn = p.joins[blockIdx.x];
  if (jn.pieces < 2) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = p.c.g, row = blockIdx.y * 8 + warp;
  const ChunkRequest r = chunk_request(p.c, jn.b, nullptr);
  const int tok = jn.item * (kChunkRows / g) + row / g;
  if (tok >= r.n) return;
  const size_t slot_floats = chunk_slot_floats(D);
  const float* first = p.partials + (size_t)(2 * blockIdx.x + 1) * slot_floats;
  const float* rest = p.partials + (size_t)(2 * blockIdx.x) * slot_floats;
  auto part = [&](int k) { return k == 0 ? first : rest + (size_t)(2 * k) * slot_floats; };
  float M = -INFINITY;
  for (int k = lane; k < jn.pieces; k += 32) M = fmaxf(M, part(k)[row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float acc[E] = {}, L = 0.f;
  for (int k0 = 0; k0 < jn.pieces; k0 += 32) {
    float w = 0.f, wl = 0.f;  // a piece none of whose keys count for this row adds nothing
    if (k0 + lane < jn.pieces) {
      const float* q = part(k0 + lane);
      const float mk = q[row];
      if (mk != -INFINITY) {
        w = ex2(mk - ref);
        wl = w * q[kChunkRows + row];
      }
    }
    const uint32_t some = __ballot_sync(kFull, w != 0.f);  // true for NaN too
    const int n = min(32, jn.pieces - k0);
    for (int k = 0; k < n; k += kInFlight) {
      float o[kInFlight][E];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
#pragma unroll
        for (int e = 0; e < E; ++e) o[u][e] = 0.f;
        if (k + u < n && (some >> (k + u) & 1))
          *reinterpret_cast<V*>(o[u]) = *reinterpret_cast<const V*>(
              part(k0 + k + u) + 2 * kChunkRows + (size_t)row * D + lane * E);
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const float wk = __shfl_sync(kFull, w, (k + u) & 31);
        if (k + u >= n) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, o[u][e], acc[e]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wl += __shfl_xor_sync(kFull, wl, o);
    L += wl;
  }
  const float inv = L > 0.f ? 1.0f / L : L;
  const size_t at = (size_t)(r.row0 + tok) * p.Hq + jn.h * g + row % g;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.out + at * D + lane * E + e) =
        pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) p.lse[at] = L == 0.f ? -INFINITY : M * 0.69314718055994530942f + logf(L);
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
  Params p{{a.q_offsets, kv.seq_lens, kv.batch, kv.num_kv_heads, g, kv.max_pages, P, a.num_tokens,
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
  return launch_pdl(chunk_join_kernel<D>, dim3(a.num_sms, (unsigned)((item_rows + 7) / 8)), dim3(256),
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
