// append_rows.cu - new tokens into the cache with positions on several axes, or into 8-bit
// pages: per-head norms, position rotation, the write of K and V and the fold of the keys into
// the page summaries, in one pass over the packed rows (the bf16 call with one axis is
// norm_rotate.cu's).
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos - b sin, b cos + a sin)
//   8 bits: e = min{e : max|y| <= 448 2^e}, element = e4m3(y 2^-e); its value is exact in bf16
//
// One work item is one page of one request: the new tokens that fall into it. CTAs take items
// in turn; a loader warp looks the next ones up and streams their tokens' rows (contiguous in
// the packed array) through a ring of shared-memory stages. HBM gives rows about as fast as the
// SMs can issue the arithmetic, so a row takes as few instructions as it can: a lane holds 16 of
// its channels (four rows of 128 channels a warp, three shuffles for a sum over a row), and norm
// weight and rotation are one linear map of a pair, whose four factors are made once a token and
// side (queries, keys) and serve all heads:
//   a' = r (a (wa cos) - b (wb sin)),  b' = r (b (wb cos) + a (wa sin))
// Four or eight tokens are worked on at once, two warps or one each (fewer tokens: more warps
// each). A warp has one group of key heads at most and folds their minima and maxima in shared
// memory of its own (in registers they would spill others, and a spilled register comes back from
// L2 where the rings have all of the SM's memory); at the item's end the warps' meet: summaries
// are written once, without atomics.
//
// Few tokens in long pages: an item of a whole page would leave most SMs idle. Only the keys want
// one (their summary); then blocks of 16 slots are items for the queries and values, whole pages
// for the keys, and the two kinds of items go to different CTAs.
//
// The angle: a frequency becomes a 64-bit fixed-point fraction of a turn, whose product with
// the integer position wraps exactly modulo one turn; what it is past the nearest quarter turn
// goes into the series of sine and cosine, so that they keep fp32's full precision.
//
// Measured: 18k tokens of 48 heads (d = 128) into 8-bit pages in 77 us, 5.3 TB/s read and
// written (the copy of the same bytes would take 60); 7k tokens on three axes into bf16 in 37 us
// (26), of which a seventh is SMs that make a round less. 59 us without the queries' norm,
// rotation and stores: what is left is some 230 instructions for four rows, at 60% of the issue
// slots. Two rows a warp (16 lanes each) took 108 us, rows loaded from global memory by each
// warp 111, the key heads' minima in registers, ten more than there are, 89. 64 decoded tokens:
// 5.5 us. Half of the channels turned (rotary_dim 64): 87 and 41 us (pairs side by side 81 and
// 37), with accesses of 8 bytes instead of 16 and up to 20 bytes of spills.
#include <cuda_fp16.h>

#include "tc.cuh"

namespace asp {
namespace {

constexpr int kWarps = 8, kThreads = (kWarps + 1) * 32;  // and a loader
constexpr int kCtas = 2;         // CTAs of an SM
constexpr int kMaxStages = 16;
constexpr int kTurnTokens = 16;  // tokens whose angles are computed together
constexpr int kItems = 3;        // items known ahead
constexpr int kMaxPage = 64;
constexpr unsigned kFull = 0xffffffffu;
// The smallest and largest exponent of a row's scale: the smallest e4m3 step, 2^-9, times 2^-117
// is bf16's smallest normal number, and 448 * 2^119 is below its largest.
constexpr int kMinExp = -117, kMaxExp = 119;

struct Params {
  const uint16_t* qkv;
  const int32_t* q_offsets;
  const int32_t* positions;  // [num_axes, num_tokens], or null: the slots
  const int32_t* pair_axis;  // null: all of axis 0
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const float* inv_freq;
  uint16_t* q_out;
  float* q_out_f32;
  uint16_t* k;
  uint16_t* v;
  uint8_t* k8;
  uint8_t* v8;
  uint8_t* scales;
  uint16_t* summ;
  const int32_t* bt;
  const int32_t* seq_lens;
  uint32_t* err;
  int B, Hq, Hkv, max_pages, num_phys, num_tokens, num_axes, rot, items;
  int P, lp;  // tokens of a page, and log2 of it
  int nq, nk, nv, stages;  // query, key and value heads of a CTA; tokens of its ring
  // CTAs (in y) for blocks of 16 slots, their queries and values; the others in y are for the
  // keys, by page. Not kApart: every CTA has pages, and all three.
  int block_ctas, block_items;
  float eps;
};

struct Item {
  int b, page, lo, cnt;  // the new slots lo .. lo + cnt - 1, all in this page; b < 0: no more
  int row0, phys;        // the first's packed row; physical page, -1: none
};

// The first item from `it` on that has tokens, found by a whole warp; moves `it` behind it.
// ls: log2 of an item's slots. One row per request: item b is request b.
__device__ __forceinline__ Item find_item(const Params& p, int& it, int lane, int ls, int items) {
  for (; it < items; it += gridDim.x) {
    int b = it, page_of_b = 0;
    if (p.q_offsets) {
      b = request_of_item(p.q_offsets, p.B, p.num_tokens, ls, it, lane);
      if (b < 0) continue;
      page_of_b = it - first_item(p.q_offsets, b, p.num_tokens, ls);
    }
    uint32_t* err = lane == 0 ? p.err : nullptr;
    const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, p.P, err);
    const NewRows nr = new_rows(p.q_offsets, b, T, p.num_tokens, err);
    const int first = T - nr.n;  // slot of the first new token
    Item x;
    x.b = b;
    const int at = (first >> ls) + page_of_b;  // the page, or block of slots
    x.lo = max(first, at << ls);
    x.cnt = min(T, (at + 1) << ls) - x.lo;
    if (x.cnt <= 0) continue;
    x.page = x.lo >> p.lp;
    x.row0 = nr.row0 + (x.lo - first);
    x.phys = p.bt[(size_t)b * p.max_pages + x.page];  // checked by the caller
    it += gridDim.x;
    return x;
  }
  return Item{-1, 0, 0, 0, 0, -1};
}

__device__ __forceinline__ float2 unpack(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float2 f) { return pack_bf16(f.x, f.y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// The larger magnitude; NaN if any is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two floats in e4m3 (nearest, ties to even, at most 448), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float2 f) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(f.y), "f"(f.x));
  return r;
}
// What two e4m3 elements stand for, in bf16.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t x, float scale) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
  return pack(mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), both(scale)));
}

// cos and sin of 2 pi phase 2^-64. What the phase is past its nearest quarter turn (at most an
// eighth of a turn, exact in fp32's 24 bits to 2^-27 of a turn) goes into the Taylor series:
// x^11 / 11! < 2e-9 and x^12 / 12! < 2e-10 are left out at pi / 4.
__device__ __forceinline__ float2 cos_sin(unsigned long long phase) {
  const unsigned long long near = phase + (1ull << 61);
  const uint32_t quarter = (uint32_t)(near >> 62);
  const int rest = (int)((phase - (near & (3ull << 62))) >> 32);
  const float x = (float)rest * 1.4629180792671596e-09f;  // 2 pi 2^-32
  const float z = x * x;
  float sn = fmaf(z, 2.7557319224e-06f, -1.9841269841e-04f);  // 1/9!, -1/7!
  sn = fmaf(z, sn, 8.3333333333e-03f);
  sn = fmaf(z, sn, -1.6666666667e-01f);
  sn = fmaf(z * x, sn, x);
  float c = fmaf(z, -2.7557319224e-07f, 2.4801587302e-05f);  // -1/10!, 1/8!
  c = fmaf(z, c, -1.3888888889e-03f);
  c = fmaf(z, c, 4.1666666667e-02f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const float a = quarter & 1 ? sn : c, b = quarter & 1 ? c : sn;
  return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

// A lane's channels of a row are two quads of four rotated pairs: of quad u the first four
// channels (ca[u]) and the second four (cb[u]). Halves rotated against each other: pair i is
// channel i of the first and of the second four; interleaved, or not rotated at all: eight
// channels in a row. Where every quad turns (kAll: rot = D) a lane's quads are chosen so that it
// has two pieces of eight channels in a row, 8 l and D / 2 + 8 l: 16-byte accesses, no two of
// eight lanes in one bank.
template <int D, bool kInterleaved, bool kAll>
struct Lane {
  static constexpr int kLanes = D / 16;
  static constexpr bool kSplit = kAll && !kInterleaved;
  int sub, l;
  int ca[2], cb[2];
  bool turn[2];
  __device__ __forceinline__ Lane(int lane, int rot) {
    sub = lane / kLanes, l = lane % kLanes;
    if (kAll) rot = D;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = kSplit ? 2 * l + u : l + kLanes * u;
      turn[u] = kAll || 8 * t < rot;
      const bool split = turn[u] && !kInterleaved;
      ca[u] = split ? 4 * t : 8 * t, cb[u] = split ? rot / 2 + 4 * t : 8 * t + 4;
    }
  }
  // Where the table of a token's angles has pair i: a lane's eight, two by two, lie kLanes apart.
  static __device__ __forceinline__ int place(int i) {
    const int l = kSplit ? i >> 3 : (i >> 2) % kLanes, u = kSplit ? i >> 2 & 1 : (i >> 2) / kLanes;
    return ((2 * u + (i >> 1 & 1)) * kLanes + l) * 2 + (i & 1);
  }
  // x: first fours of the quads, second fours
  __device__ __forceinline__ void load(const uint16_t* row, uint2 (&x)[4]) const {
    if constexpr (kAll) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + 8 * l);
      const uint4 b = *reinterpret_cast<const uint4*>(row + D / 2 + 8 * l);
      x[0] = make_uint2(a.x, a.y), x[3] = make_uint2(b.z, b.w);
      x[kSplit ? 1 : 2] = make_uint2(a.z, a.w), x[kSplit ? 2 : 1] = make_uint2(b.x, b.y);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        x[u] = *reinterpret_cast<const uint2*>(row + ca[u]),
        x[2 + u] = *reinterpret_cast<const uint2*>(row + cb[u]);
    }
  }
  // The same order back, four channels an element of x.
  template <typename T4, typename T>
  __device__ __forceinline__ void store(T* row, const T4 (&x)[4]) const {
    if constexpr (kAll && sizeof(T4) == 8) {
      const T4 &a = x[kSplit ? 1 : 2], &b = x[kSplit ? 2 : 1];
      *reinterpret_cast<uint4*>(row + 8 * l) = make_uint4(x[0].x, x[0].y, a.x, a.y);
      *reinterpret_cast<uint4*>(row + D / 2 + 8 * l) = make_uint4(b.x, b.y, x[3].x, x[3].y);
    } else if constexpr (kAll && sizeof(T4) == 4) {
      *reinterpret_cast<uint2*>(row + 8 * l) = make_uint2(x[0], x[kSplit ? 1 : 2]);
      *reinterpret_cast<uint2*>(row + D / 2 + 8 * l) = make_uint2(x[kSplit ? 2 : 1], x[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<T4*>(row + ca[u]) = x[u], *reinterpret_cast<T4*>(row + cb[u]) = x[2 + u];
    }
  }
  // Sum, or any other combination, over a row's lanes.
  template <typename F>
  static __device__ __forceinline__ float over_row(float x, F f) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) x = f(x, __shfl_xor_sync(kFull, x, o));
    return x;
  }
};

// The linear map of a lane's pairs for one token and side: factors of the channel itself and of
// its pair's other channel, for both quads' first and second fours.
template <int D, bool kInterleaved, bool kAll>
struct Map {
  using L = Lane<D, kInterleaved, kAll>;
  float2 own[2][4], other[2][4];
  // turn: (cos, sin) of the token's pairs; weight: the norm's, in bf16
  __device__ __forceinline__ void make(const L& ln, const float2* turn, const uint16_t* weight) {
    uint2 w[4];
    ln.load(weight, w);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float2 wa[2] = {unpack(w[u].x), unpack(w[u].y)};
      const float2 wb[2] = {unpack(w[2 + u].x), unpack(w[2 + u].y)};
      float4 cs[2] = {make_float4(1.f, 0.f, 1.f, 0.f), make_float4(1.f, 0.f, 1.f, 0.f)};
      if (ln.turn[u]) {
        const float4* src = reinterpret_cast<const float4*>(turn) + 2 * u * L::kLanes + ln.l;
        cs[0] = src[0], cs[1] = src[L::kLanes];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (kInterleaved) {  // wa, wb: pairs 0, 1 and 2, 3, their channels side by side
          const float2 wp[2] = {wa[i], wb[i]};
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // pair 2 j + i
            const float c = i ? cs[j].z : cs[j].x, s = i ? cs[j].w : cs[j].y;
            own[u][2 * j + i] = mul2(wp[j], both(c));
            other[u][2 * j + i] = make_float2(-wp[j].y * s, wp[j].x * s);
          }
        } else {  // pairs 2 i, 2 i + 1
          const float2 c = make_float2(cs[i].x, cs[i].z), s = make_float2(cs[i].y, cs[i].w);
          own[u][i] = mul2(wa[i], c), own[u][2 + i] = mul2(wb[i], c);
          other[u][i] = mul2(wb[i], make_float2(-s.x, -s.y)), other[u][2 + i] = mul2(wa[i], s);
        }
      }
    }
  }
};

// A lane's 16 channels in fp32: of each quad the first four (0, 1) and the second four (2, 3).
template <int D, bool kInterleaved, bool kAll>
struct Row {
  using L = Lane<D, kInterleaved, kAll>;
  float2 f[2][4];
  __device__ __forceinline__ void set(const uint2 (&x)[4]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f[u][0] = unpack(x[u].x), f[u][1] = unpack(x[u].y);
      f[u][2] = unpack(x[2 + u].x), f[u][3] = unpack(x[2 + u].y);
    }
  }
  __device__ __forceinline__ float norm(float eps) const {
    float2 a = mul2(f[0][0], f[0][0]), b = mul2(f[1][0], f[1][0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) a = fma2(f[0][i], f[0][i], a), b = fma2(f[1][i], f[1][i], b);
    const float ss = L::over_row((a.x + b.x) + (a.y + b.y), [](float x, float y) { return x + y; });
    const float v = fmaf(ss, 1.0f / D, eps), r = rsqrtf(v);
    const float e = fmaf(-v * r, r, 1.0f);
    return e == e ? fmaf(r * 0.5f, e, r) : r;  // one step towards the exact root; not from 0 or inf
  }
  // r: what multiplies the row after the map
  __device__ __forceinline__ void apply(const Map<D, kInterleaved, kAll>& m, const L& ln, float r) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float2 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul2(f[u][i], m.own[u][i]);
      if (kAll || ln.turn[u]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 o = kInterleaved ? make_float2(f[u][i].y, f[u][i].x) : f[u][i ^ 2];
          y[i] = fma2(o, m.other[u][i], y[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) f[u][i] = mul2(y[i], both(r));
    }
  }
  // in the order of Lane::load
  __device__ __forceinline__ void bf16(uint2 (&x)[4]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) x[2 * h + u] = make_uint2(pack(f[u][2 * h]), pack(f[u][2 * h + 1]));
  }
  __device__ __forceinline__ void fp32(float4 (&x)[4]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[2 * h + u] = make_float4(f[u][2 * h].x, f[u][2 * h].y, f[u][2 * h + 1].x, f[u][2 * h + 1].y);
  }
  // e4m3 elements in the order of Lane::load and the row's scale byte; a row with a NaN or an
  // infinity is NaN.
  __device__ __forceinline__ uint32_t quantise(uint32_t (&x)[4]) const {
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max_abs(top, f[u][i].x, f[u][i].y);
    top = L::over_row(top, [](float a, float b) { return max_abs(a, a, b); });
    const uint32_t bits = __float_as_uint(top);
    // 448 = 1.75 * 2^8
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    const int held = min(max(e, kMinExp), kMaxExp);
    const float inv = __uint_as_float((uint32_t)(127 - held) << 23);
    const bool fine = bits < 0x7f800000u;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t y = to_e4m3x2(mul2(f[u][2 * h], both(inv))) |
                           to_e4m3x2(mul2(f[u][2 * h + 1], both(inv))) << 16;
        x[2 * h + u] = fine ? y : 0;
      }
    return fine ? (uint32_t)(held + 127) : 255u;
  }
};

// Shared memory behind the ring.
template <int D>
struct Shared {
  float2 turn[2][kTurnTokens * (D / 2)];  // (cos, sin) of [token][pair]
  uint32_t fold[kWarps][16][32];          // a warp's minima, then maxima, by lane
  unsigned long long turns_of[D / 2];     // 2^64 * inv_freq / (2 pi), modulo 2^64
  int axis[D / 2];
  __align__(16) uint16_t weight[2][D];    // the norms' of queries and keys, or ones
  int pos[kItems][ASP_MAX_AXES][kMaxPage];
  Item item[kItems];
  uint64_t full[kMaxStages], empty[kMaxStages], item_full[kItems], item_empty[kItems], meet[2];
};

template <int D, bool kInterleaved, bool kQ8, bool kAll, bool kApart>
__global__ void __launch_bounds__(kThreads, kCtas) append_kernel(const Params p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // lanes of a row, rows of a warp
  using RowT = Row<D, kInterleaved, kAll>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // this CTA's kind of items and its heads: a share of the query, the key and the value heads
  const bool blocks = kApart && (int)blockIdx.y < p.block_ctas, keys = kApart && !blocks;
  const int y = blockIdx.y - (keys ? p.block_ctas : 0);
  const int q0 = y * p.nq, nq = keys ? 0 : max(0, min(p.nq, p.Hq - q0));
  const int k0 = y * p.nk, nk = blocks ? 0 : max(0, min(p.nk, p.Hkv - k0));
  const int v0 = kApart ? y * p.nv : k0;
  const int nv = !kApart ? nk : keys ? 0 : max(0, min(p.nv, p.Hkv - v0));
  const int ls = blocks ? 4 : p.lp, items = blocks ? p.block_items : p.items;
  const int nvs = kApart ? p.nv : p.nk;  // value heads of a token's place in the ring
  const int stage_bytes = (p.nq + p.nk + nvs) * D * 2;
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem + p.stages * stage_bytes);
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], kWarps);
    }
    mbar_init(&sh.meet[0], kWarps);
    mbar_init(&sh.meet[1], kWarps);
    mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int half = (kAll ? D : p.rot) / 2;
  if (warp == kWarps) {
    // ------------------------------------------------------------ loader
    const uint32_t bytes = (uint32_t)(nq + nk + nv) * D * 2;
    const int Hall = p.Hq + 2 * p.Hkv;
    uint32_t tk = 0, n = 0;  // tokens loaded, items handed on
    bool ok = true;
    auto load = [&](const Item& x, int t) {
      const int st = tk % p.stages;
      ok = __all_sync(kFull, mbar_wait(&sh.empty[st], ((tk / p.stages) & 1) ^ 1));
      if (!ok) return;
      if (lane == 0) {
        const uint16_t* row = p.qkv + (size_t)(x.row0 + t) * Hall * D;
        uint8_t* dst = smem + st * stage_bytes;
        mbar_arrive_expect_tx(&sh.full[st], bytes);
        if (nq == p.Hq && nk == p.Hkv && nv == p.Hkv) {  // the whole row
          bulk_g2s(dst, row, bytes, &sh.full[st]);
        } else {
          if (nq > 0) bulk_g2s(dst, row + q0 * D, nq * D * 2, &sh.full[st]);
          dst += p.nq * D * 2;
          if (nk > 0) bulk_g2s(dst, row + (p.Hq + k0) * D, nk * D * 2, &sh.full[st]);
          dst += p.nk * D * 2;
          if (nv > 0) bulk_g2s(dst, row + (p.Hq + p.Hkv + v0) * D, nv * D * 2, &sh.full[st]);
        }
      }
      ++tk;
    };
    for (int it = blockIdx.x; ok; ++n) {
      Item x = find_item(p, it, lane, ls, items);
      if (n == 0) __syncthreads();  // the barriers are there
      // the first row is on its way while the positions are looked up
      if (x.b >= 0 && bytes) load(x, 0);
      if (!ok) break;
      const int slot = n % kItems;
      ok = __all_sync(kFull, mbar_wait(&sh.item_empty[slot], ((n / kItems) & 1) ^ 1));
      if (!ok) break;
      if (x.b >= 0) {
        for (int t = lane; t < x.cnt; t += 32)
          for (int a = 0; a < p.num_axes; ++a)
            sh.pos[slot][a][t] =
                p.positions ? p.positions[(size_t)a * p.num_tokens + x.row0 + t] : x.lo + t;
        if (x.phys < 0 || x.phys >= p.num_phys) {
          if (lane == 0) report(p.err, ASP_DEVERR_PAGE_RANGE);
          x.phys = -1;
        }
      }
      __syncwarp();
      if (lane == 0) {
        sh.item[slot] = x;
        mbar_arrive(&sh.item_full[slot]);
      }
      if (x.b < 0) break;
      for (int t = 1; t < x.cnt && bytes && ok; ++t) load(x, t);
    }
    if (p.q_offsets && blockIdx.x == 0 && blockIdx.y == 0) {  // every request's rows are checked
      for (int x = lane; x < p.B; x += 32)
        new_rows(p.q_offsets, x, clamp_seq_len(p.seq_lens[x], p.max_pages, p.P, p.err),
                 p.num_tokens, p.err);
    }
    if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
    // the CTA's memory stays until its copies have ended
    if (bytes && lane == 0)
      for (uint32_t i = tk > (uint32_t)p.stages ? tk - p.stages : 0; i < tk; ++i)
        mbar_wait(&sh.full[i % p.stages], (i / p.stages) & 1);
    return;
  }

  for (int i = tid; i < 2 * D; i += kWarps * 32) {
    const uint16_t* w = i < D ? p.q_weight : p.k_weight;
    sh.weight[i / D][i % D] = w ? w[i % D] : 0x3f80;
  }
  if (tid < half) {
    double t = (double)p.inv_freq[tid] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    sh.turns_of[tid] = (unsigned long long)(t * 18446744073709551616.0);
    int axis = p.pair_axis ? p.pair_axis[tid] : 0;
    if (axis < 0 || axis >= p.num_axes) {
      report(p.err, ASP_DEVERR_AXIS_RANGE);
      axis = 0;
      sh.turns_of[tid] = 0;
    }
    sh.axis[tid] = axis;
  }
  __syncthreads();
  const Lane<D, kInterleaved, kAll> ln(lane, p.rot);
  const int groups = (nk + kRows - 1) / kRows, q_groups = (nq + kRows - 1) / kRows;
  const int v_groups = (nv + kRows - 1) / kRows;
  // this thread's first (token, pair) of the angles, and the step to its next
  const int tt0 = half ? tid / half : 0, f0 = half ? tid % half : 0;
  const int tt_step = half ? kWarps * 32 / half : 0, f_step = half ? kWarps * 32 % half : 0;
  // Four tokens at once, or eight where the ring holds them: a warp has one group of key heads
  // at most.
  const int at_once_log2 = max(groups, v_groups) <= 1 && p.stages >= kWarps ? 3 : 2;
  uint32_t tk = 0, blk = 0;
  int st = 0, phase = 0;  // of token tk
  bool ok = true;
  uint32_t meets = 0;
  auto meet = [&]() {  // all warps but the loader; a bounded wait, like every other
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.meet[meets & 1]);
    ok = __all_sync(kFull, mbar_wait(&sh.meet[meets & 1], (meets >> 1) & 1));
    ++meets;
  };
  for (uint32_t n = 0; ok; ++n) {
    const int islot = n % kItems;
    ok = __all_sync(kFull, mbar_wait(&sh.item_full[islot], (n / kItems) & 1));
    if (!ok) break;
    const Item x = sh.item[islot];
    if (x.b < 0) break;
    const bool mapped = x.phys >= 0;
    // tokens at once (a power of two), the warps of one, this one's place among them; the
    // first of them take a group of key heads, the last one of value heads
    const int lt = min(at_once_log2, 31 - __clz(x.cnt)), at_once = 1 << lt, wpt = kWarps >> lt;
    const int cls = warp & (at_once - 1), j = warp >> lt, jv = wpt - 1 - j;
    const bool k_mine = mapped && j < groups, v_mine = mapped && jv < v_groups;
    const int kh = j * kRows + ln.sub, kh_read = min(kh, nk - 1);
    const int vh = jv * kRows + ln.sub, vh_read = min(vh, nv - 1);
    const size_t page = (size_t)(mapped ? x.phys : 0) * p.Hkv;
    const size_t k_block = (page + k0 + kh_read) << p.lp, v_block = (page + v0 + vh_read) << p.lp;
    for (int t = 0; t < x.cnt; ++t, ++tk) {
      const float2* turn = sh.turn[(blk - 1) & 1];
      if (t % kTurnTokens == 0) {
        // the angles of the next tokens, into the table that no warp reads any more: all have
        // passed the barrier of the one between
        float2* to = sh.turn[blk++ & 1];
        turn = to;
        if (half > 0) {
          const int cnt = min(kTurnTokens, x.cnt - t);
          int tt = tt0, f = f0;
          while (tt < cnt) {
            const int pos = sh.pos[islot][sh.axis[f]][t + tt];
            to[tt * (D / 2) + ln.place(f)] = cos_sin(sh.turns_of[f] * (unsigned long long)(long long)pos);
            tt += tt_step, f += f_step;
            if (f >= half) f -= half, ++tt;
          }
        }
        meet();
        if (!ok) break;
      }
      if (nq + nk + nv > 0) ok = __all_sync(kFull, mbar_wait(&sh.full[st], phase));
      if (!ok) break;
      if ((t & (at_once - 1)) == cls) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(smem + st * stage_bytes);
        const uint16_t* k = q + p.nq * D;
        const float2* cs = turn + t % kTurnTokens * (D / 2);
        const int slot = (x.lo + t) & (p.P - 1);
        Map<D, kInterleaved, kAll> map;
        if (k_mine) {
          uint2 y[4];
          ln.load(k + kh_read * D, y);
          map.make(ln, cs, sh.weight[1]);
          RowT row;
          row.set(y);
          const float r = p.k_weight ? row.norm(p.eps) : 1.0f;
          row.apply(map, ln, r);
          const bool k_row = kh < nk, first = t == cls;
          auto fold = [&](int i, uint32_t val) {  // the warp's first key of the item starts them
            uint32_t &a = sh.fold[warp][i][lane], &b = sh.fold[warp][8 + i][lane];
            a = bmin2(first ? kNanPair : a, val), b = bmax2(first ? kNanPair : b, val);
          };
          if constexpr (kQ8) {
            uint32_t c[4];
            const uint32_t scale = row.quantise(c);
            const float f = __uint_as_float(scale << 23);
            if (k_row) {
              ln.store(p.k8 + (k_block + slot) * D, c);
              if (ln.l == 0) p.scales[k_block * 2 + slot] = (uint8_t)scale;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t val = scale == 255 ? kNanPair : from_e4m3x2(c[i / 2] >> (16 * (i & 1)) & 0xffff, f);
              fold(i, val);
            }
          } else {
            uint2 c[4];
            row.bf16(c);
            if (k_row) ln.store(p.k + (k_block + slot) * D, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              fold(i, i & 1 ? c[i / 2].y : c[i / 2].x);
            }
          }
        }
        if (v_mine) {  // 8 channels of the row's first half and 8 of its second
          const uint16_t* src = k + (p.nk + vh_read) * D + 8 * ln.l;
          const uint4 y[2] = {*reinterpret_cast<const uint4*>(src),
                              *reinterpret_cast<const uint4*>(src + D / 2)};
          const bool v_row = vh < nv;
          if constexpr (kQ8) {
            RowT row;
#pragma unroll
            for (int u = 0; u < 2; ++u)
              row.f[u][0] = unpack(y[u].x), row.f[u][1] = unpack(y[u].y),
              row.f[u][2] = unpack(y[u].z), row.f[u][3] = unpack(y[u].w);
            uint32_t c[4];
            const uint32_t scale = row.quantise(c);
            if (v_row) {
              uint8_t* dst = p.v8 + (v_block + slot) * D + 8 * ln.l;
              *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[2]);
              *reinterpret_cast<uint2*>(dst + D / 2) = make_uint2(c[1], c[3]);
              if (ln.l == 0) p.scales[v_block * 2 + p.P + slot] = (uint8_t)scale;
            }
          } else if (v_row) {
            uint16_t* dst = p.v + (v_block + slot) * D + 8 * ln.l;
            *reinterpret_cast<uint4*>(dst) = y[0];
            *reinterpret_cast<uint4*>(dst + D / 2) = y[1];
          }
        }
        const int j_q = (j - groups + wpt) % wpt;  // few tokens: not those with key heads first
        if (j_q < q_groups) {
          map.make(ln, cs, sh.weight[0]);
          const size_t out = ((size_t)(x.row0 + t) * p.Hq + q0) * D;
          for (int g = j_q; g < q_groups; g += wpt) {
            const int h = g * kRows + ln.sub;
            uint2 y[4];
            ln.load(q + min(h, nq - 1) * D, y);
            RowT row;
            row.set(y);
            const float r = p.q_weight ? row.norm(p.eps) : 1.0f;
            row.apply(map, ln, r);
            if (h < nq) {
              const size_t o = out + h * D;
              if (p.q_out) {
                uint2 c[4];
                row.bf16(c);
                ln.store(p.q_out + o, c);
              }
              if (p.q_out_f32) {
                float4 c[4];
                row.fp32(c);
                ln.store(p.q_out_f32 + o, c);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
      if (++st == p.stages) st = 0, phase ^= 1;
    }
    if (!ok) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_empty[islot]);
    // ---- the summary: of the minima and maxima of the warps that had a group of key heads (the
    // next item's first are written after its angles' barrier)
    meet();
    if (!ok) break;
    // minima and maxima by a warp each, where there are two
    for (int side = cls; side < 2 && k_mine && kh < nk; side += at_once) {
      uint32_t m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = kNanPair;
      for (int c = 0; c < at_once; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t y = sh.fold[j << lt | c][side * 8 + i][lane];
          m[i] = side ? bmax2(m[i], y) : bmin2(m[i], y);
        }
      uint16_t* s = p.summ + (((size_t)x.b * p.Hkv + k0 + kh) * p.max_pages + x.page) * 2 * D + side * D;
      uint2 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = make_uint2(m[2 * i], m[2 * i + 1]);
      if (x.lo != x.page << p.lp) {  // the page had tokens before
        uint2 old[4];
        ln.load(s, old);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = side ? vmax(old[i], y[i]) : vmin(old[i], y[i]);
      }
      ln.store(s, y);
    }
    __syncwarp();
  }
  if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
}

template <int D, bool kInterleaved, bool kQ8>
cudaError_t launch_t(const NormRotateArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  const int P = kv.page_size, items = a.q_offsets ? a.num_tokens / P + 2 * kv.batch : kv.batch;
  // CTAs take items in turn, so that the next is looked up and its rows are loaded while the
  // last is worked on. An item's heads are split over several CTAs (each computes the angles
  // again, about a tenth of the work) where that fills the SMs better: the rounds that the
  // busiest CTA makes, in whole items.
  const int slots = kCtas * a.num_sms, most = max(1, kv.num_q_heads * D / (8 * 256));
  int split = 1;
  float best = 1e30f;
  for (int s = 1; s <= most && s <= 8; s *= 2) {
    const float cost = (float)(((long long)items * s + slots - 1) / slots) * (1.0f / s + 0.1f);
    if (cost < best) best = cost, split = s;
  }
  int ctas = min(items, max(1, slots / split)), block_ctas = 0, block_items = 0;
  int nq = ceil_div(kv.num_q_heads, split), nk = ceil_div(kv.num_kv_heads, split), nv = nk;
  // Long pages whose items and blocks of slots all run at once: 139 tokens of 64/8 heads in pages
  // of 64, four items, 35 us by page, 28 by blocks and pages; 2 x 2000 tokens 46 and 37.
  if (P > kTurnTokens && a.q_offsets) {
    const int blocks = a.num_tokens / kTurnTokens + 2 * kv.batch;
    int bs = 1, ks = 1;  // CTAs in y for blocks and for keys
    if (blocks + items <= slots) {
      while (ks * 2 <= kv.num_kv_heads && blocks * bs + items * ks * 2 <= slots && ks < 8) ks *= 2;
      while (bs * 2 <= kv.num_kv_heads && blocks * bs * 2 + items * ks <= slots && bs < 8) bs *= 2;
      split = bs + ks, block_ctas = bs, block_items = blocks, ctas = blocks;
      nq = ceil_div(kv.num_q_heads, bs), nv = ceil_div(kv.num_kv_heads, bs);
      nk = ceil_div(kv.num_kv_heads, ks);
    }
  }
  const int stage_bytes = (nq + nk + nv) * D * 2;
  constexpr int kBudget = 72 * 1024;  // up to sixteen tokens in a third of an SM's shared memory
  const int stages = max(2, min(kMaxStages, kBudget / stage_bytes));
  const Params p{a.qkv, a.q_offsets, a.positions, a.pair_axis, a.q_weight, a.k_weight, a.inv_freq,
                 a.q_out, a.q_out_f32, kv.k_cache, kv.v_cache, a.q8 ? a.q8->k : nullptr,
                 a.q8 ? a.q8->v : nullptr, a.q8 ? a.q8->scales : nullptr, kv.summaries,
                 kv.block_table, kv.seq_lens, a.err, kv.batch, kv.num_q_heads, kv.num_kv_heads,
                 kv.max_pages, kv.num_phys_pages, a.num_tokens, a.num_axes, a.rotary_dim, items,
                 P, P == 64 ? 6 : P == 32 ? 5 : 4, nq, nk, nv, stages,
                 block_ctas, block_items, a.eps};
  auto kernel = a.rotary_dim == D ? append_kernel<D, kInterleaved, kQ8, true, false>
                                  : append_kernel<D, kInterleaved, kQ8, false, false>;
  // An instance of its own: the choice at run time cost full pages of 16 a twentieth (77 to 80 us).
  if (block_ctas > 0)
    kernel = a.rotary_dim == D ? append_kernel<D, kInterleaved, kQ8, true, true>
                               : append_kernel<D, kInterleaved, kQ8, false, true>;
  const int smem = stages * stage_bytes + (int)sizeof(Shared<D>);
  const cudaError_t e = set_max_dynamic_smem((const void*)kernel, kBudget + (int)sizeof(Shared<D>));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas, split), dim3(kThreads), smem, stream, p);
}

}  // namespace

cudaError_t launch_append_rows(const NormRotateArgs& a, cudaStream_t stream) {
  if (a.kv->head_dim == 128)
    return a.interleaved ? (a.q8 ? launch_t<128, true, true>(a, stream) : launch_t<128, true, false>(a, stream))
                         : (a.q8 ? launch_t<128, false, true>(a, stream) : launch_t<128, false, false>(a, stream));
  return a.interleaved ? (a.q8 ? launch_t<64, true, true>(a, stream) : launch_t<64, true, false>(a, stream))
                       : (a.q8 ? launch_t<64, false, true>(a, stream) : launch_t<64, false, false>(a, stream));
}

}  // namespace asp
