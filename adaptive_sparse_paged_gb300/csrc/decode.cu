// decode.cu - self-planning sparse attention over ragged page lists (MOIRA
// abstract: each thread block derives its own share of the work from the
// list lengths, so the decode step needs no host-side plan and stays inside
// the CUDA graph).
//
// Plan (every CTA, on the device): load lens[B*Hkv] into shared memory and
// take their inclusive prefix; the concatenated lists form one sequence of
// `total` pages. Each (segment, CTA) piece ends in a CTA-wide merge of the
// warps' states: the warps, which drift apart over a piece, all wait for the
// last one, so the CTA's copy pipeline idles for several microseconds. The
// first page of every non-empty list therefore weighs 1 + piece_cost pages
// (about 256 KiB of K and V) and the sequence is split evenly by weight over the G
// CTAs: a CTA whose range starts more lists takes fewer pages, and the split
// still depends on the list lengths alone. Each piece produces one partial
// (m, l, o) in slot segment + CTA of the workspace, which is unique because
// both indices grow along the sequence; a segment held whole by one CTA is
// written out directly. A split segment is merged by log-sum-exp by the last
// of its CTAs to finish: each counts its piece in with one atomic after its
// stream has ended (never at a piece end, where the round trip, 1.5-2 us
// under full HBM load, would stall the copy pipeline), and the CTA that
// completes the count folds the pieces in CTA order, so the result does not
// depend on timing. No CTA ever waits on another.
//
// The kernel is written over a page format (Bf16Pages, Q8Pages below): what a
// stage holds, how it is copied and what a warp computes on it. The plan, the
// pipelines and the merges are the same for both. What follows is the bf16 form.
//
// Data path (per CTA: 8 warps, one CTA per SM): every warp runs its own
// pipeline. Warp w takes stages w, w+8, ... of the CTA's slice (a stage is a
// 16-token sub-tile of one page: K then V, [16 rows x 64 channels] 2-D TMA
// boxes with the 128-byte swizzle), keeps kSlots of them in flight in its own
// shared-memory slots, each with its own mbarrier, and refills a slot as soon
// as it has consumed it. Its lanes resolve list entry -> logical page ->
// physical row for the next 32 stages ahead of time. Independent issuers per
// SM are what reach the copy bandwidth on this gather; one issuing thread per
// CTA does not. Each warp keeps its own online-softmax state; the warps are
// merged in shared memory at the end of each piece.
//
// Per page the contraction is small (g <= 8 queries against P tokens), so it
// runs on mma.sync m16n8k16 bf16 with tokens as the M dimension and the query
// group (padded to 8) as N:
//   S^T[16 x 8] = K[16 x d] . Q^T[d x 8]      (Q split into bf16 hi + lo)
//   O^T[d x 8] += V^T[d x 16] . P^T[16 x 8]   (probabilities rounded to bf16)
// The S^T accumulator becomes the P^T operand through movmatrix.trans, and the
// swizzled tiles make every ldmatrix conflict-free. A page is 4-32 KiB of HBM
// against 4-8 flop per byte, far below any tensor-core limit: the kernel is
// bound by HBM, and the ring (128 KiB, or 192 KiB when the segment prefix
// leaves room in shared memory) keeps that much per SM in flight.
#include "asp_internal.cuh"

#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <climits>

#include <mutex>

namespace asp {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct DecParams {
  const float* q;
  const int32_t* lists;
  const int32_t* lens;
  const int32_t* bt;
  const int32_t* seq_lens;
  float* out;
  float* lse;
  float* partials;
  int32_t* arrivals;  // [S]: pieces of each split segment done; zero between calls
  const uint8_t* scales;  // of 8-bit pages
  uint32_t* err;
  int B, Hq, Hkv, g, max_pages, num_phys, slot_floats;
  int piece_cost;  // extra weight of a list's first page in the split, in pages
  float scale_log2;
};

// ------------------------------------------------------------ mma helpers
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Byte offset of (row r < 16, channel c, c % 8 == 0) inside a stage's K or V
// part, laid out as kHalves tiles of [16 rows x 128 B] with the 128-byte
// swizzle (16-byte chunk index XOR row % 8; tiles start on 1 KiB boundaries).
__device__ __forceinline__ uint32_t swz(int r, int c) {
  const int hh = c >> 6, chunk = (c & 63) >> 3;
  return hh * (16 * 128) + r * 128 + ((chunk ^ (r & 7)) << 4);
}

// ------------------------------------------------------------ bf16 pages
// What the kernel asks of a page format: the sizes of its stages, the copies of
// one, and the state of a lane's softmax with the step over one stage.
//
// A stage is a 16-token sub-tile of a page (P/16 stages per page): 8 KiB (d=128)
// or 4 KiB (d=64). Each warp owns kSlots stages of the ring: 128 KiB per CTA,
// or 192 KiB (Deep) when the segment prefix leaves room in shared memory.
// While a warp computes on one stage the others stay in flight, so the extra
// slot is what keeps each SM's share of the copy bandwidth requested.
template <int kDim, int kPage, bool Deep>
struct Bf16Pages {
  static constexpr int D = kDim, P = kPage, kWarps = 8;
  static constexpr int kHalves = D / 64;
  static constexpr int kSubs = P / 16;                      // stages per page
  static constexpr int kTileBytes = 16 * 128;               // [16 rows x 64 bf16], swizzled
  static constexpr int kPartBytes = kHalves * kTileBytes;   // K (or V) of 16 tokens
  static constexpr int kStageBytes = 2 * kPartBytes;        // K then V
  static constexpr int kExtraBytes = 0;
  static constexpr int kSlots = (D == 128 ? 2 : 4) * (Deep ? 3 : 2) / 2;  // stages per warp
  static constexpr bool kNanStays = false;
  static constexpr int kMinPages = 1;

  static __device__ __forceinline__ void issue(uint8_t* dst, uint8_t*, const CUtensorMap& tmK,
                                               const CUtensorMap& tmV, const DecParams&, int row, int,
                                               uint64_t* bar, uint64_t pol) {
    mbar_arrive_expect_tx(bar, kStageBytes);
#pragma unroll
    for (int hh = 0; hh < kHalves; ++hh) {
      tma_load_2d_hint(dst + hh * kTileBytes, &tmK, hh * 64, row, bar, pol);
      tma_load_2d_hint(dst + kPartBytes + hh * kTileBytes, &tmV, hh * 64, row, bar, pol);
    }
  }

  // Channel that position pos of the accumulators holds.
  static __device__ __forceinline__ int channel(int pos) { return pos; }

  struct State {
    float m0, m1, l0, l1;   // of query columns 2 tq, 2 tq + 1
    float o[D / 16][4];     // positions 16 dt + gid (0, 1) and + 8 (2, 3) of those columns
    // Q^T fragments (B operand): rows d = kk*16 + 2*tq (+1, +8, +9), column gid
    uint32_t qhi[D / 16][2], qlo[D / 16][2];

    __device__ __forceinline__ void load_q(const DecParams& p, int seg, int gid, int tq) {
      const int qb = seg / p.Hkv, qh = seg % p.Hkv;
      const bool live = gid < p.g;
      const float* qr = p.q + ((size_t)qb * p.Hq + qh * p.g + (live ? gid : 0)) * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float2 v = make_float2(0.f, 0.f);
          if (live) v = *reinterpret_cast<const float2*>(qr + kk * 16 + half * 8 + 2 * tq);
          v.x *= p.scale_log2;
          v.y *= p.scale_log2;
          const __nv_bfloat162 hv = __floats2bfloat162_rn(v.x, v.y);
          const float2 hf = __bfloat1622float2(hv);
          qhi[kk][half] = *reinterpret_cast<const uint32_t*>(&hv);
          qlo[kk][half] = pack_bf16(v.x - hf.x, v.y - hf.y);
        }
    }

    __device__ __forceinline__ void start() {
      m0 = m1 = -INFINITY, l0 = l1 = 0.f;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) o[dt][0] = o[dt][1] = o[dt][2] = o[dt][3] = 0.f;
    }

    __device__ __forceinline__ void step(uint8_t* st, const uint8_t*, int ntok, int lane) {
      const int gid = lane >> 2, j = lane >> 3;
      const uint32_t kb = smem_u32(st);
      const uint32_t vb = kb + kPartBytes;
      // ---- S^T[16 x 8] = K[16 x d] . Q^T[d x 8]
      float sv[4];
      {
        // four independent accumulator chains (hi/lo x even/odd k-step)
        float acc[4][4] = {};
        const int r = (j & 1) * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a[4];
          ldsm_x4(kb + swz(r, kk * 16 + (j >> 1) * 8), a);
          mma16816(acc[(kk & 1) * 2], a, qhi[kk][0], qhi[kk][1]);
          mma16816(acc[(kk & 1) * 2 + 1], a, qlo[kk][0], qlo[kk][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sv[i] = (acc[0][i] + acc[2][i]) + (acc[1][i] + acc[3][i]);
      }
      // ---- mask tokens past the sequence, online softmax (log2 domain)
      if (gid >= ntok) sv[0] = sv[1] = -INFINITY;
      if (gid + 8 >= ntok) sv[2] = sv[3] = -INFINITY;
      float cm0 = fmaxf(sv[0], sv[2]), cm1 = fmaxf(sv[1], sv[3]);
#pragma unroll
      for (int off2 = 4; off2 < 32; off2 <<= 1) {
        cm0 = fmaxf(cm0, __shfl_xor_sync(kFull, cm0, off2));
        cm1 = fmaxf(cm1, __shfl_xor_sync(kFull, cm1, off2));
      }
      const float n0 = fmaxf(m0, cm0), n1 = fmaxf(m1, cm1);
      const float al0 = exp2f(m0 - n0), al1 = exp2f(m1 - n1);
      m0 = n0;
      m1 = n1;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        o[dt][0] *= al0;
        o[dt][1] *= al1;
        o[dt][2] *= al0;
        o[dt][3] *= al1;
      }
      const float p0 = exp2f(sv[0] - n0), p1 = exp2f(sv[1] - n1);
      const float p2 = exp2f(sv[2] - n0), p3 = exp2f(sv[3] - n1);
      l0 = l0 * al0 + (p0 + p2);
      l1 = l1 * al1 + (p1 + p3);
      const uint32_t pb0 = movm_t(pack_bf16(p0, p1));
      const uint32_t pb1 = movm_t(pack_bf16(p2, p3));
      // ---- rows past the sequence may hold anything: zero them in V
      if (ntok < 16) {
        const int chunks = (16 - ntok) * kHalves * 8;
        for (int e = lane; e < chunks; e += 32) {
          const int r = ntok + e / (kHalves * 8);
          const int hh = (e / 8) % kHalves;
          *reinterpret_cast<uint4*>(st + kPartBytes + hh * kTileBytes + r * 128 + (e % 8) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // ---- O^T[d x 8] += V^T[d x 16] . P^T[16 x 8]
      {
        const int r = (j >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          uint32_t a[4];
          ldsm_x4_t(vb + swz(r, dt * 16 + (j & 1) * 8), a);
          mma16816(o[dt], a, pb0, pb1);
        }
      }
    }

    // After the last step of a piece; l0 and l1 are the whole columns' sums by then.
    __device__ __forceinline__ void end() {}
  };
};

// ------------------------------------------------------------ 8-bit pages
// The same step on e4m3 elements with a power of two a row. K and V become fp16 in
// registers (exactly; half a conversion an element) and the products run on the fp16
// m16n8k16: fp32 accumulators, queries and probabilities as two fp16 terms each (a bf16
// product could hold neither those terms' range nor, for the same work, their bits).
//   S^T[t] = 2^ek[t] * (K8 . (Q hi + Q lo)^T),  Q scaled by a power of two to below 2^15
//   O^T   += V8^T . (P hi + P lo)^T,            P = 2^((s - m) + ev - r + 7)
// The values' powers of two go into the probabilities, which have a reference r of their own
// (of s - m + ev), apart from m (of s), which the sum's terms go by: neither the sum nor the
// largest terms of O then depend on how the scales of different tokens lie. All of it is formed
// from s - m, which is exact where it counts: s + ev would round ev off large logits. The
// references move only when a score is more than 2^8 above them; until then O stays untouched.
// P's terms end at fp16's smallest step, 2^-25 where the largest P is 2^7 at least: a token
// whose P lies 2^-d below it keeps 32 - d bits, where an fp32 product would keep 24. Products
// of a narrower range (P scaled a stage at a time) would cost an fp32 multiply-add of all of O
// a stage. Groups of up to four heads are packed: the two terms are columns 0 - 3 and 4 - 7 of
// one product.
//
// Fragments are read with wide loads, not ldmatrix: a lane's 16 bytes of a K row are four
// k-steps (which channels a k-step holds is free, so long as Q agrees), and 16 bytes of
// each of four V rows are the A operand of 16 channels once the rows' bytes are paired
// (which channel an output position holds is free: channel() says it). Which token a row of
// the products holds is free too: at d = 128 rows 2i and 2i + 1 are tokens i and i + 4,
// whose 128-byte rows the swizzle sends to different halves, so that every load is free of
// bank conflicts; at d = 64 V's 8-byte loads take two passes.
//
// A 16-token step is some 300 instructions on half the bytes of a bf16 one, most of them
// conversions and byte pairing, in chains that eight warps do not cover: 12 warps (168
// registers; 16 at d = 64, where a lane holds half as much) and the references that stay took
// 30% of 4 x 128k tokens from 78 to 56 us. All of them stream at 6.7 TB/s; what is left of 55 us
// is 39 of bytes, 6 before the first arrive, 4 of CTAs that end at different times and 4 of
// joining their parts. Tried and dropped: the warps' states scaled before they are added
// (spills), the first copies ahead of the plan's last steps (what the first data wait for is all
// SMs' rings filling at once).
template <int kDim, int kPage, bool kPack>
struct Q8Pages {
  static constexpr int D = kDim, P = kPage, kWarps = D == 128 ? 12 : 16;
  static constexpr int kSubs = P / 16;
  static constexpr int kPartBytes = 16 * D;
  static constexpr int kStageBytes = 2 * kPartBytes;  // K then V: 4 KiB (d=128) or 2 KiB
  static constexpr int kExtraBytes = 32;              // the tokens' K scales, then their V scales
  static constexpr int kSlots = D == 128 ? 3 : 5;
  static constexpr bool kNanStays = true;
  // A CTA takes a stage for each of its warps at least: short lists go to fewer CTAs, whose
  // parts take less time to join (2k tokens of two heads: 17.9 us over all CTAs, 10.8 so).
  static constexpr int kMinPages = kWarps / kSubs;
  static constexpr float kMove = 8.f;  // m and r move when a score is more than 2^8 above them
  static constexpr float kTop = 7.f;   // 2^(7 + 8) is below fp16's largest number

  static __device__ __forceinline__ void issue(uint8_t* dst, uint8_t* extra, const CUtensorMap& tmK,
                                               const CUtensorMap& tmV, const DecParams& p, int row,
                                               int sub, uint64_t* bar, uint64_t pol) {
    mbar_arrive_expect_tx(bar, kStageBytes + kExtraBytes);
    tma_load_2d_hint(dst, &tmK, 0, row, bar, pol);
    tma_load_2d_hint(dst + kPartBytes, &tmV, 0, row, bar, pol);
    // [page, head][K, V][P]; row is the page and head's first plus 16 sub
    const uint8_t* sc = p.scales + 2 * (size_t)row - 16 * sub;
    if (P == 16) {
      bulk_g2s_hint(extra, sc, 32, bar, pol);
    } else {
      bulk_g2s_hint(extra, sc, 16, bar, pol);
      bulk_g2s_hint(extra + 16, sc + P, 16, bar, pol);
    }
  }

  // Row r of a part at its 16-byte chunk c.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
  // Token (below 8) that row r of the products holds; row r + 8 holds it + 8.
  static __device__ __forceinline__ int token(int r) { return D == 128 ? (r & 1) << 2 | r >> 1 : r; }
  static __device__ __forceinline__ int channel(int pos) {
    const int r = pos & 7, hi = pos >> 3 & 1, dt = pos >> 4;
    return (D == 128 ? (r & 1) << 2 | r >> 1 : r) * (D / 8) + 2 * dt + hi;
  }
  static __device__ __forceinline__ uint32_t f16x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
  }
  static __device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
  }
  static __device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // Two floats as fp16 and what that leaves of them.
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_f16(x, y);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack_f16(x - h.x, y - h.y);
  }
  // 2^e of a scale byte e + 127 (255: NaN; 0, which no append writes, is 2^-127), and e.
  static __device__ __forceinline__ float power(uint32_t c) {
    return __uint_as_float(max(c << 23, 1u << 22) + (((c + 1) & 256) << 14));
  }
  static __device__ __forceinline__ float exponent(uint32_t c) {
    return c == 255 ? __uint_as_float(0x7fc00000u) : (float)((int)c - 127);
  }

  struct State {
    float m0, m1, l0, l1;
    float o[D / 16][4];
    float u0, u1;        // kTop - r of the two columns
    float qs0, qs1;      // the power of two that their queries were divided by
    uint32_t qf[D / 16][2];                // the first terms; packed: of columns 4 .. 7 the second
    uint32_t qlo[kPack ? 1 : D / 16][2];   // the second terms

    __device__ __forceinline__ void load_q(const DecParams& p, int seg, int gid, int tq) {
      const int qb = seg / p.Hkv, qh = seg % p.Hkv, head = kPack ? gid & 3 : gid;
      const bool live = head < p.g;
      const float* qr = p.q + ((size_t)qb * p.Hq + qh * p.g + (live ? head : 0)) * D;
      float2 v[D / 16][2];
      uint32_t top = 0;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float2& x = v[kk][half];
          x = make_float2(0.f, 0.f);
          // k-step kk is word kk % 4 of the lane's chunk tq + 4 (kk / 4)
          const int c = (tq + 4 * (kk / 4)) * 16 + (kk % 4) * 4 + 2 * half;
          if (live) x = *reinterpret_cast<const float2*>(qr + c);
          x.x *= p.scale_log2;
          x.y *= p.scale_log2;
          top = max(top, max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu));
        }
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      // the largest in [2^14, 2^15); a zero, infinite or NaN row as it is
      int e = (int)(top >> 23) - 127 - 14;
      e = top == 0 || top >= 0x7f800000u ? 0 : max(e, -126);
      const float inv = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t hi, lo;
          split(v[kk][half].x * inv, v[kk][half].y * inv, hi, lo);
          qf[kk][half] = kPack && gid >= 4 ? lo : hi;
          if (!kPack) qlo[kPack ? 0 : kk][half] = lo;
        }
      // columns 2 tq and 2 tq + 1 are loaded by the lanes whose gid they are
      const float pw = __uint_as_float((uint32_t)(127 + min(e, 126)) << 23);
      qs0 = __shfl_sync(kFull, pw, 8 * tq);
      qs1 = __shfl_sync(kFull, pw, 8 * tq + 4);
    }

    __device__ __forceinline__ void start() {
      m0 = m1 = -INFINITY, u0 = u1 = INFINITY, l0 = l1 = 0.f;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) o[dt][0] = o[dt][1] = o[dt][2] = o[dt][3] = 0.f;
    }

    __device__ __forceinline__ void step(uint8_t* st, const uint8_t* extra, int ntok, int lane) {
      const int gid = lane >> 2, tq = lane & 3, tok = token(gid);
      // ---- S^T[16 x 8] = K[16 x d] . Q^T[d x 8]
      float sv[4];
      {
        float acc[kPack ? 2 : 4][4] = {};  // chains: even and odd k-steps
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh) {
          const uint4 x = *reinterpret_cast<const uint4*>(st + at(tok, tq + 4 * hh));
          const uint4 y = *reinterpret_cast<const uint4*>(st + at(tok + 8, tq + 4 * hh));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int kk = 4 * hh + w;
            const uint32_t a[4] = {f16x2(xw[w] & 0xffff), f16x2(yw[w] & 0xffff), f16x2(xw[w] >> 16),
                                   f16x2(yw[w] >> 16)};
            mma(acc[kk & 1], a, qf[kk][0], qf[kk][1]);
            if (!kPack) mma(acc[kPack ? 0 : 2 + (kk & 1)], a, qlo[kPack ? 0 : kk][0], qlo[kPack ? 0 : kk][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sv[i] = acc[0][i] + acc[1][i];
        if (!kPack) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sv[i] += acc[kPack ? 0 : 2][i] + acc[kPack ? 0 : 3][i];
        }
      }
      if (ntok < 16) {  // rows past the sequence may hold anything: zero them in V
        for (int e = lane; e < (16 - ntok) * (D / 16); e += 32)
          *reinterpret_cast<uint4*>(st + kPartBytes + ntok * D + e * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
      }
      uint32_t h0, h1, w0 = 0, w1 = 0;  // P^T fragments: rows below 8 and from 8 on
      if constexpr (kPack) {
        // Lanes tq and tq ^ 2 hold the two terms' columns of the same heads: the first takes
        // rows below 8, the second the others, so that no exponential is computed twice.
        const bool low = tq < 2;
        const float g0 = __shfl_xor_sync(kFull, low ? sv[2] : sv[0], 2);
        const float g1 = __shfl_xor_sync(kFull, low ? sv[3] : sv[1], 2);
        const int t = low ? tok : tok + 8;
        const float k = power(extra[t]);
        float ev = exponent(extra[16 + t]);
        float x0 = ((low ? sv[0] : sv[2]) + g0) * (qs0 * k), x1 = ((low ? sv[1] : sv[3]) + g1) * (qs1 * k);
        if (t >= ntok) x0 = x1 = -INFINITY, ev = 0.f;
        float t0 = x0 - m0, t1 = x1 - m1, y0 = t0 + (ev + u0), y1 = t1 + (ev + u1);
        const bool moves = fmaxf(fmaxf(t0, t1), fmaxf(y0, y1) - kTop) > kMove;
        if (__any_sync(kFull, moves)) {
          move_m(x0, x1);
          t0 = x0 - m0, t1 = x1 - m1;
          move_r(t0 + ev, t1 + ev);
          y0 = t0 + (ev + u0), y1 = t1 + (ev + u1);
        }
        l0 += ex2(t0);
        l1 += ex2(t1);
        uint32_t hi, lo;
        split(ex2(y0), ex2(y1), hi, lo);
        const uint32_t got = __shfl_xor_sync(kFull, low ? lo : hi, 2);
        h0 = movm_t(low ? hi : got), h1 = movm_t(low ? got : lo);
      } else {
        const float k0 = power(extra[tok]), k1 = power(extra[tok + 8]);
        float e0 = exponent(extra[16 + tok]), e1 = exponent(extra[24 + tok]);
        sv[0] *= qs0 * k0, sv[1] *= qs1 * k0, sv[2] *= qs0 * k1, sv[3] *= qs1 * k1;
        if (tok >= ntok) sv[0] = sv[1] = -INFINITY, e0 = 0.f;
        if (tok + 8 >= ntok) sv[2] = sv[3] = -INFINITY, e1 = 0.f;
        float t[4], y[4];
        auto terms = [&]() {
          t[0] = sv[0] - m0, t[1] = sv[1] - m1, t[2] = sv[2] - m0, t[3] = sv[3] - m1;
          y[0] = t[0] + (e0 + u0), y[1] = t[1] + (e0 + u1);
          y[2] = t[2] + (e1 + u0), y[3] = t[3] + (e1 + u1);
        };
        terms();
        const bool moves = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])),
                                 fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) - kTop) > kMove;
        if (__any_sync(kFull, moves)) {
          move_m(fmaxf(sv[0], sv[2]), fmaxf(sv[1], sv[3]));
          move_r(fmaxf(sv[0] - m0 + e0, sv[2] - m0 + e1), fmaxf(sv[1] - m1 + e0, sv[3] - m1 + e1));
          terms();
        }
        l0 += ex2(t[0]) + ex2(t[2]);
        l1 += ex2(t[1]) + ex2(t[3]);
        split(ex2(y[0]), ex2(y[1]), h0, w0);
        split(ex2(y[2]), ex2(y[3]), h1, w1);
        h0 = movm_t(h0), h1 = movm_t(h1), w0 = movm_t(w0), w1 = movm_t(w1);
      }
      // ---- O^T[d x 8] += V^T[d x 16] . P^T[16 x 8]
      constexpr int kWords = D / 32;  // of a lane's d / 8 bytes of a row
      uint32_t x[4][kWords];          // rows 2 tq, 2 tq + 1 of the products, and those + 8
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = token(2 * tq + (i & 1)) + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint4 y = *reinterpret_cast<const uint4*>(st + kPartBytes + at(t, tok));
          x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
        } else {
          const uint2 y = *reinterpret_cast<const uint2*>(st + kPartBytes + at(t, gid >> 1) + (gid & 1) * 8);
          x[i][0] = y.x, x[i][1] = y.y;
        }
      }
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        // bytes 2 (dt % 2) and + 1 of both rows, side by side
        const uint32_t pick = dt & 1 ? 0x7362 : 0x5140;
        const uint32_t y0 = __byte_perm(x[0][dt / 2], x[1][dt / 2], pick);
        const uint32_t y1 = __byte_perm(x[2][dt / 2], x[3][dt / 2], pick);
        const uint32_t a[4] = {f16x2(y0 & 0xffff), f16x2(y0 >> 16), f16x2(y1 & 0xffff),
                               f16x2(y1 >> 16)};
        mma(o[dt], a, h0, h1);
        if (!kPack) mma(o[dt], a, w0, w1);
      }
    }

    // The largest of a column's tokens; x: this lane's of the stage.
    static __device__ __forceinline__ float of_column(float x) {
#pragma unroll
      for (int off = kPack ? 2 : 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
      return x;
    }
    // A new reference m: the largest score so far. r is of what lies above m: it moves against it.
    __device__ __forceinline__ void move_m(float b0, float b1) {
      b0 = fmaxf(m0, of_column(b0)), b1 = fmaxf(m1, of_column(b1));
      l0 *= exp2f(m0 - b0), l1 *= exp2f(m1 - b1);
      u0 += b0 - m0, u1 += b1 - m1;
      m0 = b0, m1 = b1;
    }
    // A new reference r, after m: the largest score above m with its value's scale so far.
    __device__ __forceinline__ void move_r(float c0, float c1) {
      c0 = fminf(u0, kTop - of_column(c0)), c1 = fminf(u1, kTop - of_column(c1));
      const float f0 = exp2f(c0 - u0), f1 = exp2f(c1 - u1);
      u0 = c0, u1 = c1;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        o[dt][0] *= f0;
        o[dt][1] *= f1;
        o[dt][2] *= f0;
        o[dt][3] *= f1;
      }
    }

    // O to the scale of m. A NaN sum keeps a finite m, so that the merges carry it on. 2^-u may
    // be as small as fp32 holds no more in full (values of the smallest scales): two steps.
    __device__ __forceinline__ void end() {
      if (kPack) {
        l0 += __shfl_xor_sync(kFull, l0, 2);
        l1 += __shfl_xor_sync(kFull, l1, 2);
      }
      if (l0 != l0) m0 = 0.f;
      if (l1 != l1) m1 = 0.f;
      float f[2], g[2];  // of each column: the fraction and half of the power, the other half
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float u = i ? u1 : u0, x = u == INFINITY ? 0.f : -u, whole = rintf(x);
        const int n = (int)fminf(fmaxf(whole, -200.f), 200.f), half = n >> 1;
        f[i] = exp2f(x - whole) * __int_as_float((127 + half) << 23);
        g[i] = __int_as_float((127 + n - half) << 23);
      }
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[dt][i] *= f[i & 1];
          o[dt][i] *= g[i & 1];
          if (kPack) o[dt][i] += __shfl_xor_sync(kFull, o[dt][i], 2);  // the two terms' columns
        }
      }
    }
  };
};

__device__ __forceinline__ int seg_of(const int* prefix, int S, int pos) {
  int lo = 0, hi = S - 1;  // largest s with prefix[s] <= pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Log-sum-exp merge of four output elements (query column col, channels
// o_off .. o_off + 3 with o_off = col * d + channel) over the np partials
// (m, l, o) of a segment, stored slot_floats apart from base: pieces are
// folded in CTA order with an online rescale in the log2 domain, eight
// pieces' loads in flight at once. The partials were written by other CTAs
// of this grid: loads go through L2.
__device__ __forceinline__ void fold_pieces4(const float* base, int np, int slot_floats, int col,
                                             int o_off, float& M, float& L, float4& acc) {
  M = -INFINITY;
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kU = 8;
  for (int c = 0; c < np; c += kU) {
    float m[kU], l[kU];
    float4 o[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      m[u] = -INFINITY;
      if (c + u < np) {
        const float* q = base + (size_t)(c + u) * slot_floats;
        m[u] = __ldcg(q + col);
        l[u] = __ldcg(q + 8 + col);
        o[u] = __ldcg(reinterpret_cast<const float4*>(q + 16 + o_off));
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (m[u] == -INFINITY) continue;  // a piece with no valid token (or none)
      if (m[u] > M) {
        const float sc = exp2f(M - m[u]);  // 0 while M is still -inf
        acc.x *= sc;
        acc.y *= sc;
        acc.z *= sc;
        acc.w *= sc;
        L *= sc;
        M = m[u];
      }
      const float w = exp2f(m[u] - M);
      acc.x += w * o[u].x;
      acc.y += w * o[u].y;
      acc.z += w * o[u].z;
      acc.w += w * o[u].w;
      L += w * l[u];
    }
  }
}

// floats of a warp's part of the merge area, and of a partial: m[8], l[8], o[8][D]
template <class F>
constexpr int kStateFloats = 2 * 8 + 8 * F::D;

template <class F>
__global__ void __launch_bounds__(F::kWarps * 32, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const DecParams p) {
  constexpr int D = F::D, P = F::P, kThreads = F::kWarps * 32;
  constexpr int kRingBytes = F::kWarps * F::kSlots * F::kStageBytes;
  constexpr int kSlotFloats = kStateFloats<F>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;                                                  // [warp][slot][stage]
  float* merge = reinterpret_cast<float*>(ring + kRingBytes);
  uint8_t* extra = reinterpret_cast<uint8_t*>(merge + F::kWarps * kSlotFloats);  // [warp][slot]
  uint64_t* full = reinterpret_cast<uint64_t*>(extra + F::kWarps * F::kSlots * F::kExtraBytes);
  int* meta = reinterpret_cast<int*>(full + F::kWarps * F::kSlots);     // [warp][slot]: tokens
  int* flags = meta + F::kWarps * F::kSlots;                             // [0..1] merge, [8..] scan
  int* prefix = flags + 48;                                              // [S + 1]

  // Split weight at the start of each segment, W(prefix[s]) = prefix[s] +
  // piece_cost * (non-empty segments before s); [S + 1] ints in the ring,
  // read only while planning, before the first copy lands there.
  int* wstart = reinterpret_cast<int*>(ring);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.B * p.Hkv;
  const int G = gridDim.x, cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < F::kWarps * F::kSlots; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
    prefix[0] = 0;
    wstart[0] = 0;
  }
  pdl_launch_dependents();
  pdl_wait_predecessor();
  // ---- self-plan: lengths (validated) -> inclusive prefix of pages and of
  // non-empty segments in shared memory
  const int per = ceil_div(S, kThreads);
  const int a0 = min(S, tid * per), a1 = min(S, a0 + per);
  int run = 0, nzr = 0, longest = 0;
  // Range errors are collected and reported once after the loop: an atomic
  // on the error word between loads would keep the later loads in order.
  uint32_t bad = 0;
  const long long t_cap = (long long)p.max_pages * P;
  for (int s = a0; s < a1; ++s) {  // wstart[s + 1] first holds non-empty segments up to s
    int Tb = p.seq_lens[s / p.Hkv];
    int n = p.lens[s];
    if (Tb < 0 || (long long)Tb > t_cap) {
      bad |= ASP_DEVERR_SEQ_RANGE;
      Tb = Tb < 0 ? 0 : (int)t_cap;
    }
    const int n_b = ceil_div(Tb, P);
    if (n < 0 || n > n_b) {
      bad |= ASP_DEVERR_LEN_RANGE;
      n = n < 0 ? 0 : n_b;
    }
    run += n;
    longest = max(longest, n);
    nzr += n > 0 ? 1 : 0;
    prefix[s + 1] = run;
    wstart[s + 1] = nzr;
  }
  if (bad) report(p.err, bad);
  int x = run, y = nzr;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int xo = __shfl_up_sync(kFull, x, o), yo = __shfl_up_sync(kFull, y, o);
    if (lane >= o) {
      x += xo;
      y += yo;
    }
  }
  if (F::kMinPages > 1) longest = __reduce_max_sync(kFull, longest);
  if (lane == 31) {
    if (F::kMinPages > 1) meta[warp] = longest;  // unused until the first copies
    flags[8 + warp] = x;
    flags[8 + F::kWarps + warp] = y;
  }
  __syncthreads();
  int off = 0, offn = 0, total = 0, nonempty = 0;
  for (int w = 0; w < F::kWarps; ++w) {
    if (w < warp) {
      off += flags[8 + w];
      offn += flags[8 + F::kWarps + w];
    }
    total += flags[8 + w];  // < 2^31, checked on the host
    nonempty += flags[8 + F::kWarps + w];
    if (F::kMinPages > 1) longest = max(longest, meta[w]);
  }
  off += x - run;
  offn += y - nzr;
  // Every share of the weight must hold a page (X + 1 <= share size), so that
  // the CTAs holding pieces of one segment are consecutive, as the merge at
  // the end assumes (it folds the partial slots of CTAs cf..cl): X is capped
  // at total / G - 1.
  const int X = max(0, min(p.piece_cost, total / G - 1));
  // Whole lists (8-bit pages): where no list is long, each goes to one CTA, which then writes it
  // out, rather than in even shares that are joined. In stages that a CTA takes in the same
  // time (12 or 16 warps take one each in about a microsecond): the end of a piece costs 3 a
  // warp, parts to be joined 7. Measured, even shares and whole lists: 8 lists of one page 20.9
  // and 8.0 us, 68 of some 17 pages of 32 tokens 21.2 and 15.3.
  bool lists_whole = false;
  if (F::kMinPages > 1) {
    const int end = 3 * F::kWarps, parts = 7 * F::kWarps;
    const long long by_list = (long long)ceil_div(nonempty, G) * ((long long)longest * F::kSubs + end);
    const long long even = (long long)total * F::kSubs / G + (nonempty / G + 1) * end + parts;
    lists_whole = by_list <= even;
  }
  for (int s = a0; s < a1; ++s) {
    prefix[s + 1] += off;
    const int lists = wstart[s + 1] + offn;
    wstart[s + 1] = lists_whole ? lists : prefix[s + 1] + X * lists;  // whole: a list weighs 1
  }
  __syncthreads();

  // Weighted split: page j of segment s weighs 1, plus X when j = prefix[s];
  // W(j) = weight of the pages before j. CTA c takes the pages whose W lies
  // in the c-th even share of the total weight (< 2^31: the host checks
  // B * Hkv * (max_pages + 128)).
  const int wtotal = wstart[S];
  // CTAs with work: one a page (or whole list) as far as they go, or, where the format asks for
  // more pages a CTA, one a non-empty list at least
  const int geff = min(min(G, wtotal), F::kMinPages == 1 || lists_whole
                                           ? wtotal
                                           : max(nonempty, ceil_div(wtotal, F::kMinPages)));
  const EvenSplit split(wtotal, geff > 0 ? geff : 1);
  auto weight_at = [&](int s, int j) {  // W(j) for page j of segment s
    return j == prefix[s] || lists_whole ? wstart[s] : j + (wstart[s] - prefix[s]) + X;
  };
  auto page_at = [&](int cut) {  // first page j with W(j) >= cut
    if (cut >= wtotal) return total;
    int lo = 0, hi = S - 1;  // largest s with wstart[s] <= cut: a non-empty segment
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (wstart[mid] <= cut) lo = mid; else hi = mid - 1;
    }
    const int j0 = prefix[lo];
    if (cut <= wstart[lo]) return j0;
    return min(max(cut - (wstart[lo] - j0) - X, j0 + 1), prefix[lo + 1]);
  };
  long long beg = 0, end = 0;
  if (cta < geff) {
    beg = page_at(split.begin(cta));
    end = page_at(split.end(cta));
  }
  const float kLn2 = 0.69314718055994530942f;
  auto lse_of = [&](float M, float L) {
    return L > 0.f ? (M + log2f(L)) * kLn2 : F::kNanStays && L != 0.f ? L : -INFINITY;
  };

  // segments with an empty list: out = 0, lse = -inf
  for (int s = cta; s < S; s += G) {
    if (prefix[s + 1] != prefix[s]) continue;
    const int b = s / p.Hkv, h = s % p.Hkv;
    for (int e = tid; e < p.g * D; e += kThreads)
      p.out[((size_t)b * p.Hq + h * p.g + e / D) * D + e % D] = 0.f;
    for (int e = tid; e < p.g; e += kThreads) p.lse[(size_t)b * p.Hq + h * p.g + e] = -INFINITY;
  }
  // Only a CTA's first and last pieces can hold part of a segment (a middle
  // piece holds a whole one). For each, the CTAs cf..cf+np-1 holding that
  // segment: the last of them to finish merges it.
  int seg_a = -1, seg_b = -1, cf_a = 0, cf_b = 0, np_a = 0, np_b = 0;
  if (beg < end) {
    auto holders = [&](int s, int& cf) {
      cf = split.part_of(wstart[s]);
      return split.part_of(weight_at(s, prefix[s + 1] - 1)) - cf + 1;
    };
    seg_a = seg_of(prefix, S, (int)beg);
    seg_b = seg_of(prefix, S, (int)(end - 1));
    np_a = holders(seg_a, cf_a);
    if (seg_b != seg_a) np_b = holders(seg_b, cf_b);
  }
  __syncthreads();  // the weights are done with: the ring is free for copies
  if (beg >= end) return;
  if (tid == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }

  // ---- this warp's stages: CTA stage it = warp + kWarps n covers page position
  // beg + it / kSubs, sub-tile it % kSubs (= warp % kSubs, since kSubs | kWarps)
  static_assert(F::kWarps % F::kSubs == 0 && 8 + 2 * F::kWarps <= 48);
  const long long nst = (end - beg) * F::kSubs;
  const int n_total = nst > warp ? (int)((nst - warp + F::kWarps - 1) / F::kWarps) : 0;
  const int sub = warp % F::kSubs;
  uint8_t* my_ring = ring + warp * F::kSlots * F::kStageBytes;
  uint64_t* my_full = full + warp * F::kSlots;
  int* my_meta = meta + warp * F::kSlots;
  uint8_t* my_extra = extra + warp * F::kSlots * F::kExtraBytes;

  // Lookups for warp stages [nb, nb + 32): lane j owns stage nb + j. The
  // list entry (and sequence length) are fetched two batches ahead and the
  // block-table entry one batch ahead of the stages being issued.
  constexpr int kNoPage = INT_MIN;
  auto lookup_list = [&](int nb, int& seg, int& T, int& lp) {
    seg = 0; T = 0; lp = -1;
    const int n = nb + lane;
    if (n < n_total) {
      const long long pos = beg + (warp + (long long)F::kWarps * n) / F::kSubs;
      seg = seg_of(prefix, S, (int)pos);
      T = __ldg(p.seq_lens + seg / p.Hkv);
      lp = __ldg(p.lists + (size_t)seg * p.max_pages + (int)(pos - prefix[seg]));
    }
  };
  auto lookup_page = [&](int nb, int seg, int T, int lp) {
    int phys = kNoPage;
    if (nb + lane < n_total) {
      T = min(max(T, 0), p.max_pages * P);
      if (lp < 0 || lp >= ceil_div(T, P)) {
        if (sub == 0) report(p.err, ASP_DEVERR_LIST_RANGE);
      } else {
        phys = __ldg(p.bt + (size_t)(seg / p.Hkv) * p.max_pages + lp);
      }
    }
    return phys;
  };
  // Row of the sub-tile in the [rows, d] view (a multiple of 16, below 2^31), over 16, in bits
  // 5 - 31; valid tokens in it, 0 to 16, in bits 0 - 4.
  auto finalize = [&](int seg, int T, int lp, int phys) {
    if (phys == kNoPage) return 0u;
    if (phys < 0 || phys >= p.num_phys) {
      if (sub == 0) report(p.err, ASP_DEVERR_PAGE_RANGE);
      return 0u;
    }
    T = min(max(T, 0), p.max_pages * P);
    const int row = (phys * p.Hkv + seg % p.Hkv) * (P / 16) + sub;
    return (uint32_t)row << 5 | (uint32_t)min(16, max(0, min(P, T - lp * P) - 16 * sub));
  };

  int sB, TB, lpB, sC, TC, lpC, phB;
  uint32_t whatA;
  {
    int sA, TA, lpA;
    lookup_list(0, sA, TA, lpA);
    lookup_list(32, sB, TB, lpB);
    const int phA = lookup_page(0, sA, TA, lpA);
    whatA = finalize(sA, TA, lpA, phA);
    phB = lookup_page(32, sB, TB, lpB);
    lookup_list(64, sC, TC, lpC);
  }
  const uint64_t pol = l2_evict_first_policy();  // K/V pages are read once
  int ib = 0;   // first warp stage of batch A
  int ni = 0, slot_i = 0;  // next warp stage to issue, and its slot
  bool aborted = false;
  auto issue_next = [&]() {
    if (ni >= ib + 32) {  // rotate the lookup batches (warp-uniform)
      whatA = finalize(sB, TB, lpB, phB);
      ib += 32;
      const int phC = lookup_page(ib + 32, sC, TC, lpC);
      sB = sC; TB = TC; lpB = lpC; phB = phC;
      lookup_list(ib + 64, sC, TC, lpC);
    }
    const uint32_t what = __shfl_sync(kFull, whatA, ni - ib);
    if (lane == 0) {
      my_meta[slot_i] = what & 31;
      if (what & 31) {
        F::issue(my_ring + slot_i * F::kStageBytes, my_extra + slot_i * F::kExtraBytes, tmK, tmV, p,
                 (int)(what >> 5) * 16, sub, &my_full[slot_i], pol);
      } else {
        mbar_arrive(&my_full[slot_i]);
      }
    }
    ++ni;
    if (++slot_i == F::kSlots) slot_i = 0;
  };
  while (ni < min(F::kSlots, n_total)) issue_next();

  // ================================================================ pieces
  const int gid = lane >> 2, tq = lane & 3;
  int nc = 0, slot = 0, phase = 0;  // next warp stage to consume, its slot, the slot's phase
  int waited = 0;  // stages whose copies are known complete
  typename F::State st;
  long long pos = beg;
  st.load_q(p, seg_of(prefix, S, (int)pos), gid, tq);
  while (pos < end) {
    const int s = seg_of(prefix, S, (int)pos);
    const long long seg_lo = prefix[s], seg_hi = prefix[s + 1];
    const long long pe = seg_hi < end ? seg_hi : end;
    const int b = s / p.Hkv, h = s % p.Hkv;

    st.start();
    const long long it_end = (pe - beg) * F::kSubs;
    const int nc_end =  // of this piece
        it_end > warp ? (int)min((long long)n_total, (it_end - warp + F::kWarps - 1) / F::kWarps) : 0;
    while (nc < nc_end) {
      if (!aborted) {
        // warp-uniform outcome: the refill below shuffles across all lanes
        const bool got = mbar_wait(&my_full[slot], phase);
        if (__all_sync(kFull, got)) {
          waited = nc + 1;
        } else {
          if (lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
          aborted = true;
        }
      }
      const int ntok = my_meta[slot];
      if (!aborted && ntok > 0)
        st.step(my_ring + slot * F::kStageBytes, my_extra + slot * F::kExtraBytes, ntok, lane);
      // the slot's reads (and any zeroing writes) are done: refill it
      __syncwarp();
      if (!aborted && ni < n_total) {
        fence_proxy_async_smem();
        issue_next();
      }
      ++nc;
      if (++slot == F::kSlots) slot = 0, phase ^= 1;
    }

    // ---- merge the warps' states of this piece
#pragma unroll
    for (int off2 = 4; off2 < 32; off2 <<= 1) {
      st.l0 += __shfl_xor_sync(kFull, st.l0, off2);
      st.l1 += __shfl_xor_sync(kFull, st.l1, off2);
    }
    st.end();
    float* mw = merge + warp * kSlotFloats;  // m[8], l[8], o[8][D]
    if (gid == 0) {
      mw[2 * tq] = st.m0;
      mw[2 * tq + 1] = st.m1;
      mw[8 + 2 * tq] = st.l0;
      mw[8 + 2 * tq + 1] = st.l1;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      const int d0 = dt * 16 + gid;
      mw[16 + (2 * tq) * D + d0] = st.o[dt][0];
      mw[16 + (2 * tq + 1) * D + d0] = st.o[dt][1];
      mw[16 + (2 * tq) * D + d0 + 8] = st.o[dt][2];
      mw[16 + (2 * tq + 1) * D + d0 + 8] = st.o[dt][3];
    }
    if (pe < end) st.load_q(p, seg_of(prefix, S, (int)pe), gid, tq);  // next piece's queries overlap the merge
    __syncthreads();
    const bool whole = (pos == seg_lo) && (pe == seg_hi);
    float* pslot = p.partials + (size_t)(s + cta) * p.slot_floats;
    for (int e = tid; e < p.g * D; e += kThreads) {
      const int col = e / D, d = e % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < F::kWarps; ++w) M = fmaxf(M, merge[w * kSlotFloats + col]);
      float L = 0.f, acc = 0.f;
      if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < F::kWarps; ++w) {
          const float* q = merge + w * kSlotFloats;
          const float sc = exp2f(q[col] - M);
          L += sc * q[8 + col];
          acc += sc * q[16 + col * D + d];
        }
      }
      if (whole) {
        const size_t row = (size_t)b * p.Hq + h * p.g + col;
        p.out[row * D + F::channel(d)] = L > 0.f ? acc / L : F::kNanStays ? L : 0.f;
        if (d == 0) p.lse[row] = lse_of(M, L);
      } else {
        pslot[16 + col * D + d] = acc;
        if (d == 0) {
          pslot[col] = M;
          pslot[8 + col] = L;
        }
      }
    }
    __syncthreads();  // the merge area is rewritten by the next piece
    pos = pe;
  }
  // never leave the CTA with copies in flight (only after a timeout can any remain)
  if (lane == 0)
    for (int n = waited; n < ni; ++n) mbar_wait(&my_full[n % F::kSlots], (n / F::kSlots) & 1);

  // ---- split segments: count this CTA's pieces in; the CTA that brings a
  // segment's count to its number of pieces merges that segment's partials
  // (in CTA order, so the result does not depend on which CTA it is) and
  // resets the count for the next call.
  if (np_a < 2 && np_b < 2) return;  // CTA-uniform
  __syncthreads();  // every partial store of this CTA has been issued
  if (tid == 0) {
    __threadfence();  // ... and is ordered before the arrivals (cumulative over the CTA)
    const int oa = np_a > 1 ? atomicAdd(&p.arrivals[seg_a], 1) : -1;
    const int ob = np_b > 1 ? atomicAdd(&p.arrivals[seg_b], 1) : -1;
    flags[0] = np_a > 1 && oa == np_a - 1 ? 1 : 0;
    flags[1] = np_b > 1 && ob == np_b - 1 ? 1 : 0;
    __threadfence();  // the other CTAs' partials, seen through the arrivals, before the loads
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!flags[k]) continue;  // CTA-uniform
    const int ms = k ? seg_b : seg_a, cf = k ? cf_b : cf_a, np = k ? np_b : np_a;
    const float* base = p.partials + (size_t)(ms + cf) * p.slot_floats;
    const int mb = ms / p.Hkv, mh = ms % p.Hkv;
    for (int e = 4 * tid; e < p.g * D; e += 4 * kThreads) {  // one pass when g * d <= 1024
      const int col = e / D, d = e % D;
      float M, L;
      float4 acc;
      fold_pieces4(base, np, p.slot_floats, col, e, M, L, acc);
      const size_t row = (size_t)mb * p.Hq + mh * p.g + col;
      float* o = p.out + row * D;  // the caller's buffer: 4-byte alignment only
      const float none = F::kNanStays ? L : 0.f;
      o[F::channel(d)] = L > 0.f ? acc.x / L : none;
      o[F::channel(d + 1)] = L > 0.f ? acc.y / L : none;
      o[F::channel(d + 2)] = L > 0.f ? acc.z / L : none;
      o[F::channel(d + 3)] = L > 0.f ? acc.w / L : none;
      if (d == 0) p.lse[row] = lse_of(M, L);
    }
    if (tid == 0) p.arrivals[ms] = 0;
  }
}

// ----------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

}  // namespace

cudaError_t encode_bf16_2d_swizzled(CUtensorMap* map, const void* base, unsigned long long inner,
                                    unsigned long long rows, unsigned box_inner, unsigned box_rows) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_bf16_3d_swizzled(CUtensorMap* map, const void* base,
                                    const unsigned long long (&dims)[3],
                                    const unsigned long long (&strides)[2],
                                    const unsigned (&box)[3]) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
  cuuint64_t st[2] = {strides[0], strides[1]};
  cuuint32_t bx[3] = {box[0], box[1], box[2]};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), d, st, bx,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

// [rows = num_phys*Hkv*P, D] viewed as 2-D; box = [16 rows x 64 channels] of bf16, or 16 whole
// rows of bytes, swizzled over their width.
cudaError_t make_page_map(CUtensorMap* map, const void* base, long long rows, int D, bool q8) {
  if (!q8)
    return encode_bf16_2d_swizzled(map, base, (unsigned long long)D, (unsigned long long)rows, 64,
                                   16);
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {(cuuint32_t)D, 16};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Dynamic shared memory of decode_kernel: 1 KiB alignment slack, the ring,
// the warp-merge area, per-slot metadata, scales and mbarriers, flags, prefix[S + 1].
template <class F>
size_t decode_smem_bytes(int S) {
  return 1024 + (size_t)F::kWarps * F::kSlots * F::kStageBytes + F::kWarps * kStateFloats<F> * 4 +
         F::kWarps * F::kSlots * (sizeof(int) + F::kExtraBytes + 8) + 48 * 4 + (size_t)(S + 1) * 4;
}

int max_optin_smem() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
    return 0;
  return v;
}

template <class F>
cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  const int S = kv.batch * kv.num_kv_heads;
  const size_t smem = decode_smem_bytes<F>(S);
  cudaError_t e = set_max_dynamic_smem((const void*)decode_kernel<F>, (int)smem);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)kv.num_phys_pages * kv.num_kv_heads * F::P;
  CUtensorMap tk, tv;
  const void* k = a.q8 ? (const void*)a.q8->k : kv.k_cache;
  const void* v = a.q8 ? (const void*)a.q8->v : kv.v_cache;
  if ((e = make_page_map(&tk, k, rows, F::D, a.q8 != nullptr)) != cudaSuccess) return e;
  if ((e = make_page_map(&tv, v, rows, F::D, a.q8 != nullptr)) != cudaSuccess) return e;
  DecParams p{a.q, a.lists, a.lens, kv.block_table, kv.seq_lens, a.out, a.lse, a.partials,
              a.arrivals, a.q8 ? a.q8->scales : nullptr, a.err, kv.batch, kv.num_q_heads,
              kv.num_kv_heads, kv.num_q_heads / kv.num_kv_heads, kv.max_pages, kv.num_phys_pages,
              a.slot_floats, decode_piece_cost(F::D, F::P), a.sm_scale * 1.4426950408889634f};
  return launch_pdl(decode_kernel<F>, dim3(a.grid), dim3(F::kWarps * 32), smem, stream, tk, tv, p);
}

// The deeper ring when its shared memory (which grows with the segment
// count through the prefix of list lengths) fits the device's per-block limit.
template <int D, int P>
cudaError_t launch_decode_dp(const DecodeArgs& a, cudaStream_t stream) {
  const int S = a.kv->batch * a.kv->num_kv_heads;
  if (decode_smem_bytes<Bf16Pages<D, P, true>>(S) <= (size_t)max_optin_smem())
    return launch_decode_t<Bf16Pages<D, P, true>>(a, stream);
  return launch_decode_t<Bf16Pages<D, P, false>>(a, stream);
}

template <bool kPack>
cudaError_t launch_q8(const DecodeArgs& a, cudaStream_t stream) {
  const int d = a.kv->head_dim, P = a.kv->page_size;
  if (d == 128 && P == 16) return launch_decode_t<Q8Pages<128, 16, kPack>>(a, stream);
  if (d == 128 && P == 32) return launch_decode_t<Q8Pages<128, 32, kPack>>(a, stream);
  if (d == 128 && P == 64) return launch_decode_t<Q8Pages<128, 64, kPack>>(a, stream);
  if (d == 64 && P == 16) return launch_decode_t<Q8Pages<64, 16, kPack>>(a, stream);
  if (d == 64 && P == 32) return launch_decode_t<Q8Pages<64, 32, kPack>>(a, stream);
  if (d == 64 && P == 64) return launch_decode_t<Q8Pages<64, 64, kPack>>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  const int d = a.kv->head_dim, P = a.kv->page_size;
  if (d == 128 && P == 16) return launch_decode_dp<128, 16>(a, stream);
  if (d == 128 && P == 32) return launch_decode_dp<128, 32>(a, stream);
  if (d == 128 && P == 64) return launch_decode_dp<128, 64>(a, stream);
  if (d == 64 && P == 16) return launch_decode_dp<64, 16>(a, stream);
  if (d == 64 && P == 32) return launch_decode_dp<64, 32>(a, stream);
  if (d == 64 && P == 64) return launch_decode_dp<64, 64>(a, stream);
  return cudaErrorInvalidValue;
}
// Groups of up to four heads are packed: all of 4 x 128k tokens, four heads a group, in 96.8 us
// instead of 105.0 at d = 64 and 144.0 instead of 144.5 at d = 128; 2k tokens of d = 64, all
// latency, in 11.4 instead of 10.9.
cudaError_t launch_q8_decode(const DecodeArgs& a, cudaStream_t stream) {
  return a.kv->num_q_heads / a.kv->num_kv_heads <= 4 ? launch_q8<true>(a, stream)
                                                     : launch_q8<false>(a, stream);
}

}  // namespace asp
