// norm_rotate.cu - new tokens into the paged cache: per-head norms of queries
// and keys, position rotation, the write of K and V into their pages and the
// fold of the keys into the page summaries, in one pass over the packed rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// One work item is one page of one request: the new tokens that fall into it. CTAs
// take items in turn; a loader warp looks the next ones up and streams their
// tokens' rows (contiguous in the packed array) through a ring of shared-memory stages.
// The angles of 16 tokens are computed once, in shared memory, for all heads.
//
// HBM gives the rows about as fast as the SMs can issue the arithmetic, so rows take few
// instructions (d / 8 lanes hold a row, a lane the two halves of four rotated pairs, so
// that a pair never crosses lanes; two-wide fp32 operations) and many warps cover one
// another's latencies: two CTAs an SM, in registers that do not spill (with all of the
// SM's memory given to the rings a spilled register comes back from L2). A warp keeps the
// same key heads for all tokens of an item, their channel minima and maxima in registers
// until the page is done: the summary is written once, without atomics.
//
// Measured: 16k new tokens of 48 heads (d = 128) in 93 us, 4.8 TB/s read and written; 76 us
// without norm and rotation, so it is the rows' chains of shuffles and fp32 work that keep it
// from the copy rate. More warps an SM, or two tokens at once, spill (135 us). 64 decoded
// tokens: 5.1 us.
//
// The angle: a frequency becomes a 64-bit fixed-point fraction of a turn, whose
// product with the integer position wraps exactly modulo one turn, so that
// position 2^31 is as exact as position 0 (in 32-bit floats an angle of 10^5
// radians is off by 0.004).
#include "tc.cuh"

namespace asp {
namespace {

constexpr int kWarps = 7;
constexpr int kThreads = (kWarps + 1) * 32;  // and a loader
constexpr int kCtas = 2;                     // CTAs of an SM
constexpr int kMaxStages = 16;
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
  int rot, nq, nk, stages, items;  // nq, nk: query and KV heads of a CTA
  float eps;
};

__device__ __forceinline__ float2 unpack(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float2 f) { return pack_bf16(f.x, f.y); }

__device__ __forceinline__ uint2 load4(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint2*>(p));
}

// A lane's eight channels of a row, two to an element: 0, 1 its first four, 2, 3 its second
// four. Halves rotated against each other: pair i is channel i of the first and of the
// second four; interleaved: channels 2i and 2i + 1 of the eight.
struct Row {
  float2 f[4];
  __device__ __forceinline__ void set(const uint2& a, const uint2& b) {
    f[0] = unpack(a.x), f[1] = unpack(a.y), f[2] = unpack(b.x), f[3] = unpack(b.y);
  }
  __device__ __forceinline__ uint2 first() const { return make_uint2(pack(f[0]), pack(f[1])); }
  __device__ __forceinline__ uint2 second() const { return make_uint2(pack(f[2]), pack(f[3])); }
  // kLanes lanes of a row; w: the lane's weights, as bf16
  template <int kLanes>
  __device__ __forceinline__ void norm(const uint2 (&w)[2], float inv_d, float eps) {
    float2 sq = mul2(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sq = fma2(f[i], f[i], sq);
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float r = rsqrtf(fmaf(ss, inv_d, eps));
    const float2 rr = make_float2(r, r);
    Row wf;
    wf.set(w[0], w[1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], wf.f[i]), rr);
  }
  // cs: (cos, sin) of the four pairs
  template <bool kInterleaved>
  __device__ __forceinline__ void turn(const float4 (&cs)[2]) {
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = i & 1 ? cs[i / 2].z : cs[i / 2].x, sn = i & 1 ? cs[i / 2].w : cs[i / 2].y;
        f[i] = make_float2(f[i].x * c - f[i].y * sn, f[i].y * c + f[i].x * sn);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = f[i], b = f[2 + i];
        const float2 c = make_float2(cs[i].x, cs[i].z), sn = make_float2(cs[i].y, cs[i].w);
        f[i] = fma2(b, make_float2(-sn.x, -sn.y), mul2(a, c));
        f[2 + i] = fma2(a, sn, mul2(b, c));
      }
    }
  }
};

// A work item, found by the loader warp; b < 0: no more.
struct Item {
  int b, page, lo, cnt;  // the new slots lo .. lo + cnt - 1, all in this page
  int row0, phys;        // the first's packed row; physical page, -1: none
};
constexpr int kItems = 3;      // items known ahead
constexpr int kTurnTokens = 16;  // tokens whose angles are computed together

// Shared memory of a CTA: the ring, then these.
template <int D>
struct Shared {
  float2 turn[2][kTurnTokens * (D / 2)];  // (cos, sin) of [token][pair]
  unsigned long long turns_of[D / 2];     // 2^64 * inv_freq / (2 pi), modulo 2^64
  Item item[kItems];
  uint64_t full[kMaxStages], empty[kMaxStages], item_full[kItems], item_empty[kItems], turn_full[2];
};

template <int D, int P, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kCtas) norm_rotate_kernel(const Params p) {
  constexpr int kLanes = D / 8;        // lanes of one row
  constexpr int kRows = 32 / kLanes;   // rows a warp takes at once
  static_assert(kWarps * kRows >= 8, "a group of key heads a warp at most");
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / kLanes, l = lane % kLanes;
  // this CTA's heads: a share of the query heads and of the KV heads
  const int q0 = blockIdx.y * p.nq, nq = max(0, min(p.nq, p.Hq - q0));
  const int k0 = blockIdx.y * p.nk, nk = max(0, min(p.nk, p.Hkv - k0));
  const int stage_bytes = (p.nq + 2 * p.nk) * D * 2;
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
    mbar_init(&sh.turn_full[0], kWarps);
    mbar_init(&sh.turn_full[1], kWarps);
    mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait_predecessor();
  const int half = p.rot / 2;
  if (tid < half) {
    double t = (double)p.inv_freq[tid] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    sh.turns_of[tid] = (unsigned long long)(t * 18446744073709551616.0);
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ loader
    if (p.q_offsets && blockIdx.x == 0 && blockIdx.y == 0) {  // every request's rows are checked
      for (int x = lane; x < p.B; x += 32)
        new_rows(p.q_offsets, x, clamp_seq_len(p.seq_lens[x], p.max_pages, P, p.err),
                 p.num_tokens, p.err);
    }
    const uint32_t bytes = (uint32_t)(nq + 2 * nk) * D * 2;
    const int Hall = p.Hq + 2 * p.Hkv;
    uint32_t tk = 0, n = 0;  // tokens loaded, items handed on
    bool ok = true;
    for (int it = blockIdx.x; ok; it += gridDim.x) {
      Item x{-1, 0, 0, 0, 0, -1};
      if (it < p.items) {
        int b = it, page_of_b = 0;  // one row per request: item b is request b
        if (p.q_offsets) {
          constexpr int kLog = P == 64 ? 6 : P == 32 ? 5 : 4;
          b = request_of_item(p.q_offsets, p.B, p.num_tokens, kLog, it, lane);
          if (b < 0) continue;
          page_of_b = it - first_item(p.q_offsets, b, p.num_tokens, kLog);
        }
        uint32_t* err = lane == 0 ? p.err : nullptr;
        const int T = clamp_seq_len(p.seq_lens[b], p.max_pages, P, err);
        const NewRows nr = new_rows(p.q_offsets, b, T, p.num_tokens, err);
        const int first = T - nr.n;  // slot of the first new token
        x.page = first / P + page_of_b;
        x.lo = max(first, x.page * P);
        x.cnt = min(T, (x.page + 1) * P) - x.lo;
        if (x.cnt <= 0) continue;
        x.b = b;
        x.row0 = nr.row0 + (x.lo - first);
        x.phys = p.bt[(size_t)b * p.max_pages + x.page];
        if (x.phys < 0 || x.phys >= p.num_phys) {
          report(err, ASP_DEVERR_PAGE_RANGE);
          x.phys = -1;
        }
      }
      const int slot = n % kItems;
      ok = __all_sync(kFull, mbar_wait(&sh.item_empty[slot], ((n / kItems) & 1) ^ 1));
      if (!ok) break;
      if (lane == 0) {
        sh.item[slot] = x;
        mbar_arrive(&sh.item_full[slot]);
      }
      ++n;
      if (x.b < 0) break;
      if (bytes == 0) continue;
      for (int t = 0; t < x.cnt; ++t, ++tk) {
        const int st = tk % p.stages;
        ok = __all_sync(kFull, mbar_wait(&sh.empty[st], ((tk / p.stages) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          const uint16_t* row = p.qkv + (size_t)(x.row0 + t) * Hall * D;
          uint8_t* dst = smem + st * stage_bytes;
          mbar_arrive_expect_tx(&sh.full[st], bytes);
          if (nq > 0) bulk_g2s(dst, row + q0 * D, nq * D * 2, &sh.full[st]);
          if (nk > 0) {
            dst += p.nq * D * 2;
            bulk_g2s(dst, row + (p.Hq + k0) * D, nk * D * 2, &sh.full[st]);
            bulk_g2s(dst + p.nk * D * 2, row + (p.Hq + p.Hkv + k0) * D, nk * D * 2, &sh.full[st]);
          }
        }
      }
    }
    if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
    // the CTA's memory stays until its copies have ended
    if (bytes && lane == 0)
      for (uint32_t i = tk > (uint32_t)p.stages ? tk - p.stages : 0; i < tk; ++i)
        mbar_wait(&sh.full[i % p.stages], (i / p.stages) & 1);
    return;
  }

  // the lane's channels and weights
  const bool turns = 8 * l < p.rot, split = turns && !kInterleaved;
  const int ca = split ? 4 * l : 8 * l, cb = split ? half + 4 * l : 8 * l + 4;
  const float inv_d = 1.0f / D;
  uint2 wq[2] = {}, wk[2] = {};
  if (p.q_weight) {
    wq[0] = load4(p.q_weight + ca);
    wq[1] = load4(p.q_weight + cb);
  }
  if (p.k_weight) {
    wk[0] = load4(p.k_weight + ca);
    wk[1] = load4(p.k_weight + cb);
  }
  // The warp's rows of a stage, kRows at a time: the groups of key heads go to the first
  // warps, those of query heads on from there in turn, those of value heads from the last.
  const int k_groups = ceil_div(nk, kRows);
  const int kh = warp * kRows + sub, vh = (kWarps - 1 - warp) * kRows + sub;
  const bool k_mine = warp < k_groups, k_row = kh < nk;
  const int q_first = (warp - k_groups + kWarps) % kWarps;
  uint32_t tk = 0, blk = 0;
  bool ok = true;
  for (uint32_t n = 0; ok; ++n) {
    const int slot = n % kItems;
    ok = __all_sync(kFull, mbar_wait(&sh.item_full[slot], (n / kItems) & 1));
    if (!ok) break;
    const Item it = sh.item[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_empty[slot]);
    if (it.b < 0) break;
    const bool mapped = it.phys >= 0;
    const size_t k_block = mapped ? ((size_t)it.phys * p.Hkv + k0) * P : 0;
    const uint2 start = make_uint2(kNanPair, kNanPair);  // any key replaces it
    uint2 mn[2] = {start, start}, mx[2] = {start, start};
    for (int t = 0; t < it.cnt; ++t, ++tk) {
      const float2* turn = sh.turn[(blk - 1) & 1];
      if (t % kTurnTokens == 0) {
        // the angles of the next tokens, into the table that no warp reads any more: all
        // have passed the barrier of the one between
        float2* to = sh.turn[blk & 1];
        turn = to;
        const int cnt = min(kTurnTokens, it.cnt - t);
        for (int i = tid; i < cnt * half; i += kWarps * 32) {
          const int tt = t + i / half, f = i % half;
          const int pos = p.positions ? p.positions[it.row0 + tt] : it.lo + tt;
          const unsigned long long phase = sh.turns_of[f] * (unsigned long long)(long long)pos;
          float sn, c;
          // 2 * 2^-32 half turns
          sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, &sn, &c);
          to[i / half * (D / 2) + f] = make_float2(c, sn);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.turn_full[blk & 1]);
        ok = __all_sync(kFull, mbar_wait(&sh.turn_full[blk & 1], (blk >> 1) & 1));
        if (!ok) break;
        ++blk;
      }
      const int st = tk % p.stages;
      if (nq + nk > 0) ok = __all_sync(kFull, mbar_wait(&sh.full[st], (tk / p.stages) & 1));
      if (!ok) break;
      const uint16_t* q = reinterpret_cast<const uint16_t*>(smem + st * stage_bytes);
      const uint16_t* k = q + p.nq * D;
      float4 cs[2];
      if (turns) {
        const float4* src =
            reinterpret_cast<const float4*>(turn + t % kTurnTokens * (D / 2) + 4 * l);
        cs[0] = src[0], cs[1] = src[1];
      }
      auto make = [&](const uint16_t* src, const uint2 (&w)[2], bool normed, Row& x) {
        x.set(*reinterpret_cast<const uint2*>(src + ca), *reinterpret_cast<const uint2*>(src + cb));
        if (normed) x.norm<kLanes>(w, inv_d, p.eps);
        if (turns) x.turn<kInterleaved>(cs);
      };
      const size_t slot = (size_t)((it.lo + t) % P) * D;
      if (mapped && k_mine) {
        Row x;
        make(k + min(kh, nk - 1) * D, wk, p.k_weight != nullptr, x);
        if (k_row) {
          uint16_t* dst = p.k + (k_block + (size_t)kh * P) * D + slot;
          const uint2 a = x.first(), b = x.second();
          *reinterpret_cast<uint2*>(dst + ca) = a;
          *reinterpret_cast<uint2*>(dst + cb) = b;
          mn[0] = vmin(mn[0], a), mn[1] = vmin(mn[1], b);
          mx[0] = vmax(mx[0], a), mx[1] = vmax(mx[1], b);
        }
      }
      for (int r0 = q_first * kRows; r0 < nq; r0 += kWarps * kRows) {
        const int r = r0 + sub;
        Row x;
        make(q + min(r, nq - 1) * D, wq, p.q_weight != nullptr, x);
        if (r >= nq) continue;
        const size_t o = ((size_t)(it.row0 + t) * p.Hq + q0 + r) * D;
        if (p.q_out) {
          *reinterpret_cast<uint2*>(p.q_out + o + ca) = x.first();
          *reinterpret_cast<uint2*>(p.q_out + o + cb) = x.second();
        }
        if (p.q_out_f32) {
          *reinterpret_cast<float4*>(p.q_out_f32 + o + ca) =
              make_float4(x.f[0].x, x.f[0].y, x.f[1].x, x.f[1].y);
          *reinterpret_cast<float4*>(p.q_out_f32 + o + cb) =
              make_float4(x.f[2].x, x.f[2].y, x.f[3].x, x.f[3].y);
        }
      }
      if (mapped && vh < nk)
        *reinterpret_cast<uint4*>(p.v + (k_block + (size_t)vh * P) * D + slot + 8 * l) =
            *reinterpret_cast<const uint4*>(k + (p.nk + vh) * D + 8 * l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
    }
    if (!ok) break;
    if (!mapped || !k_row) continue;
    uint16_t* s = p.summ + (((size_t)it.b * p.Hkv + k0 + kh) * p.max_pages + it.page) * 2 * D;
    const bool fresh = it.lo == it.page * P;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint2* smin = reinterpret_cast<uint2*>(s + (i ? cb : ca));
      uint2* smax = reinterpret_cast<uint2*>(s + D + (i ? cb : ca));
      *smin = fresh ? mn[i] : vmin(*smin, mn[i]);
      *smax = fresh ? mx[i] : vmax(*smax, mx[i]);
    }
  }
  if (!ok && lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
}

template <int D, int P>
cudaError_t launch_t(const NormRotateArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  const int items = a.q_offsets ? a.num_tokens / P + 2 * kv.batch : kv.batch;
  // Few items: split their heads over several CTAs (each computes the angles
  // again) until there are about four CTAs an SM, but not below a step of query
  // rows for every warp. Many: kCtas an SM take them in turn, so that the next
  // item is looked up and its rows are loaded while the last is worked on.
  const int split = max(1, min(4 * a.num_sms / items, kv.num_q_heads * D / (8 * 256)));
  const int ctas = min(items, split == 1 ? kCtas * a.num_sms : items);
  const int nq = ceil_div(kv.num_q_heads, split), nk = ceil_div(kv.num_kv_heads, split);
  const int stage_bytes = (nq + 2 * nk) * D * 2;
  // up to sixteen tokens in a third of an SM's shared memory
  constexpr int kBudget = 72 * 1024;
  const int stages = max(2, min(kMaxStages, kBudget / stage_bytes));
  Params p{a.qkv, a.q_offsets, a.positions, a.q_weight, a.k_weight, a.inv_freq, a.q_out,
           a.q_out_f32, kv.k_cache, kv.v_cache, kv.summaries, kv.block_table, kv.seq_lens, a.err,
           kv.batch, kv.num_q_heads, kv.num_kv_heads, kv.max_pages, kv.num_phys_pages,
           a.num_tokens, a.rotary_dim, nq, nk, stages, items, a.eps};
  auto kernel = a.interleaved ? norm_rotate_kernel<D, P, true> : norm_rotate_kernel<D, P, false>;
  const int smem = stages * stage_bytes + (int)sizeof(Shared<D>);
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, kBudget + (int)sizeof(Shared<D>));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas, split), dim3(kThreads), smem, stream, p);
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
