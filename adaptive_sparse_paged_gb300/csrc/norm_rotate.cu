// norm_rotate.cu - new tokens into the paged cache: per-head norms of queries
// and keys, position rotation, the write of K and V into their pages and the
// fold of the keys into the page summaries, in one pass over the packed rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// One work item is one page of one request: the new tokens that fall into it.
// Its CTA computes each token's cosines and sines once, in shared memory, for all
// heads, while a loader thread streams the tokens' rows (contiguous in the packed
// array) through a ring of shared-memory stages, so that what is in flight does
// not cost registers: with the loads in registers the kernel took 110 us for 16k
// tokens of 48 heads, and 173 where smaller register budgets made them spill.
// Warps take rows; a row is d / 8 lanes wide, and a lane holds the two halves of
// four rotated pairs, so a pair never crosses lanes. A warp keeps the same key
// heads for all tokens, their channel minima and maxima in registers until the
// page is done: the summary is written once, without atomics.
//
// The angle: a frequency becomes a 64-bit fixed-point fraction of a turn, whose
// product with the integer position wraps exactly modulo one turn, so that
// position 2^31 is as exact as position 0 (in 32-bit floats an angle of 10^5
// radians is off by 0.004).
#include "tc.cuh"

namespace asp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = (kWarps + 1) * 32;  // and a loader
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
  int rot, nq, nk, stages;  // nq, nk: query and KV heads of a CTA
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

// The a and b of a lane's four pairs: its first four channels and its second four, or,
// interleaved, the even and the odd ones.
__device__ __forceinline__ void pairs(const uint2 (&v)[2], float* a, float* b, bool interleaved) {
  const float2 f[4] = {unpack(v[0].x), unpack(v[0].y), unpack(v[1].x), unpack(v[1].y)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (interleaved) {
      a[i] = f[i].x;
      b[i] = f[i].y;
    } else {
      float* to = i < 2 ? a : b;
      to[2 * (i & 1)] = f[i].x;
      to[2 * (i & 1) + 1] = f[i].y;
    }
  }
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  return make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
}
__device__ __forceinline__ uint2 load4(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint2*>(p));
}

// A lane's eight channels of a row are two times four. Halves rotated against each
// other: channels a + i and b + i are pair i; interleaved: eight in a row. Lanes
// past the rotated channels hold eight plain ones.
// Weight and rotation of a lane's four pairs as one linear map, the same for all rows of
// a token: (a, b) -> (a ac - b bs, b bc + a as), with the weights in the factors. Halves
// that do not turn have cosine 1 and sine 0. Two pairs to a register pair.
struct Map {
  float2 ac[2], bs[2], bc[2], as[2];
};

__device__ __forceinline__ Map make_map(const float4 (&cs)[2], const uint2 (&w)[2], bool weighted,
                                        bool turns, bool interleaved) {
  float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
  if (weighted) pairs(w, wa, wb, interleaved);
  const float co[4] = {cs[0].x, cs[0].z, cs[1].x, cs[1].z};
  const float si[4] = {cs[0].y, cs[0].w, cs[1].y, cs[1].w};
  Map m;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = make_float2(wa[2 * i], wa[2 * i + 1]), b = make_float2(wb[2 * i], wb[2 * i + 1]);
    const float2 c = turns ? make_float2(co[2 * i], co[2 * i + 1]) : make_float2(1.f, 1.f);
    const float2 n = turns ? make_float2(si[2 * i], si[2 * i + 1]) : make_float2(0.f, 0.f);
    m.ac[i] = mul2(a, c);
    m.bs[i] = mul2(b, make_float2(-n.x, -n.y));
    m.bc[i] = mul2(b, c);
    m.as[i] = mul2(a, n);
  }
  return m;
}

// A row: the lane's channels x (two times four) normed and mapped; kLanes lanes of a row.
template <int kLanes, bool kInterleaved>
__device__ __forceinline__ void norm_rotate(const uint2 (&x)[2], const Map& m, bool norm,
                                            float inv_d, float eps, float (&y)[8]) {
  float fa[4], fb[4];
  pairs(x, fa, fb, kInterleaved);
  float2 a[2], b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = make_float2(fa[2 * i], fa[2 * i + 1]);
    b[i] = make_float2(fb[2 * i], fb[2 * i + 1]);
  }
  if (norm) {
    float2 sq = mul2(a[0], a[0]);
    sq = fma2(a[1], a[1], sq);
    sq = fma2(b[0], b[0], sq);
    sq = fma2(b[1], b[1], sq);
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float r = rsqrtf(fmaf(ss, inv_d, eps));
    const float2 rr = make_float2(r, r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = mul2(a[i], rr);
      b[i] = mul2(b[i], rr);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 ya = fma2(b[i], m.bs[i], mul2(a[i], m.ac[i]));
    const float2 yb = fma2(a[i], m.as[i], mul2(b[i], m.bc[i]));
    y[kInterleaved ? 4 * i : 2 * i] = ya.x;
    y[kInterleaved ? 4 * i + 1 : 4 + 2 * i] = yb.x;
    y[kInterleaved ? 4 * i + 2 : 2 * i + 1] = ya.y;
    y[kInterleaved ? 4 * i + 3 : 5 + 2 * i] = yb.y;
  }
}

// Shared memory of a CTA: the ring, then these.
template <int D, int P>
struct Shared {
  float2 turn[P * (D / 2)];             // (cos, sin) of [token of the page][pair]
  unsigned long long turns_of[D / 2];   // 2^64 * inv_freq / (2 pi), modulo 2^64
  uint64_t full[kMaxStages], empty[kMaxStages];
};

template <int D, int P, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rotate_kernel(const Params p) {
  constexpr int kLanes = D / 8;        // lanes of one row
  constexpr int kRows = 32 / kLanes;   // rows a warp takes at once
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / kLanes, l = lane % kLanes;
  // this CTA's heads: a share of the query heads and of the KV heads
  const int q0 = blockIdx.y * p.nq, nq = max(0, min(p.nq, p.Hq - q0));
  const int k0 = blockIdx.y * p.nk, nk = max(0, min(p.nk, p.Hkv - k0));
  const int stage_bytes = (p.nq + 2 * p.nk) * D * 2;
  Shared<D, P>& sh = *reinterpret_cast<Shared<D, P>*>(smem + p.stages * stage_bytes);
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait_predecessor();

  if (p.q_offsets && blockIdx.x == 0 && blockIdx.y == 0) {  // every request's rows are checked
    for (int x = tid; x < p.B; x += kThreads)
      new_rows(p.q_offsets, x, clamp_seq_len(p.seq_lens[x], p.max_pages, P, p.err), p.num_tokens,
               p.err);
  }
  const int half = p.rot / 2;
  if (tid < half) {
    double t = (double)p.inv_freq[tid] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    sh.turns_of[tid] = (unsigned long long)(t * 18446744073709551616.0);
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
  const int Hall = p.Hq + 2 * p.Hkv;
  __syncthreads();  // barriers and turns_of are set

  if (warp == kWarps) {
    // ------------------------------------------------------------ loader
    if (lane != 0) return;
    const uint32_t bytes = (uint32_t)(nq + 2 * nk) * D * 2;
    if (bytes == 0) return;
    int t = 0;
    bool ok = true;
    for (; t < cnt; ++t) {
      const int st = t % p.stages;
      ok = mbar_wait(&sh.empty[st], ((t / p.stages) & 1) ^ 1);
      if (!ok) break;
      const uint16_t* row = p.qkv + (size_t)(row0 + t) * Hall * D;
      uint8_t* dst = smem + st * stage_bytes;
      mbar_arrive_expect_tx(&sh.full[st], bytes);
      if (nq > 0) bulk_g2s(dst, row + q0 * D, nq * D * 2, &sh.full[st]);
      if (nk > 0) {
        dst += p.nq * D * 2;
        bulk_g2s(dst, row + (p.Hq + k0) * D, nk * D * 2, &sh.full[st]);
        bulk_g2s(dst + p.nk * D * 2, row + (p.Hq + p.Hkv + k0) * D, nk * D * 2, &sh.full[st]);
      }
    }
    // the CTA's memory stays until its copies have ended
    if (!ok) report(p.err, ASP_DEVERR_TIMEOUT);
    for (int i = max(0, t - p.stages); i < t; ++i)
      mbar_wait(&sh.full[i % p.stages], (i / p.stages) & 1);
    return;
  }

  for (int i = tid; i < cnt * half; i += kWarps * 32) {
    const int t = i / half, f = i % half;
    const int pos = p.positions ? p.positions[row0 + t] : lo + t;
    const unsigned long long phase = sh.turns_of[f] * (unsigned long long)(long long)pos;
    float s, c;
    sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // 2 * 2^-32 half turns
    sh.turn[t * (D / 2) + f] = make_float2(c, s);
  }
  const int phys = p.bt[(size_t)b * p.max_pages + page];
  const bool mapped = phys >= 0 && phys < p.num_phys;
  if (!mapped && tid == 0) report(p.err, ASP_DEVERR_PAGE_RANGE);
  named_bar_sync(1, kWarps * 32);

  // the lane's channels, and its weights
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
  // rows of this warp: query rows (warp + 8 i) * kRows + sub, one group of key heads,
  // and, from the other end, groups of value heads
  const int kh = warp * kRows + sub;
  const bool k_mine = warp * kRows < nk, k_row = kh < nk;
  const size_t k_block = mapped ? ((size_t)phys * p.Hkv + k0) * P : 0;
  // folding starts from values that any key replaces
  uint2 mn[2] = {make_uint2(0x7f807f80u, 0x7f807f80u), make_uint2(0x7f807f80u, 0x7f807f80u)};
  uint2 mx[2] = {make_uint2(0xff80ff80u, 0xff80ff80u), make_uint2(0xff80ff80u, 0xff80ff80u)};
  bool ok = true;
  for (int t = 0; t < cnt; ++t) {
    const int st = t % p.stages;
    if (nq + nk > 0) ok = __all_sync(kFull, mbar_wait(&sh.full[st], (t / p.stages) & 1));
    if (!ok) break;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(smem + st * stage_bytes);
    const uint16_t* k = q + p.nq * D;
    const uint16_t* v = k + p.nk * D;
    float4 cs[2];
    if (turns) {
      const float4* src = reinterpret_cast<const float4*>(sh.turn + t * (D / 2) + 4 * l);
      cs[0] = src[0], cs[1] = src[1];
    }
    const Map mq = make_map(cs, wq, p.q_weight != nullptr, turns, kInterleaved);
    auto row_at = [&](const uint16_t* base, int r, uint2 (&x)[2]) {
      x[0] = *reinterpret_cast<const uint2*>(base + r * D + ca);
      x[1] = *reinterpret_cast<const uint2*>(base + r * D + cb);
    };
#pragma unroll 2
    for (int g = warp; g * kRows < nq; g += kWarps) {
      const int r = g * kRows + sub;
      uint2 in[2];
      float x[8];
      row_at(q, min(r, nq - 1), in);
      norm_rotate<kLanes, kInterleaved>(in, mq, p.q_weight != nullptr, inv_d, p.eps, x);
      if (r >= nq) continue;
      const size_t o = ((size_t)(row0 + t) * p.Hq + q0 + r) * D;
      if (p.q_out) {
        *reinterpret_cast<uint2*>(p.q_out + o + ca) = pack4(x);
        *reinterpret_cast<uint2*>(p.q_out + o + cb) = pack4(x + 4);
      }
      if (p.q_out_f32) {
        *reinterpret_cast<float4*>(p.q_out_f32 + o + ca) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p.q_out_f32 + o + cb) = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
    if (mapped && k_mine) {
      uint2 in[2];
      float x[8];
      row_at(k, min(kh, nk - 1), in);
      const Map mk = make_map(cs, wk, p.k_weight != nullptr, turns, kInterleaved);
      norm_rotate<kLanes, kInterleaved>(in, mk, p.k_weight != nullptr, inv_d, p.eps, x);
      if (k_row) {
        uint16_t* dst = p.k + (k_block + (size_t)kh * P + (lo + t) % P) * D;
        const uint2 ya = pack4(x), yb = pack4(x + 4);
        *reinterpret_cast<uint2*>(dst + ca) = ya;
        *reinterpret_cast<uint2*>(dst + cb) = yb;
        mn[0] = vmin(mn[0], ya), mn[1] = vmin(mn[1], yb);
        mx[0] = vmax(mx[0], ya), mx[1] = vmax(mx[1], yb);
      }
    }
    if (mapped) {
      const int vh = (kWarps - 1 - warp) * kRows + sub;  // nk <= 8: one group at most
      if (vh < nk)
        *reinterpret_cast<uint4*>(p.v + (k_block + (size_t)vh * P + (lo + t) % P) * D + 8 * l) =
            *reinterpret_cast<const uint4*>(v + vh * D + 8 * l);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[st]);
  }
  if (!ok) {
    if (lane == 0) report(p.err, ASP_DEVERR_TIMEOUT);
    return;
  }
  if (!mapped || !k_row) return;
  uint16_t* s = p.summ + (((size_t)b * p.Hkv + k0 + kh) * p.max_pages + page) * 2 * D;
  const bool fresh = lo == page * P;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint2* smin = reinterpret_cast<uint2*>(s + (i ? cb : ca));
    uint2* smax = reinterpret_cast<uint2*>(s + D + (i ? cb : ca));
    *smin = fresh ? mn[i] : vmin(*smin, mn[i]);
    *smax = fresh ? mx[i] : vmax(*smax, mx[i]);
  }
}

template <int D, int P>
cudaError_t launch_t(const NormRotateArgs& a, cudaStream_t stream) {
  const asp_paged_kv& kv = *a.kv;
  const int items = a.q_offsets ? a.num_tokens / P + 2 * kv.batch : kv.batch;
  // Few items: split their heads over several CTAs (each computes the angles
  // again) until there are about four CTAs an SM, but not below a step of query rows for every warp.
  const int split = max(1, min(4 * a.num_sms / items, kv.num_q_heads * D / (kWarps * 256)));
  const int nq = ceil_div(kv.num_q_heads, split), nk = ceil_div(kv.num_kv_heads, split);
  const int stage_bytes = (nq + 2 * nk) * D * 2;
  // as many stages as an item has tokens, in a third of an SM's shared memory at most
  constexpr int kBudget = 72 * 1024;
  const int stages = max(2, min(min(kMaxStages, P), kBudget / stage_bytes));
  Params p{a.qkv, a.q_offsets, a.positions, a.q_weight, a.k_weight, a.inv_freq, a.q_out,
           a.q_out_f32, kv.k_cache, kv.v_cache, kv.summaries, kv.block_table, kv.seq_lens, a.err,
           kv.batch, kv.num_q_heads, kv.num_kv_heads, kv.max_pages, kv.num_phys_pages,
           a.num_tokens, a.rotary_dim, nq, nk, stages, a.eps};
  auto kernel = a.interleaved ? norm_rotate_kernel<D, P, true> : norm_rotate_kernel<D, P, false>;
  const int smem = stages * stage_bytes + (int)sizeof(Shared<D, P>);
  cudaError_t e = set_max_dynamic_smem((const void*)kernel, kBudget + (int)sizeof(Shared<D, P>));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(items, split), dim3(kThreads), smem, stream, p);
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
