// chunk_plan.cuh - how the work on a packed batch of new tokens is cut into
// items and units and shared out over the CTAs, on the device: the host knows
// neither lengths nor offsets, so a call can be captured and replayed as they
// change.
//
// A cut says how many items a head of a request has and how many units an item:
//   RowCut   item: up to 256 query rows, a row being one (token, head of the
//            group), token-major; unit: those rows against 128 keys that they see.
//   KeyCut   item: 256 keys; unit: those keys against 128 query rows.
// The items in order (request, head, item) form one sequence of units, of which
// every CTA takes an equal, contiguous share.
#pragma once

#include "asp_internal.cuh"

namespace asp {

constexpr int kTileKeys = 128;
constexpr int kTileRows = 128, kLogTileRows = 7;
constexpr int kLogChunkRows = 8;
static_assert(1 << kLogTileRows == kTileRows && 1 << kLogChunkRows == kChunkRows);
constexpr int kItemKeys = 2 * kTileKeys;

struct ChunkDims {
  const int32_t* q_offsets;
  const int32_t* seq_lens;
  int B, Hkv, g, lg, max_pages, P, num_tokens;  // lg: log2(g)
  unsigned long long inv_ctas;  // chunk_inverse of the grid
};

// One request: its tokens, and its rows. One that is skipped has no tokens either, so that no
// cut has items of it.
struct ChunkRequest {
  int T, n, row0;
};
__device__ __forceinline__ ChunkRequest chunk_request(const ChunkDims& c, int b, uint32_t* err) {
  const int T = clamp_seq_len(c.seq_lens[b], c.max_pages, c.P, err);
  const NewRows r = new_rows(c.q_offsets, b, T, c.num_tokens, err);
  return ChunkRequest{r.bad ? 0 : T, r.n, r.row0};
}

// lg: log2 of the group. The plan divides by shifts: it stands before all other work of a
// call, and a division by a value that is not known when the code is compiled is some forty
// dependent instructions.
struct RowCut {
  // Units of rows whose last token is `last` (counted in the chunk).
  static __device__ __forceinline__ int units_to(const ChunkRequest& r, int last) {
    return (r.T - r.n + last) / kTileKeys + 1;
  }
  static __device__ __forceinline__ int items(const ChunkRequest& r, int lg) {
    return (r.n + (kChunkRows >> lg) - 1) >> (kLogChunkRows - lg);
  }
  static __device__ __forceinline__ int units(const ChunkRequest& r, int lg, int item) {
    return units_to(r, min(r.n, (item + 1) * (kChunkRows >> lg)) - 1);
  }
  // Units of a head's first m items.
  static __device__ __forceinline__ long long before(const ChunkRequest& r, int lg, int m) {
    const int tpi = kChunkRows >> lg, all = items(r, lg);
    const int whole = m < all ? m : all - 1;  // items that end on their last possible token
    long long sum = 0;
    if (whole > 0) {
      // item i of them has floor((a + tpi (i + 1) - 1) / 128) + 1 units; the floors
      // repeat, plus `step`, every `period` items
      const int a = r.T - r.n, lp = max(0, lg - 1), period = 1 << lp;
      const int step = max(1, tpi / kTileKeys);
      for (int s = 0; s < period; ++s) {
        const long long cnt = (whole - s + period - 1) >> lp;
        if (cnt <= 0) break;
        sum += cnt * ((a + tpi * (s + 1) - 1) / kTileKeys + 1) + step * (cnt * (cnt - 1) >> 1);
      }
    }
    if (m == all && all > 0) sum += units_to(r, r.n - 1);
    return sum;
  }
};

struct KeyCut {
  static __device__ __forceinline__ int items(const ChunkRequest& r, int) {
    return ceil_div(r.T, kItemKeys);
  }
  // First tile of rows that sees a key of the item.
  static __device__ __forceinline__ int first_tile(const ChunkRequest& r, int lg, int item) {
    return max(0, item * kItemKeys - (r.T - r.n)) >> (kLogTileRows - lg);
  }
  static __device__ __forceinline__ int tiles(const ChunkRequest& r, int lg) {
    return (r.n + (kTileRows >> lg) - 1) >> (kLogTileRows - lg);
  }
  // A request without new rows still has its weights carried over: one empty unit.
  static __device__ __forceinline__ int units(const ChunkRequest& r, int lg, int item) {
    return r.n == 0 ? 1 : tiles(r, lg) - first_tile(r, lg, item);
  }
  static __device__ __forceinline__ long long before(const ChunkRequest& r, int lg, int m) {
    if (r.n == 0) return m;
    const int a = r.T - r.n, nq = tiles(r, lg), seen = a / kItemKeys + 1;
    const int full = min(m, seen);   // items that every tile of rows sees
    long long sum = (long long)full * nq;
    const long long cut = m - full;  // the others: 2 g tiles fewer each time
    if (cut > 0)
      sum += cut * (nq - ((kItemKeys * seen - a) >> (kLogTileRows - lg))) -
             ((long long)(kItemKeys / kTileRows) << lg) * (cut * (cut - 1) >> 1);
    return sum;
  }
};

// Even shares of `total` units over G CTAs: the first r = total % G take q + 1, the
// others q = total / G. The division is a product with 2^64 / G rounded up, which is
// exact for totals under 2^63 / G (a 64-bit division is a called routine, whose code
// alone takes microseconds to fetch at a kernel's start).
struct ChunkShares {
  long long q;
  int r;
  __device__ __forceinline__ ChunkShares() {}
  __device__ __forceinline__ ChunkShares(long long total, int G, unsigned long long inv) {
    q = (long long)__umul64hi((unsigned long long)total, inv);
    r = (int)(total - q * G);
  }
  __device__ __forceinline__ long long begin(int c) const { return c * q + min(c, r); }
  // The CTA that takes `unit`, which CTA c or a later one does.
  __device__ __forceinline__ int taker(long long unit, int c) const {
    while (begin(c + 1) <= unit) ++c;
    return c;
  }
};
inline int chunk_log2(int g) { return g == 8 ? 3 : g == 4 ? 2 : g == 2 ? 1 : 0; }
// 2^64 / G rounded up (G > 1: the devices of this library have 152 SMs).
inline unsigned long long chunk_inverse(int G) { return ~0ull / (unsigned)G + 1; }

// Where a CTA's share begins: unit `u` of item (b, h, item); and the share.
struct ChunkStart {
  int b, h, item, u;
  ChunkRequest r;
  long long first, count;
  ChunkShares shares;
};

// Fills *start (shared memory) for this CTA; every thread of the block calls it.
// scratch: one long long for each warp. Two passes over a thread's requests through one loop:
// the first adds their units up, the second, once the shares are known, finds the one where
// this CTA's begins. (The plan is code that runs once, before everything else, so what it
// costs is mostly its fetching: there is one copy of Cut::before in it.)
template <typename Cut>
__device__ __forceinline__ void chunk_plan(const ChunkDims& c, ChunkStart* start, long long* scratch,
                                           uint32_t* err) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = ceil_div(c.B, nt), b0 = min(c.B, tid * per), b1 = min(c.B, b0 + per);
  if (tid == 0) start->count = 0;
  if (blockIdx.x != 0) err = nullptr;
  ChunkShares shares;
  long long mine = 0, at = 0, first = 0, count = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    bool found = false;
#pragma unroll 1
    for (int b = b0; b < b1 && !found; ++b) {
      const ChunkRequest r = chunk_request(c, b, err);
      int lo = 0, hi = Cut::items(r, c.lg), x = hi, h = -1;  // h < 0: x is all of a head's items
      long long in_h = 0, lo_units = 0;
#pragma unroll 1
      while (true) {
        const long long v = Cut::before(r, c.lg, x);
        if (h < 0) {
          const long long all = c.Hkv * v;
          if (pass == 0) {
            mine += all;
            break;
          }
          if (first >= at + all) {
            at += all;
            break;
          }
          in_h = first - at;
          for (h = 0; in_h >= v; in_h -= v) ++h;  // fewer than Hkv <= 8 steps
          --hi;
        } else if (v <= in_h) {
          lo = x;
          lo_units = v;
        } else {
          hi = x - 1;
        }
        if (lo >= hi) {
          *start = ChunkStart{b, h, lo, (int)(in_h - lo_units), r, first, count, shares};
          found = true;
          break;
        }
        x = (lo + hi + 1) >> 1;
      }
    }
    if (pass == 1) break;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < nt / 32; ++w) {
      if (w < warp) at += scratch[w];
      total += scratch[w];
    }
    at += sum - mine;
    shares = ChunkShares(total, gridDim.x, c.inv_ctas);
    first = shares.begin(blockIdx.x);
    count = shares.begin(blockIdx.x + 1) - first;
    err = nullptr;
    if (count <= 0 || first < at || first >= at + mine) break;
  }
  __syncthreads();
}

// Walks a CTA's pieces: piece = units [u0, u1) of one item.
template <typename Cut>
struct ChunkWalk {
  const ChunkDims& c;
  ChunkRequest r;
  long long left, at;   // units still to take, global index of the piece's first unit
  int b, h, item, items;
  int u0, u1, units;    // the piece, and the whole item's units

  __device__ __forceinline__ ChunkWalk(const ChunkDims& dims, const ChunkStart& s)
      : c(dims), left(s.count), at(s.first), b(s.b), h(s.h), item(s.item) {
    if (left <= 0) return;
    r = s.r;
    items = Cut::items(r, c.lg);
    u0 = s.u;
    set();
  }
  __device__ __forceinline__ void set() {
    units = Cut::units(r, c.lg, item);
    u1 = (int)min((long long)units, u0 + left);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
  __device__ __forceinline__ void next() {
    left -= u1 - u0;
    at += u1 - u0;
    if (left <= 0) return;
    u0 = 0;
    if (++item >= items) {
      item = 0;
      if (++h >= c.Hkv) {
        h = 0;
        do {  // the total counts units that are still to come: some later request has items
          if (++b >= c.B) {
            left = 0;
            return;
          }
          r = chunk_request(c, b, nullptr);
          items = Cut::items(r, c.lg);
        } while (items == 0);
      }
    }
    set();
  }
};

// ------------------------------------------------------------ handing out pieces
// One thread of the CTA walks the share and hands its pieces to the other warps
// through a ring in shared memory, ahead of them: the walk is long straight code that
// runs once a piece, and in every role's way it costs more than its arithmetic (its
// instructions come from L2, some hundred cycles a line: 8 us between two items where
// every warp walked for itself).
struct alignas(16) ChunkTask {
  int b, h, item;       // b < 0: no more pieces
  int u0;               // first unit
  int T, n, row0;       // the request (ChunkRequest)
  int whole;            // the piece is the whole item
  int x[4];             // what the kernel's roles want to know of it
};
constexpr int kTaskRing = 4;
struct ChunkTasks {
  ChunkTask task[kTaskRing];
  uint64_t full[kTaskRing], empty[kTaskRing];
};

__device__ __forceinline__ void chunk_tasks_init(ChunkTasks& r, int readers) {
  for (int i = 0; i < kTaskRing; ++i) {
    mbar_init(&r.full[i], 1);
    mbar_init(&r.empty[i], readers);
  }
}

// The handing thread: fill(walk, task) sets task.x. Returns false where a wait ran out; *join
// then says that there is nothing to join, whatever an earlier call left there.
template <typename Cut, typename Fill>
__device__ __forceinline__ bool chunk_hand_out(ChunkTasks& r, const ChunkDims& c,
                                               const ChunkStart& start, ChunkJoin* join,
                                               Fill fill) {
  ChunkWalk<Cut> w(c, start);
  ChunkJoin jn{0, 0, 0, 0};
  *join = jn;
  for (uint32_t i = 0;; ++i) {
    const int slot = i % kTaskRing;
    if (!mbar_wait(&r.empty[slot], ((i / kTaskRing) & 1) ^ 1)) return false;
    ChunkTask& t = r.task[slot];
    if (!w.more()) {
      t.b = -1;
      mbar_arrive(&r.full[slot]);
      break;
    }
    t.b = w.b, t.h = w.h, t.item = w.item, t.u0 = w.u0;
    t.T = w.r.T, t.n = w.r.n, t.row0 = w.r.row0;
    t.whole = w.whole();
    fill(w, t);
    mbar_arrive(&r.full[slot]);
    if (w.u0 == 0 && !w.whole())  // the last piece: other CTAs end this item
      jn = ChunkJoin{w.b, w.h, w.item,
                     start.shares.taker(w.at + w.units - 1, blockIdx.x) - (int)blockIdx.x + 1};
    w.next();
  }
  *join = jn;
  return true;
}

// A warp that takes pieces, all its lanes together.
struct ChunkReader {
  ChunkTasks& r;
  uint32_t i = 0;
  bool ok = true;  // false: a wait ran out
  __device__ __forceinline__ explicit ChunkReader(ChunkTasks& ring) : r(ring) {}
  __device__ __forceinline__ bool next(ChunkTask& t) {
    const int slot = i % kTaskRing;
    ok = __all_sync(0xffffffffu, mbar_wait(&r.full[slot], (i / kTaskRing) & 1)) != 0;
    if (!ok) return false;
    ++i;
    const int4* src = reinterpret_cast<const int4*>(&r.task[slot]);
    int4* dst = reinterpret_cast<int4*>(&t);
    dst[0] = src[0], dst[1] = src[1], dst[2] = src[2];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[slot]);
    return t.b >= 0;
  }
};

// The joining kernels: the join that CTA blockIdx.x of the kernel before left, if there is one
// to follow, and its request. A wait that ran out in any CTA may have left partials of an
// earlier call: then nothing is joined.
template <typename Cut>
__device__ __forceinline__ bool chunk_join(const ChunkDims& c, const ChunkJoin* joins,
                                           const uint32_t* err, ChunkJoin& jn, ChunkRequest& r) {
  const uint32_t bits = *err;
  jn = joins[blockIdx.x];
  if (!chunk_join_valid(jn, c.B, c.Hkv, blockIdx.x, gridDim.x) || (bits & ASP_DEVERR_TIMEOUT))
    return false;
  r = chunk_request(c, jn.b, nullptr);
  return jn.item < Cut::items(r, c.lg);
}

}  // namespace asp
