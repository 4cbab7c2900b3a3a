// chunk_plan.cuh - how a packed batch of new tokens is cut into tiles and
// shared out over the CTAs, on the device: the host knows neither lengths nor
// offsets, so a call can be captured and replayed as they change.
//
// An item is (request, KV head, up to 256 query rows); a row is one
// (token, head of the group), token-major, so an item holds 256 / g tokens. A
// unit is one item against one tile of 128 keys; causality gives the item
// (t_last / 128 + 1) units. The items in order (request, head, tile) form one
// sequence of units, of which every CTA takes an equal, contiguous share.
#pragma once

#include "asp_internal.cuh"

namespace asp {

constexpr int kTileKeys = 128;
constexpr int kItemRows = kChunkRows;

struct ChunkDims {
  const int32_t* q_offsets;
  const int32_t* seq_lens;
  int B, Hkv, g, max_pages, P, num_tokens;
};

// One request: its rows and its tokens.
struct ChunkRequest {
  int T, n, row0;
};
__device__ __forceinline__ ChunkRequest chunk_request(const ChunkDims& c, int b, uint32_t* err) {
  const int T = clamp_seq_len(c.seq_lens[b], c.max_pages, c.P, err);
  const NewRows r = new_rows(c.q_offsets, b, T, c.num_tokens, err);
  return ChunkRequest{T, r.n, r.row0};
}
__device__ __forceinline__ int chunk_items(const ChunkRequest& r, int tokens_per_item) {
  return ceil_div(r.n, tokens_per_item);
}
// Units of the item whose last token is `last` (counted in the chunk).
__device__ __forceinline__ int chunk_units(const ChunkRequest& r, int last) {
  return (r.T - r.n + last) / kTileKeys + 1;
}
// Units of a head's first m items.
__device__ __forceinline__ long long chunk_units_before(const ChunkRequest& r, int tpi, int m) {
  const int items = chunk_items(r, tpi);
  long long sum = 0;
  const int whole = m < items ? m : items - 1;  // items that end on their last possible token
  if (whole > 0) {
    // item i of them has floor((a + tpi (i + 1) - 1) / 128) + 1 units; the floors
    // repeat, plus one, every `period` items
    const int a = r.T - r.n, period = tpi < kTileKeys ? kTileKeys / tpi : 1;
    const int step = tpi < kTileKeys ? 1 : tpi / kTileKeys;
    for (int s = 0; s < period; ++s) {
      const long long cnt = (whole - s + period - 1) / period;
      if (cnt <= 0) break;
      sum += cnt * ((a + tpi * (s + 1) - 1) / kTileKeys + 1) + step * cnt * (cnt - 1) / 2;
    }
  }
  if (m == items && items > 0) sum += chunk_units(r, r.n - 1);
  return sum;
}

// Where a CTA's share begins: item (b, h, qt), its unit `u`; and how many units it takes.
struct ChunkStart {
  int b, h, qt, u;
  long long first, count, total;
};

// Even shares of `total` units over G CTAs: the first total % G take one more.
__device__ __forceinline__ long long chunk_share_begin(long long total, int G, int c) {
  const long long q = total / G, r = total % G;
  return c * q + (c < r ? c : r);
}
__device__ __forceinline__ int chunk_share_of(long long total, int G, long long unit) {
  const long long q = total / G, r = total % G, big = r * (q + 1);
  return (int)(unit < big ? unit / (q + 1) : r + (unit - big) / q);
}

// Fills *start (shared memory) for this CTA; every thread of the block calls it.
// scratch: one long long for each warp.
__device__ __forceinline__ void chunk_plan(const ChunkDims& c, ChunkStart* start, long long* scratch,
                                           uint32_t* err) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int tpi = kItemRows / c.g;
  const int per = ceil_div(c.B, nt), b0 = min(c.B, tid * per), b1 = min(c.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const ChunkRequest r = chunk_request(c, b, blockIdx.x == 0 ? err : nullptr);
    mine += (long long)c.Hkv * chunk_units_before(r, tpi, chunk_items(r, tpi));
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  if (tid == 0) start->count = 0;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  before += x - mine;
  const long long first = chunk_share_begin(total, gridDim.x, blockIdx.x);
  const long long count = chunk_share_begin(total, gridDim.x, blockIdx.x + 1) - first;
  if (count > 0 && first >= before && first < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const ChunkRequest r = chunk_request(c, b, nullptr);
      const int items = chunk_items(r, tpi);
      const long long head = chunk_units_before(r, tpi, items);
      if (first >= at + c.Hkv * head) {
        at += c.Hkv * head;
        continue;
      }
      const long long in_b = first - at;
      const int h = (int)(in_b / head);
      const long long in_h = in_b - h * head;
      int lo = 0, hi = items - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (chunk_units_before(r, tpi, mid) <= in_h) lo = mid; else hi = mid - 1;
      }
      *start = ChunkStart{b, h, lo, (int)(in_h - chunk_units_before(r, tpi, lo)), first, count, total};
      break;
    }
  }
  __syncthreads();
}

// Walks a CTA's pieces: piece = units [u0, u1) of one item.
struct ChunkWalk {
  ChunkDims c;
  ChunkRequest r;
  long long left, at;   // units still to take, global index of the piece's first unit
  int b, h, qt, tpi, items;
  int u0, u1, units;    // the piece, and the whole item's units
  int tok0, ntok;       // the item's first token of the chunk, and its tokens

  __device__ __forceinline__ ChunkWalk(const ChunkDims& dims, const ChunkStart& s)
      : c(dims), left(s.count), at(s.first), b(s.b), h(s.h), qt(s.qt), tpi(kItemRows / dims.g) {
    if (left <= 0) return;
    r = chunk_request(c, b, nullptr);
    items = chunk_items(r, tpi);
    u0 = s.u;
    set();
  }
  __device__ __forceinline__ void set() {
    tok0 = qt * tpi;
    ntok = min(tpi, r.n - tok0);
    units = chunk_units(r, tok0 + ntok - 1);
    u1 = (int)min((long long)units, u0 + left);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next() {
    left -= u1 - u0;
    at += u1 - u0;
    if (left <= 0) return;
    u0 = 0;
    if (++qt >= items) {
      qt = 0;
      if (++h >= c.Hkv) {
        h = 0;
        do {  // the total counts units that are still to come: some later request has rows
          if (++b >= c.B) {
            left = 0;
            return;
          }
          r = chunk_request(c, b, nullptr);
        } while (r.n == 0);
        items = chunk_items(r, tpi);
      }
    }
    set();
  }
  // Units of this piece that the rows of tokens [t0, t1) of the chunk need.
  __device__ __forceinline__ int units_for(int t0, int t1) const {
    if (t1 <= t0) return 0;
    return max(0, min(u1, chunk_units(r, t1 - 1)) - u0);
  }
};

}  // namespace asp
