// select_params.cuh - what the cluster selection kernel (select_cluster.cu) is launched with.
#pragma once

#include <cmath>

#include "asp_internal.cuh"

namespace asp {

struct CsParams {
  uint16_t* summ;  // written only by the append variant
  const float* q;
  const int32_t* seq_lens;
  int32_t* lists;
  int32_t* lens;
  uint32_t* err;
  int Hq, Hkv, P, max_pages;
  float inv_sqrt_d;
  float gamma;
  int budget;
  int pf_pieces;  // pieces per warp fetched into L2 before the predecessor ends
  // K/V of kept pages fetched into L2 for the decode that follows: the first
  // kv_pf_pages kept pages (in id order) of each CTA's range. 0 where the cache has no
  // bf16 pages (both pointers null): nothing may then be counted from them
  const int32_t* bt;
  uint16_t* k_cache;  // written only by the append variant
  uint16_t* v_cache;
  int num_phys;
  int kv_pf_pages;
  // append variant: the new token's K and V rows, bf16 [B, Hkv, d]
  const uint16_t* k_new;
  const uint16_t* v_new;
};

// Pieces per warp fetched into L2 before the previous kernel ends, and kept
// pages per CTA whose K/V the kernel fetches into L2 for the decode (8 KiB
// each at P = 16, d = 128). Outstanding bulk prefetches hold this kernel
// open, so more pages make it slower than they make the decode faster. At
// 128k, gamma = 0.99 on one GB300 (builds alternated on one box, steps/s):
// (pages, pieces) = (0, 3) 365.5, (32, 3) 372.6, (64, 3) 369.1, (128, 3)
// 364.9, (256, 3) 339.4; on a later build of the decode, (32, 3) 390.7,
// (24, 6) 393.6, (28, 6) 393.6, (24, 8) 393.6, and on another box (16, 3)
// 391.9, (48, 3) 391.9, (32, 4) 394.8, (24, 4) 395.3 against (32, 3) 393.7.
constexpr int kCsPrefetchPieces = 6;
constexpr int kCsKvPrefetchPages = 24;

inline CsParams cs_params(const SelectArgs& a) {
  const asp_paged_kv& kv = *a.kv;
  return CsParams{kv.summaries, a.q, kv.seq_lens, a.lists, a.lens, a.err, kv.num_q_heads,
                  kv.num_kv_heads, kv.page_size, kv.max_pages,
                  1.0f / std::sqrt((float)kv.head_dim), a.gamma, a.budget, kCsPrefetchPieces,
                  kv.block_table, kv.k_cache, kv.v_cache, kv.num_phys_pages,
                  kv.k_cache && kv.v_cache ? kCsKvPrefetchPages : 0, a.k_new, a.v_new};
}

}  // namespace asp
