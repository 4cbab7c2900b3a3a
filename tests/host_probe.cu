// Host functions of the library's headers, for the tests that look at them without a GPU.
#include "select_params.cuh"

// What the cluster selection kernel is told to prefetch of this cache: pages, and whether the
// addresses it would count from are there.
extern "C" int select_prefetch(const asp_paged_kv* kv, int* k_there, int* v_there) {
  const asp::SelectArgs a{kv, nullptr, 0.9f, 0, nullptr, nullptr, nullptr, nullptr, 152};
  const asp::CsParams p = asp::cs_params(a);
  *k_there = p.k_cache != nullptr;
  *v_there = p.v_cache != nullptr;
  return p.kv_pf_pages;
}

// Where a workspace of this shape has its arrival counts (begin, end) and the chunk calls' joins
// and partials (begin, end), in bytes.
extern "C" void workspace_parts(const asp_paged_kv* kv, int sms, long long* at) {
  const asp::WsLayout w = asp::ws_layout(*kv, sms);
  at[0] = (long long)w.arrivals_off;
  at[1] = at[0] + 4ll * kv->batch * kv->num_kv_heads;
  at[2] = (long long)w.joins_off;
  at[3] = (long long)w.total;
}
