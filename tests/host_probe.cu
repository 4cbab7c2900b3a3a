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
