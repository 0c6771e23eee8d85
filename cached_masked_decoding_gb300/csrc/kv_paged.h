// The paged K/V cache, as its operators share it.
#pragma once

#include "ops8.h"

namespace dllm {

// Checks a paged cache; who names the operator.
dllm_status kv_paged_check(const dllm_kv_paged* c, const char* who);

// What the kernels read of it.
struct PagedKv {
  uint16_t *k, *v;
  const int32_t* table;
  int b, H_kv, hd, pages, page_shift, max_pages;
  long long positions;                 // max_pages << page_shift
  explicit PagedKv(const dllm_kv_paged& c)
      : k(static_cast<uint16_t*>(c.k)), v(static_cast<uint16_t*>(c.v)), table(c.table), b(c.b), H_kv(c.H_kv), hd(c.hd),
        pages(c.pages), page_shift(0), max_pages(c.max_pages), positions((long long)c.max_pages * c.page_size) {
    while ((1 << page_shift) < c.page_size) ++page_shift;
  }
  PagedKv() = default;
#ifdef __CUDACC__
  // The first element of head g's row at position t of sequence s, or -1 where t lies on no page
  // (0 <= t < positions).
  __device__ __forceinline__ long long row(int s, int g, int t) const {
    const int page = table[(long long)s * max_pages + (t >> page_shift)];
    if ((unsigned)page >= (unsigned)pages) return -1;
    return ((((long long)page * H_kv + g) << page_shift) + (t & ((1 << page_shift) - 1))) * hd;
  }
  // Keys of sequence s: its length within what the table holds.
  __device__ __forceinline__ int len(const int32_t* lens, int s) const {
    return lens ? (int)min((long long)max(lens[s], 0), positions) : (int)positions;
  }
#endif
};

}  // namespace dllm
