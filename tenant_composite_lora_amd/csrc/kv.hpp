// The paged key/value cache as the kernels see it.
#pragma once

#include <cstdint>

#include "tcl_internal.hpp"

namespace tcl {

struct KvArgs {
  uint16_t *K, *V;
  int64_t s_page, s_slot, s_head;  // elements
  int32_t n_pages, page_shift;     // page_size = 1 << page_shift
  int32_t H, D;                    // heads, head dimension
};

// offset of head 0 of a slot that lies in the cache
__device__ inline int64_t kv_slot(const KvArgs &c, int64_t slot) {
  return (slot >> c.page_shift) * c.s_page +
         (slot & ((int64_t(1) << c.page_shift) - 1)) * c.s_slot;
}

// checks a cache and fills its kernel arguments (kv.hip)
int kv_check(const tcl_kv_cache *c, KvArgs *out);

}  // namespace tcl
