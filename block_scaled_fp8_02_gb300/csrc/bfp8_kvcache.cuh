// bfp8_kvcache.cuh -- the paged e4m3 cache as the kernels see it.
#pragma once

#include <cstdint>

#include "../../include/bfp8.h"

namespace bfp8 {

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t num_pages;
  int64_t st_page, st_head, st_tok;    // codes, bytes
  int64_t ss_page, ss_head;            // scales, floats
  int32_t page_size, page_shift;
  int32_t heads, dim;
};

// Checks a caller's cache description and fills the view (bfp8_kvcache.cu).
bfp8_status check_cache(const bfp8_kv_cache* c, CacheView* view);

}  // namespace bfp8
