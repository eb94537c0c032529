// What the kernels over an NVFP4 key/value cache share: where a token lies, and the
// decoding of a block.
#pragma once

#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

// Entry b's page that holds position t (t >= 0, below the entry's capacity), -1 if the
// table names none.
__device__ __forceinline__ int64_t cache_page(const Cache& c, int64_t b, int t) {
  if (!c.table) return b;
  const int p = c.table[b * c.table_pages + (t >> c.page_shift)];
  return p >= 0 && p < c.pages ? p : -1;
}
// Position t's place in its page.
__device__ __forceinline__ int cache_place(const Cache& c, int t) {
  return c.table ? t & ((1 << c.page_shift) - 1) : t;
}
// The row (of one head's tokens in a page) with which a page's head starts.
__device__ __forceinline__ int64_t cache_rows(const Cache& c, int64_t page, int head) {
  return (page * c.kv_heads + head) * c.page_size;
}

// n / d by a product: d's magic number for 0 <= n < 2^31.
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& d) {
  return (__umulhi(n, d.magic) + n) >> d.shift;
}

}  // namespace

}  // namespace nvfp4
