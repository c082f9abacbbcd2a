// kv_device.h -- the NVFP4 key/value cache as the kernels see it, and the
// position arithmetic they share (kv_cache.hip, kv_attention.hip).
//
// A cache keeps, for keys and for values, codes [pages, heads, page_size,
// dim/2] and scales [pages, heads, page_size, dim/16]: the row-major NVFP4
// layout with one row per (page, head, token in page), so the tokens of one
// head within a page are contiguous.  Slot s is token s % page_size of page
// s / page_size.
#pragma once

#include "kv_internal.h"
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

// n / d for 0 <= n < 2^31 with the constants of KvDiv (a multiply-high, an
// add and a shift instead of the ~20 instructions of a 32-bit division).
__device__ __forceinline__ uint32_t kv_div(uint32_t n, const KvDiv& d) {
  return (__umulhi(n, d.mul) + n) >> d.shift;
}

// Row (page, head, offset) of the codes and scales: its index counted in rows.
__device__ __forceinline__ int64_t kv_row(const KvCache& c, int page, int head, int off) {
  return ((int64_t)page * c.heads + head) * c.page_size + off;
}

}  // namespace nvfp4
