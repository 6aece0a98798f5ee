// grouped_gemm.cuh -- device helpers of the products grouped by expert.
#pragma once

#include "block_common.cuh"
#include "grouped_gemm.h"

namespace moe {

// Routed rows [beg, end) of expert e below the capacity; empty where the handle
// holds no segment.
MOE_DEVICE void gemm_segment(const int32_t* offsets, const int32_t* counts, int64_t cap, int e, int64_t& beg,
                             int64_t& end) {
  const int64_t off = offsets[e], cnt = counts[e];
  beg = min64(max64(off, 0), cap);
  end = off < 0 || cnt <= 0 ? beg : max64(min64(off + cnt, cap), beg);
}

}  // namespace moe
