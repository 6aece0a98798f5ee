// grouped_gemm.h -- what the kernels of the products grouped by expert share.
#pragma once

#include "moe_internal.h"

namespace moe {

// The three products of an expert's matrix W [N][Kd] and its rows:
//   kForward  y[r]  = W x[r]            rows of Kd -> rows of N
//   kData     gx[r] = W^T gy[r]         rows of N  -> rows of Kd
//   kWeight   gW    = sum gy[r] x[r]^T  rows of N and of Kd -> a matrix
enum GemmDir { kForward = 0, kData = 1, kWeight = 2 };

struct GroupedGemm {
  const int32_t *offsets, *counts;  // [E+1], [E]
  int32_t* status;
  int64_t E, cap, T, K;  // T, K: tokens, routes a token (the most routed rows are T K)
  int64_t N, Kd;
  int32_t dtype, out_dtype;  // MOE_ELEM_*; out_dtype is that of W's gradient
  const void *a, *b;         // kForward: x, W;  kData: gy, W;  kWeight: gy, x
  int64_t sa, sb;            // strides of rows
  void* out;
  int64_t sout;
  const float* addend;  // kWeight, or NULL
  void* workspace;
};

size_t grouped_gemm_workspace_bytes(const moe_shape& s, const moe_layout& l, int64_t N, int64_t Kd);
// Whether the tiles of the rows' products can be counted (what does not fit is far
// beyond any memory).
bool grouped_gemm_counts(const moe_shape& s, const moe_layout& l, int64_t features);
cudaError_t launch_grouped_gemm(GemmDir dir, const GroupedGemm& g, cudaStream_t st);

}  // namespace moe
