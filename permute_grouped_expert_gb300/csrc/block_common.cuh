// block_common.cuh -- element types and row loads shared by the operators
// around the layer (layer norm, router, 4-bit matrix-vector products).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_common.cuh"

namespace moe {

MOE_DEVICE float to_float(float v) { return v; }
MOE_DEVICE float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
MOE_DEVICE float to_float(__half v) { return __half2float(v); }

// One rounding, to nearest even.
template <typename T>
MOE_DEVICE T from_float(float v);
template <>
MOE_DEVICE float from_float<float>(float v) {
  return v;
}
template <>
MOE_DEVICE __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
MOE_DEVICE __half from_float<__half>(float v) {
  return __float2half_rn(v);
}

MOE_DEVICE float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

MOE_DEVICE float warp_max(float v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// Sums of two values over the block, known to every thread.  `red` holds two
// floats per warp; the caller synchronises before it is used again.
MOE_DEVICE float2 block_sum2(float a, float b, float2* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  a = warp_sum(a);
  b = warp_sum(b);
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  float2 v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  return v;
}

}  // namespace moe
