// layer_norm.cu -- layer norm of hidden states, forward (with the residual sum
// in front) and backward (with the weight's and bias's gradients).
//
// forward, per row:  h = x + residual;  mean = sum h / H;
//   rstd = 1 / sqrt(sum (h - mean)^2 / H + eps);  y = (h - mean) rstd w + b
// backward, per row, with xhat = (h - mean) rstd and u = gy w:
//   gx = rstd (u - sum u / H - xhat sum(u xhat) / H) (+ gsum)
//   gw = sum over rows of gy xhat,  gb = sum over rows of gy
// Every sum is fp32: a lane's elements in order, then a fixed shuffle tree.
//
// Both passes read and write each row once (forward 2 to 4 values an element,
// backward 3 or 4), so that HBM is the floor.  Device times on one GB300 (GB/s of
// that floor beside a copy's 6793):
//   forward   8192 x 7168 bf16 + residual   73 us, 6400     65536 x 1024   47 us, 5750
//             4096 x 4096 fp32              26 us, 5200     8000 x 1001    15 us, 2070
//             one row of 7168               3.3 us
//   backward  8192 x 7168 bf16 + gsum       75 us, 6240     65536 x 1024   70 us, 5780
//             4096 x 4096 fp32              35 us, 5720     1531 x 1537 fp32 11.7 us, 2410
//             2048 x 16384 bf16             64 us, 3160     64 x 7168      7.8 us
// Calls of a few microseconds are bound by their launches and one row's chain of
// load, two sums and store; unaligned rows by their masks and, forward, by spills
// (below), narrow ones also by the finishing launch backward; forward rows beyond
// 2048 pieces (2048 x 16384 bf16 34 us, 3940) by one CTA an SM that waits at two
// barriers a row and spills.
#include "row_norm.cuh"

namespace moe {

size_t layer_norm_workspace_bytes(int64_t rows, int64_t H) {
  // a partial sum per chunk of rows or per CTA, whichever kernel runs
  const int64_t n = rows < 1 ? 1 : rows < kMaxChunks ? rows : kMaxChunks;
  return (size_t)n * (size_t)H * 2 * sizeof(float);
}

cudaError_t launch_layer_norm(const moe_norm& n, const moe_rows& x, const moe_rows* res, const void* w, const void* b,
                              const moe_rows& y, const moe_rows* sum, float* mean, float* rstd, cudaStream_t st) {
  NormParams p = {};
  p.rows = n.rows;
  p.H = n.H;
  p.eps = n.eps;
  p.x = x.data;
  p.sx = x.stride;
  if (res) p.res = res->data, p.sres = res->stride;
  if (sum) p.sum = sum->data, p.ssum = sum->stride;
  p.y = y.data;
  p.sy = y.stride;
  p.w = w;
  p.b = b;
  p.mean = mean;
  p.rstd = rstd;
  const bool f32_params = n.param_dtype == MOE_ELEM_F32;
  switch (n.dtype) {
    case MOE_ELEM_F32: return run_forward<float, float, false>(p, st);
    case MOE_ELEM_BF16:
      return f32_params ? run_forward<__nv_bfloat16, float, false>(p, st)
                        : run_forward<__nv_bfloat16, __nv_bfloat16, false>(p, st);
    default: return f32_params ? run_forward<__half, float, false>(p, st) : run_forward<__half, __half, false>(p, st);
  }
}

cudaError_t launch_layer_norm_backward(const moe_norm& n, const moe_rows& gy, const moe_rows& h, const void* w,
                                       const float* mean, const float* rstd, const moe_rows* gsum, const moe_rows& gx,
                                       float* gw, float* gb, void* workspace, cudaStream_t st) {
  NormBwdParams p = {};
  p.rows = n.rows;
  p.H = n.H;
  p.gy = gy.data;
  p.sgy = gy.stride;
  p.h = h.data;
  p.sh = h.stride;
  if (gsum) p.gsum = gsum->data, p.sgsum = gsum->stride;
  p.gx = gx.data;
  p.sgx = gx.stride;
  p.w = w;
  p.mean = mean;
  p.rstd = rstd;
  p.gw = gw;
  p.gb = gb;
  p.pw = static_cast<float*>(workspace);
  const bool f32_params = n.param_dtype == MOE_ELEM_F32;
  switch (n.dtype) {
    case MOE_ELEM_F32: return run_backward<float, float, false>(p, st);
    case MOE_ELEM_BF16:
      return f32_params ? run_backward<__nv_bfloat16, float, false>(p, st)
                        : run_backward<__nv_bfloat16, __nv_bfloat16, false>(p, st);
    default: return f32_params ? run_backward<__half, float, false>(p, st) : run_backward<__half, __half, false>(p, st);
  }
}

}  // namespace moe
