// rms_norm.cu -- root-mean-square norm of hidden states, forward (with the
// residual sum in front, and an 8-bit output) and backward (with the weight's
// gradient).
//
// forward, per row:  h = x + residual;  rstd = 1 / sqrt(sum h^2 / H + eps);  v = h rstd w
//   y = v, rounded to the rows' type;  and / or, per block of 128 elements of v,
//   scale = amax / 448,  code = E4M3(v / scale)
// backward, per row, with xhat = h rstd and u = gy w:
//   gx = rstd (u - xhat sum(u xhat) / H) (+ gsum),  gw = sum over rows of gy xhat
// Every sum is fp32: a lane's elements in order, then a fixed shuffle tree.  The
// codes are those of v in fp32, not of its rounding to the rows' type: one rounding
// less, and y need not be written for them.
//
// The kernels are the layer norm's (row_norm.cuh) with one reduction a row less.
// HBM bounds them.  Device times on one GB300 (share of a copy's rate):
//   forward   8192 x 7168 bf16, residual, y and codes   87 us, 90 %
//             65536 x 1024 residual and y 89 us, 88 %; codes in the place of y 102 us, 68 % (instructions)
//             4096 x 4096 fp32, residual, y and codes   48 us, 88 %
//             8000 x 1001 bf16 y 11.7 us, 40 %; with codes, element by element, 36 us
//             one row of 7168, residual, y and codes    3.5 us (launch, one row's chain)
//   backward  8192 x 7168 bf16 with the residual's gradient 75 us, 92 %
//             65536 x 1024 87 us, 91 %; 4096 x 4096 fp32 45 us, 88 %
#include "row_norm.cuh"

namespace moe {

size_t rms_norm_workspace_bytes(int64_t rows, int64_t H) {
  // a partial sum per chunk of rows or per CTA, whichever kernel runs
  const int64_t n = rows < 1 ? 1 : rows < kMaxChunks ? rows : kMaxChunks;
  return (size_t)n * (size_t)H * sizeof(float);
}

cudaError_t launch_rms_norm(const moe_norm& n, const moe_rows& x, const moe_rows* res, const void* w,
                            const moe_rows* y, const moe_rows* sum, float* rstd, void* codes, float* scales,
                            cudaStream_t st) {
  NormParams p = {};
  p.rows = n.rows;
  p.H = n.H;
  p.eps = n.eps;
  p.x = x.data;
  p.sx = x.stride;
  if (res) p.res = res->data, p.sres = res->stride;
  if (sum) p.sum = sum->data, p.ssum = sum->stride;
  if (y) p.y = y->data, p.sy = y->stride;
  p.w = w;
  p.rstd = rstd;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  const bool f32_params = n.param_dtype == MOE_ELEM_F32;
  switch (n.dtype) {
    case MOE_ELEM_F32: return run_forward<float, float, true>(p, st);
    case MOE_ELEM_BF16:
      return f32_params ? run_forward<__nv_bfloat16, float, true>(p, st)
                        : run_forward<__nv_bfloat16, __nv_bfloat16, true>(p, st);
    default: return f32_params ? run_forward<__half, float, true>(p, st) : run_forward<__half, __half, true>(p, st);
  }
}

cudaError_t launch_rms_norm_backward(const moe_norm& n, const moe_rows& gy, const moe_rows& h, const void* w,
                                     const float* rstd, const moe_rows* gsum, const moe_rows& gx, float* gw,
                                     void* workspace, cudaStream_t st) {
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
  p.rstd = rstd;
  p.gw = gw;
  p.pw = static_cast<float*>(workspace);
  const bool f32_params = n.param_dtype == MOE_ELEM_F32;
  switch (n.dtype) {
    case MOE_ELEM_F32: return run_backward<float, float, true>(p, st);
    case MOE_ELEM_BF16:
      return f32_params ? run_backward<__nv_bfloat16, float, true>(p, st)
                        : run_backward<__nv_bfloat16, __nv_bfloat16, true>(p, st);
    default: return f32_params ? run_backward<__half, float, true>(p, st) : run_backward<__half, __half, true>(p, st);
  }
}

}  // namespace moe
