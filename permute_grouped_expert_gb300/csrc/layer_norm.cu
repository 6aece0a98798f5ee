// layer_norm.cu -- layer norm of hidden states, forward (with the residual sum
// in front) and backward (with the weight's and bias's gradients).
//
// forward, per row:  h = x + residual;  mean = sum h / H;
//   rstd = 1 / sqrt(sum (h - mean)^2 / H + eps);  y = (h - mean) rstd w + b
// backward, per row, with xhat = (h - mean) rstd and u = gy w:
//   gx = rstd (u - sum u / H - xhat sum(u xhat) / H) (+ gsum)
//   gw = sum over rows of gy xhat,  gb = sum over rows of gy
// Every sum is fp32: a lane's elements in order, then a fixed shuffle tree.
#include "block_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct NormParams {
  int64_t rows, H;
  int64_t sx, sres, sy, ssum;
  const void *x, *res, *w, *b;
  void *y, *sum;
  float *mean, *rstd;
  float eps;
};

// Any width, stride and alignment: one CTA per row, three passes over the row
// (the second and third mostly from L1 / L2).
template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) layer_norm_any_kernel(NormParams p) {
  __shared__ float2 red[2][kWarps];
  const P* w = static_cast<const P*>(p.w);
  const P* b = static_cast<const P*>(p.b);
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + r * p.sx;
    const T* res = p.res ? static_cast<const T*>(p.res) + r * p.sres : nullptr;
    T* sum = p.sum ? static_cast<T*>(p.sum) + r * p.ssum : nullptr;
    T* y = static_cast<T*>(p.y) + r * p.sy;
    // the residual sum as it is stored; a thread rereads only what it wrote
    auto h_at = [&](int64_t c) {
      if (!res) return to_float(x[c]);
      if (sum) return to_float(sum[c]);
      return to_float(from_float<T>(to_float(x[c]) + to_float(res[c])));
    };
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < p.H; c += kThreads) {
      if (sum) sum[c] = from_float<T>(to_float(x[c]) + to_float(res[c]));
      s += h_at(c);
    }
    const float mean = block_sum2(s, 0.0f, red[0]).x / (float)p.H;
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < p.H; c += kThreads) {
      const float d = h_at(c) - mean;
      q = fmaf(d, d, q);
    }
    const float var = block_sum2(q, 0.0f, red[1]).x / (float)p.H;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    for (int64_t c = threadIdx.x; c < p.H; c += kThreads) {
      float v = (h_at(c) - mean) * rstd;
      if (w) v *= to_float(w[c]);
      if (b) v += to_float(b[c]);
      y[c] = from_float<T>(v);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
}

struct NormBwdParams {
  int64_t rows, H;
  int64_t sgy, sh, sgsum, sgx;
  const void *gy, *h, *w, *gsum;
  void* gx;
  const float *mean, *rstd;
  float *pw, *pb;  // partial sums [chunks][H]
  float *gw, *gb;
  int64_t chunks, rows_per_chunk;
};

template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) layer_norm_bwd_rows_any_kernel(NormBwdParams p) {
  __shared__ float2 red[kWarps];
  const P* w = static_cast<const P*>(p.w);
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* gy = static_cast<const T*>(p.gy) + r * p.sgy;
    const T* h = static_cast<const T*>(p.h) + r * p.sh;
    const T* gsum = p.gsum ? static_cast<const T*>(p.gsum) + r * p.sgsum : nullptr;
    T* gx = static_cast<T*>(p.gx) + r * p.sgx;
    const float mean = p.mean[r], rstd = p.rstd[r];
    float su = 0.0f, sx = 0.0f;
    for (int64_t c = threadIdx.x; c < p.H; c += kThreads) {
      const float u = to_float(gy[c]) * (w ? to_float(w[c]) : 1.0f);
      su += u;
      sx = fmaf(u, (to_float(h[c]) - mean) * rstd, sx);
    }
    const float2 t = block_sum2(su, sx, red);
    const float mu = t.x / (float)p.H, mx = t.y / (float)p.H;
    for (int64_t c = threadIdx.x; c < p.H; c += kThreads) {
      const float u = to_float(gy[c]) * (w ? to_float(w[c]) : 1.0f);
      float v = rstd * (u - mu - (to_float(h[c]) - mean) * rstd * mx);
      if (gsum) v += to_float(gsum[c]);
      gx[c] = from_float<T>(v);
    }
    __syncthreads();
  }
}

// Partial column sums: a CTA takes 32 columns and one chunk of rows, eight rows
// at a time, and adds its eight row lanes up in order.  It runs before the row
// kernel, whose gx may replace gy.
template <typename T>
__global__ void __launch_bounds__(kThreads) layer_norm_bwd_cols_kernel(NormBwdParams p) {
  __shared__ float2 part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int64_t beg = blockIdx.y * p.rows_per_chunk, end = min64(beg + p.rows_per_chunk, p.rows);
  float aw = 0.0f, ab = 0.0f;
  if (c < p.H) {
    for (int64_t r = beg + warp; r < end; r += kWarps) {
      const float g = to_float(static_cast<const T*>(p.gy)[r * p.sgy + c]);
      const float xhat = (to_float(static_cast<const T*>(p.h)[r * p.sh + c]) - p.mean[r]) * p.rstd[r];
      aw = fmaf(g, xhat, aw);
      ab += g;
    }
  }
  part[warp][lane] = make_float2(aw, ab);
  __syncthreads();
  if (warp == 0 && c < p.H) {
    float2 s = part[0][lane];
    for (int i = 1; i < kWarps; i++) {
      s.x += part[i][lane].x;
      s.y += part[i][lane].y;
    }
    p.pw[blockIdx.y * p.H + c] = s.x;
    p.pb[blockIdx.y * p.H + c] = s.y;
  }
}

// Adds the chunks' partial sums up in order.
__global__ void __launch_bounds__(kThreads) layer_norm_bwd_finish_kernel(NormBwdParams p) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.H) return;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t k = 0; k < p.chunks; k++) {
    sw += p.pw[k * p.H + c];
    sb += p.pb[k * p.H + c];
  }
  if (p.gw) p.gw[c] = sw;
  if (p.gb) p.gb[c] = sb;
}

constexpr int64_t kMaxChunks = 304;

int64_t bwd_chunks(int64_t rows) {
  int64_t n = (rows + 31) / 32;
  return n < 1 ? 1 : n > kMaxChunks ? kMaxChunks : n;
}

unsigned row_grid(int64_t rows) {
  const int64_t cap = (int64_t)device_sm_count() * (2048 / kThreads);
  return (unsigned)(rows < cap ? rows : cap);
}

template <typename T, typename P>
cudaError_t run_forward(const NormParams& p, cudaStream_t st) {
  layer_norm_any_kernel<T, P><<<row_grid(p.rows), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t run_backward(const NormBwdParams& p, cudaStream_t st) {
  if (p.gw || p.gb) {
    layer_norm_bwd_cols_kernel<T><<<dim3((unsigned)((p.H + 31) / 32), (unsigned)p.chunks), kThreads, 0, st>>>(p);
    layer_norm_bwd_finish_kernel<<<(unsigned)((p.H + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  }
  if (p.rows > 0) layer_norm_bwd_rows_any_kernel<T, P><<<row_grid(p.rows), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t layer_norm_workspace_bytes(int64_t rows, int64_t H) {
  return (size_t)bwd_chunks(rows) * (size_t)H * 2 * sizeof(float);
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
    case MOE_ELEM_F32: return run_forward<float, float>(p, st);
    case MOE_ELEM_BF16:
      return f32_params ? run_forward<__nv_bfloat16, float>(p, st) : run_forward<__nv_bfloat16, __nv_bfloat16>(p, st);
    default: return f32_params ? run_forward<__half, float>(p, st) : run_forward<__half, __half>(p, st);
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
  p.chunks = bwd_chunks(n.rows);
  p.rows_per_chunk = (n.rows + p.chunks - 1) / p.chunks;
  p.pw = static_cast<float*>(workspace);
  p.pb = p.pw ? p.pw + p.chunks * n.H : nullptr;
  const bool f32_params = n.param_dtype == MOE_ELEM_F32;
  switch (n.dtype) {
    case MOE_ELEM_F32: return run_backward<float, float>(p, st);
    case MOE_ELEM_BF16:
      return f32_params ? run_backward<__nv_bfloat16, float>(p, st)
                        : run_backward<__nv_bfloat16, __nv_bfloat16>(p, st);
    default: return f32_params ? run_backward<__half, float>(p, st) : run_backward<__half, __half>(p, st);
  }
}

}  // namespace moe
