// router.cu -- top-k router of the MoE layer (logits -> routing map and
// probabilities) and the gradient of its logits.
//
// One warp per token; lane l holds experts l, l + 32, ... in registers.  The
// selection finds the K-th largest score exactly: scores become unsigned keys
// of the same order, and the threshold is built bit by bit from the count of
// keys at or above a candidate.  Everything above it is chosen, and the lowest
// experts among those equal to it fill the rest, so ties, masked experts and
// rows with fewer than K experts left need no case of their own, and ids come
// out ascending.  Scores and sums are fp32 in a fixed order.
#include "block_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

struct RouterParams {
  int64_t T, stride;
  int E, K;
  int score, renorm, format;
  float scale;
  const void* logits;
  const float* bias;
  void* map;
  float* probs;
  int32_t* status;
};

// Unsigned key in the order of the floats (+0 and -0 equal); 0 for -inf and NaN.
MOE_DEVICE uint32_t score_key(float v) {
  if (!(v > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 -> +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// exp(l - top), with the limit 1 where l is top (both may be +inf).
MOE_DEVICE float exp_below(float l, float top) { return l == top ? 1.0f : expf(l - top); }

// sigmoid(l) * exp(-m) for m = min(largest l, 0): the common factor keeps the
// ratio of two sigmoids when both are far below the smallest float.
MOE_DEVICE float sigmoid_scaled(float l, float m) {
  return l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / (1.0f + expf(l));
}

// 1 - sigmoid(l)
MOE_DEVICE float sigmoid_rest(float l) {
  if (l < 0.0f) return 1.0f / (1.0f + expf(l));
  const float z = expf(-l);
  return z / (1.0f + z);
}

template <typename T, int V>  // V values a lane: E <= 32 V
__global__ void __launch_bounds__(kThreads) router_topk_kernel(RouterParams p) {
  const int lane = threadIdx.x & 31;
  const unsigned below = lanemask_lt();
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < p.T; t += (int64_t)gridDim.x * kWarps) {
    const T* row = static_cast<const T*>(p.logits) + t * p.stride;
    float l[V];
    uint32_t key[V];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const int e = j * 32 + lane;
      l[j] = e < p.E ? to_float(row[e]) : -INFINITY;
      bad |= l[j] != l[j];
      if (l[j] != l[j]) l[j] = -INFINITY;
      float s = l[j];
      if (p.bias && e < p.E && s > -INFINITY) {
        s = (p.score == MOE_SCORE_SIGMOID ? sigmoid_scaled(s, 0.0f) : s) + p.bias[e];
        bad |= s != s;
        if (!(s > -INFINITY)) l[j] = -INFINITY;
      }
      key[j] = score_key(s);
    }
    if (bad && p.status) atomicOr(p.status, MOE_DEV_ERR_NAN_LOGIT);

    // the K-th largest key (0 when fewer than K experts are left)
    uint32_t thr = 0;
    for (int b = 31; b >= 0; b--) {
      const uint32_t cand = thr | (1u << b);
      int n = 0;
#pragma unroll
      for (int j = 0; j < V; j++) n += key[j] >= cand;
      if (__reduce_add_sync(kAll, n) >= p.K) thr = cand;
    }
    int above = 0;
#pragma unroll
    for (int j = 0; j < V; j++) above += key[j] > thr;
    int ties = thr ? p.K - (int)__reduce_add_sync(kAll, above) : 0;

    // chosen experts in ascending order, and the largest logit among them
    unsigned chosen[V];
    float top = -INFINITY, top_all = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const bool eq = thr && key[j] == thr;
      const unsigned eqs = __ballot_sync(kAll, eq);
      const bool on = key[j] > thr || (eq && __popc(eqs & below) < ties);
      ties -= min(ties, __popc(eqs));
      chosen[j] = __ballot_sync(kAll, on);
      if (on) top = fmaxf(top, l[j]);
      top_all = fmaxf(top_all, l[j]);
    }
    top = warp_max(top);
    top_all = warp_max(top_all);

    const float m = fminf(top, 0.0f);
    float z = 0.0f, w[V];
#pragma unroll
    for (int j = 0; j < V; j++) {
      const bool on = chosen[j] >> lane & 1;
      if (p.score == MOE_SCORE_SOFTMAX) {
        w[j] = l[j] > -INFINITY ? exp_below(l[j], p.renorm ? top : top_all) : 0.0f;
        z += on || !p.renorm ? w[j] : 0.0f;
      } else {
        w[j] = on ? sigmoid_scaled(l[j], p.renorm ? m : 0.0f) : 0.0f;
        z += w[j];
      }
    }
    z = warp_sum(z);
    const bool divide = p.score == MOE_SCORE_SOFTMAX || p.renorm;
    int slot = 0;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const bool on = chosen[j] >> lane & 1;
      const int e = j * 32 + lane;
      const float v = p.scale * (divide ? w[j] / z : w[j]);
      if (p.format == MOE_ROUTING_DENSE_I16) {
        if (on) {
          const int64_t k = t * p.K + slot + __popc(chosen[j] & below);
          static_cast<int16_t*>(p.map)[k] = (int16_t)e;
          p.probs[k] = v;
        }
        slot += __popc(chosen[j]);
      } else if (e < p.E) {
        static_cast<uint8_t*>(p.map)[t * p.E + e] = on;
        p.probs[t * p.E + e] = on ? v : 0.0f;
      }
    }
    if (p.format == MOE_ROUTING_DENSE_I16) {
      for (int k = slot + lane; k < p.K; k += 32) {
        static_cast<int16_t*>(p.map)[t * p.K + k] = -1;
        p.probs[t * p.K + k] = 0.0f;
      }
    }
  }
}

struct RouterBwdParams {
  int64_t T, stride, gstride;
  int E, K;
  int score, renorm, format;
  float scale;
  const void *logits, *map;
  const float* gp;
  void* gl;
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) router_bwd_kernel(RouterBwdParams p) {
  extern __shared__ float smem[];  // dense maps: a row of gradients and one of marks per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* grow = smem + warp * 2 * p.E;
  float* mark = grow + p.E;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.T; t += (int64_t)gridDim.x * kWarps) {
    const T* row = static_cast<const T*>(p.logits) + t * p.stride;
    if (p.format == MOE_ROUTING_DENSE_I16) {
      for (int e = lane; e < p.E; e += 32) mark[e] = 0.0f;
      __syncwarp();
      for (int k = lane; k < p.K; k += 32) {
        const int e = static_cast<const int16_t*>(p.map)[t * p.K + k];
        if (e >= 0 && e < p.E) {
          grow[e] = p.gp[t * p.K + k];
          mark[e] = 1.0f;
        }
      }
      __syncwarp();
    }
    float l[V], g[V];
    unsigned on = 0;
    float top = -INFINITY, top_on = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const int e = j * 32 + lane;
      l[j] = e < p.E ? to_float(row[e]) : -INFINITY;
      if (l[j] != l[j]) l[j] = -INFINITY;
      bool c = false;
      if (e < p.E)
        c = p.format == MOE_ROUTING_DENSE_I16 ? mark[e] != 0.0f
                                              : static_cast<const uint8_t*>(p.map)[t * p.E + e] != 0;
      c = c && l[j] > -INFINITY;  // a masked expert has no gradient
      g[j] = 0.0f;
      if (c) g[j] = p.format == MOE_ROUTING_DENSE_I16 ? grow[e] : p.gp[t * p.E + e];
      on |= (unsigned)c << j;
      top = fmaxf(top, l[j]);
      if (c) top_on = fmaxf(top_on, l[j]);
    }
    top = warp_max(top);
    top_on = warp_max(top_on);
    // n: the score each expert takes part with; z its sum; dot = sum of g n
    float n[V], z = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const bool c = on >> j & 1;
      if (p.score == MOE_SCORE_SOFTMAX)
        n[j] = (c || !p.renorm) && l[j] > -INFINITY ? exp_below(l[j], p.renorm ? top_on : top) : 0.0f;
      else
        n[j] = c ? sigmoid_scaled(l[j], p.renorm ? fminf(top_on, 0.0f) : 0.0f) : 0.0f;
      z += n[j];
      dot = fmaf(g[j], n[j], dot);
    }
    const bool divide = p.score == MOE_SCORE_SOFTMAX || p.renorm;
    float inv = 1.0f;
    if (divide) {
      z = warp_sum(z);
      dot = warp_sum(dot);
      inv = z > 0.0f ? 1.0f / z : 0.0f;
      dot *= inv;
    } else {
      dot = 0.0f;
    }
    T* out = static_cast<T*>(p.gl) + t * p.gstride;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const int e = j * 32 + lane;
      float v = 0.0f;
      if (n[j] != 0.0f) {
        v = p.scale * (n[j] * inv) * (g[j] - dot);
        if (p.score == MOE_SCORE_SIGMOID) v *= sigmoid_rest(l[j]);
      }
      if (e < p.E) out[e] = from_float<T>(v);
    }
    __syncwarp();
  }
}

unsigned token_grid(int64_t T) {
  const int64_t blocks = (T + kWarps - 1) / kWarps, cap = (int64_t)device_sm_count() * (2048 / kThreads);
  return (unsigned)(blocks < cap ? blocks : cap);
}

template <typename T>
void run_topk(const RouterParams& p, cudaStream_t st) {
  const unsigned grid = token_grid(p.T);
  if (p.E <= 64)
    router_topk_kernel<T, 2><<<grid, kThreads, 0, st>>>(p);
  else if (p.E <= 128)
    router_topk_kernel<T, 4><<<grid, kThreads, 0, st>>>(p);
  else if (p.E <= 256)
    router_topk_kernel<T, 8><<<grid, kThreads, 0, st>>>(p);
  else if (p.E <= 512)
    router_topk_kernel<T, 16><<<grid, kThreads, 0, st>>>(p);
  else
    router_topk_kernel<T, 32><<<grid, kThreads, 0, st>>>(p);
}

template <typename T, int V>
cudaError_t run_bwd_v(const RouterBwdParams& p, cudaStream_t st) {
  const size_t smem = p.format == MOE_ROUTING_DENSE_I16 ? (size_t)kWarps * 2 * p.E * sizeof(float) : 0;
  static PerDeviceOnce once;  // E = 1024: 64 KB
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(router_bwd_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kWarps * 2 * 1024 * (int)sizeof(float));
  });
  if (e != cudaSuccess) return e;
  router_bwd_kernel<T, V><<<token_grid(p.T), kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_bwd(const RouterBwdParams& p, cudaStream_t st) {
  if (p.E <= 64) return run_bwd_v<T, 2>(p, st);
  if (p.E <= 128) return run_bwd_v<T, 4>(p, st);
  if (p.E <= 256) return run_bwd_v<T, 8>(p, st);
  if (p.E <= 512) return run_bwd_v<T, 16>(p, st);
  return run_bwd_v<T, 32>(p, st);
}

}  // namespace

cudaError_t launch_router_topk(const moe_router& r, const moe_rows& logits, const float* bias, int32_t format,
                               void* map, float* probs, int32_t* status, cudaStream_t st) {
  RouterParams p = {};
  p.T = r.T;
  p.E = (int)r.E;
  p.K = (int)r.K;
  p.score = r.score;
  p.renorm = r.renormalize != 0;
  p.scale = r.scale;
  p.format = format;
  p.logits = logits.data;
  p.stride = logits.stride;
  p.bias = bias;
  p.map = map;
  p.probs = probs;
  p.status = status;
  switch (r.logits_dtype) {
    case MOE_ELEM_F32: run_topk<float>(p, st); break;
    case MOE_ELEM_BF16: run_topk<__nv_bfloat16>(p, st); break;
    default: run_topk<__half>(p, st); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_router_topk_backward(const moe_router& r, const moe_rows& logits, int32_t format, const void* map,
                                        const float* grad_probs, const moe_rows& grad_logits, cudaStream_t st) {
  RouterBwdParams p = {};
  p.T = r.T;
  p.E = (int)r.E;
  p.K = (int)r.K;
  p.score = r.score;
  p.renorm = r.renormalize != 0;
  p.scale = r.scale;
  p.format = format;
  p.logits = logits.data;
  p.stride = logits.stride;
  p.map = map;
  p.gp = grad_probs;
  p.gl = grad_logits.data;
  p.gstride = grad_logits.stride;
  switch (r.logits_dtype) {
    case MOE_ELEM_F32: return run_bwd<float>(p, st);
    case MOE_ELEM_BF16: return run_bwd<__nv_bfloat16>(p, st);
    default: return run_bwd<__half>(p, st);
  }
}

}  // namespace moe
