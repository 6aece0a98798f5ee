// swiglu.cu -- SwiGLU of dispatched rows between FC1 and FC2, with the routes'
// probabilities, and its gradient.
//
// With u the first I columns of a row, g the others, s = 1 / (1 + exp(-g)), p the
// row's probability (1 without):
//   a  = p g s u
//   gu = ga p g s,  gg = ga p u s (1 + g (1 - s)),  gp = sum over columns of ga g s u
// in fp32, each result rounded once.  s and 1 - s are formed from exp(-|g|), so that
// neither overflows or cancels: with z = exp(-|g|), s = (g < 0 ? z : 1) / (1 + z) and
// 1 - s = (g < 0 ? 1 : z) / (1 + z).
//
// Each element is read and written once (3 values forward, 5 backward): HBM bounds
// both.  A team of threads takes a routed row; pad rows are known by token_of and
// left alone.  On one GB300, device time and share of a copy's rate: 65536 routed
// rows of I = 2048 in bf16 123 us forward (96 %) and 207 backward (95 %), 16384 of
// I = 4096 in fp32 121 and 198 (98 and 99 %); 64 tokens of 8 experts each among 256
// (512 routed rows of 8192) 6 and 10 us, launch and two chains of loads.
#include "block_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct SwigluParams {
  const int32_t *offsets, *token_of;
  int E;
  int64_t cap, I;
  int64_t spre, sga, sout;
  const void *pre, *ga;
  void* out;  // a, or gu and gg
  const float* probs;
  float* gp;
};

// 16 bytes of a row as they are loaded, or one element where rows are not aligned.
template <typename T, int N>
struct Raw {
  using type = uint4;
};
template <typename T>
struct Raw<T, 1> {
  using type = T;
};

template <typename T, int N>
MOE_DEVICE void unpack(float (&v)[N], const typename Raw<T, N>::type& raw) {
  if constexpr (N == 1) {
    v[0] = to_float(raw);
  } else {
    T e[N];
    *reinterpret_cast<uint4*>(e) = raw;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = to_float(e[i]);
  }
}

template <typename T, int N>
MOE_DEVICE typename Raw<T, N>::type pack(const float (&v)[N]) {
  if constexpr (N == 1) {
    return from_float<T>(v[0]);
  } else {
    T e[N];
#pragma unroll
    for (int i = 0; i < N; i++) e[i] = from_float<T>(v[i]);
    return *reinterpret_cast<const uint4*>(e);
  }
}

struct Gate {
  float s, c;  // sigmoid, 1 - sigmoid
};

// For 16-bit rows the exponential and the quotient are CUDA's fast ones, below
// (10 + 2.4 |g|) 2^-24 of s together, far below the rounding of the 16-bit results; the
// full ones would be what bounds the kernels (65536 x 2048 bf16: 215 us, so 132; backward
// 282 and 228).  Backward the exponential is the full one all the same: the gradient of
// the probabilities is fp32 whatever the rows, and has 12 2^-24 of s so whatever g (with
// the fast one 55 2^-24 was seen at g = -60; 206.5 us for 204, 4096 x 8 x 1024 60 for
// 56; with the full quotient too 252).  fp32 rows have half the elements a byte and take
// both.
template <typename T, bool FULL_EXP>
MOE_DEVICE Gate gate_of(float g) {
  constexpr bool kFast = sizeof(T) == 2;
  const float z = kFast && !FULL_EXP ? __expf(-fabsf(g)) : expf(-fabsf(g));
  const float r = kFast ? __fdividef(1.0f, 1.0f + z) : 1.0f / (1.0f + z);
  const float zr = z * r;
  return g < 0.0f ? Gate{zr, r} : Gate{r, zr};
}

// Calls f(row, probability) for the routed rows of a team.  Rows are `step` apart; a
// warp looks at 32 of them at once, so that pad rows (decode: most of them) cost no
// chain of loads each.
template <typename F>
MOE_DEVICE void routed_rows(const SwigluParams& p, int64_t first, int64_t step, F&& f) {
  const int64_t rows = min64(p.offsets[p.E], p.cap);
  const int lane = threadIdx.x & 31;
  for (int64_t base = first; base < rows; base += 32 * step) {
    const int64_t mine = base + lane * step;
    const bool routed = mine < rows && p.token_of[mine] >= 0;
    const float prob = routed && p.probs ? p.probs[mine] : 1.0f;
    for (unsigned left = __ballot_sync(0xffffffffu, routed); left; left &= left - 1) {
      const int j = __ffs(left) - 1;
      f(base + j * step, __shfl_sync(0xffffffffu, prob, j));
    }
  }
}

// TEAM threads a row: a warp, or the CTA.  A thread's loads of a batch of pieces are
// all on their way before it stores the first result, which the compiler may not do
// by itself.  Pieces of a batch: two of a 16-bit row forward (65536 x 2048: 123 us,
// four 129) and four of the others (backward 204 then, two 231; fp32 forward 121 and 131).
template <typename T, int N, int TEAM>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluParams p) {
  using R = typename Raw<T, N>::type;
  constexpr int kBatch = N == 1 ? 8 : sizeof(T) == 2 ? 2 : 4, kTeams = kThreads / TEAM, kStep = TEAM * N;
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  routed_rows(p, (int64_t)blockIdx.x * kTeams + team, (int64_t)gridDim.x * kTeams, [&](int64_t r, float prob) {
    const T* up = static_cast<const T*>(p.pre) + r * p.spre;
    const T* gate = up + p.I;
    T* a = static_cast<T*>(p.out) + r * p.sout;
    for (int64_t c0 = (int64_t)t * N; c0 < p.I; c0 += kBatch * kStep) {
      R ru[kBatch], rg[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (c0 + j * kStep < p.I) {
          ru[j] = *reinterpret_cast<const R*>(up + c0 + j * kStep);
          rg[j] = *reinterpret_cast<const R*>(gate + c0 + j * kStep);
        }
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (c0 + j * kStep < p.I) {
          float u[N], g[N];
          unpack<T, N>(u, ru[j]);
          unpack<T, N>(g, rg[j]);
#pragma unroll
          for (int i = 0; i < N; i++) u[i] = prob * (g[i] * gate_of<T, false>(g[i]).s * u[i]);
          *reinterpret_cast<R*>(a + c0 + j * kStep) = pack<T, N>(u);
        }
    }
  });
}

template <typename T, int N, int TEAM>
__global__ void __launch_bounds__(kThreads) swiglu_bwd_kernel(SwigluParams p) {
  using R = typename Raw<T, N>::type;
  constexpr int kBatch = N == 1 ? 8 : 4, kTeams = kThreads / TEAM, kStep = TEAM * N;
  __shared__ float2 red[2][kThreads / 32];
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  int phase = 0;
  routed_rows(p, (int64_t)blockIdx.x * kTeams + team, (int64_t)gridDim.x * kTeams, [&](int64_t r, float prob) {
    const T* up = static_cast<const T*>(p.pre) + r * p.spre;
    const T* gate = up + p.I;
    const T* ga = static_cast<const T*>(p.ga) + r * p.sga;
    T* gu = static_cast<T*>(p.out) + r * p.sout;
    T* gg = gu + p.I;
    float sum = 0.0f;
    for (int64_t c0 = (int64_t)t * N; c0 < p.I; c0 += kBatch * kStep) {
      R ru[kBatch], rg[kBatch], rd[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (c0 + j * kStep < p.I) {
          ru[j] = *reinterpret_cast<const R*>(up + c0 + j * kStep);
          rg[j] = *reinterpret_cast<const R*>(gate + c0 + j * kStep);
          rd[j] = *reinterpret_cast<const R*>(ga + c0 + j * kStep);
        }
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (c0 + j * kStep < p.I) {
          float u[N], g[N], d[N];
          unpack<T, N>(u, ru[j]);
          unpack<T, N>(g, rg[j]);
          unpack<T, N>(d, rd[j]);
#pragma unroll
          for (int i = 0; i < N; i++) {
            const Gate q = gate_of<T, true>(g[i]);
            const float act = g[i] * q.s;
            sum = fmaf(d[i], act * u[i], sum);
            d[i] *= prob;
            g[i] = d[i] * u[i] * (q.s * fmaf(g[i], q.c, 1.0f));
            u[i] = d[i] * act;
          }
          *reinterpret_cast<R*>(gu + c0 + j * kStep) = pack<T, N>(u);
          *reinterpret_cast<R*>(gg + c0 + j * kStep) = pack<T, N>(g);
        }
    }
    if (p.gp) {
      if (TEAM == 32)
        sum = warp_sum(sum);
      else
        sum = block_sum2(sum, 0.0f, red[phase]).x;
      phase ^= 1;
      if (t == 0) p.gp[r] = sum;
    }
  });
}

bool aligned_rows(const void* p, int64_t stride, int64_t rows, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || stride * bytes % 16 == 0);
}

template <typename T, int N, int TEAM>
cudaError_t run_team(const SwigluParams& p, bool backward, cudaStream_t st) {
  const int64_t teams = kThreads / TEAM, blocks = (p.cap + teams - 1) / teams;
  const int64_t most = (int64_t)device_sm_count() * (2048 / kThreads);
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (backward)
    swiglu_bwd_kernel<T, N, TEAM><<<grid, kThreads, 0, st>>>(p);
  else
    swiglu_kernel<T, N, TEAM><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int N>
cudaError_t run_pieces(const SwigluParams& p, int64_t routes, bool backward, cudaStream_t st) {
  // rows for every SM's CTAs, or rows too short for more than a warp: a warp a row
  if (routes >= (int64_t)device_sm_count() * 8 || p.I <= 32 * N) return run_team<T, N, 32>(p, backward, st);
  return run_team<T, N, kThreads>(p, backward, st);
}

template <typename T>
cudaError_t run(const SwigluParams& p, int64_t routes, bool backward, cudaStream_t st) {
  constexpr int b = sizeof(T), N = 16 / b;
  const bool vec = p.I * b % 16 == 0 && aligned_rows(p.pre, p.spre, p.cap, b) && aligned_rows(p.out, p.sout, p.cap, b) &&
                   aligned_rows(p.ga, p.sga, p.cap, b);
  return vec ? run_pieces<T, N>(p, routes, backward, st) : run_pieces<T, 1>(p, routes, backward, st);
}

cudaError_t dispatch(const SwigluParams& p, int32_t dtype, int64_t routes, bool backward, cudaStream_t st) {
  switch (dtype) {
    case MOE_ELEM_F32: return run<float>(p, routes, backward, st);
    case MOE_ELEM_BF16: return run<__nv_bfloat16>(p, routes, backward, st);
    default: return run<__half>(p, routes, backward, st);
  }
}

SwigluParams params(const moe_handle_dev& h, const moe_shape& s, const moe_layout& l, int64_t I, const moe_rows& pre,
                    const moe_rows& out, const float* probs) {
  SwigluParams p = {};
  p.offsets = h.padded_offsets;
  p.token_of = h.token_of;
  p.E = (int)s.E;
  p.cap = l.capacity;
  p.I = I;
  p.pre = pre.data;
  p.spre = pre.stride;
  p.out = out.data;
  p.sout = out.stride;
  p.probs = probs;
  return p;
}

}  // namespace

cudaError_t launch_swiglu(const moe_handle_dev& h, const moe_shape& s, const moe_layout& l, int64_t I, int32_t dtype,
                          const moe_rows& pre, const float* probs, const moe_rows& act, cudaStream_t st) {
  return dispatch(params(h, s, l, I, pre, act, probs), dtype, s.T * s.K, false, st);
}

cudaError_t launch_swiglu_backward(const moe_handle_dev& h, const moe_shape& s, const moe_layout& l, int64_t I,
                                   int32_t dtype, const moe_rows& pre, const float* probs, const moe_rows& grad_act,
                                   const moe_rows& grad_pre, float* grad_probs, cudaStream_t st) {
  SwigluParams p = params(h, s, l, I, pre, grad_pre, probs);
  p.ga = grad_act.data;
  p.sga = grad_act.stride;
  p.gp = grad_probs;
  return dispatch(p, dtype, s.T * s.K, true, st);
}

}  // namespace moe
