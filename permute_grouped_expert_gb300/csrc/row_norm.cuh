// row_norm.cuh -- the kernels of the norms over rows: layer norm (layer_norm.cu)
// and, with RMS set, root-mean-square norm (rms_norm.cu): no mean, no bias, and an
// 8-bit output with scales beside or in the place of the other.  Each file has its
// formulas, times and what bounds it.
#pragma once

#include <algorithm>
#include <type_traits>

#include "block_common.cuh"
#include "moe_internal.h"
#include "row_pieces.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

constexpr int kCodeBlock = 128;  // elements of a row that share a scale of the 8-bit output

// The larger of two magnitudes, NaN if either is.
MOE_DEVICE float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct NormParams {
  int64_t rows, H;
  int64_t sx, sres, sy, ssum;
  const void *x, *res, *w, *b;
  void *y, *sum;
  float *mean, *rstd;
  float eps;
  uint8_t* codes;  // [rows][H]
  float* scales;   // [rows][blocks of H]
  int64_t cut;  // SHIFTED: from this row on pieces may end behind a matrix
};

// Scale of a block of the 8-bit output, and the block's codes: scale = amax / 448,
// 1 for a block of zeros; code = E4M3(v / scale), to nearest even, saturating.  A
// scale that is subnormal or infinite goes by the division itself: its reciprocal
// and the correction step leave fp32's range.
MOE_DEVICE float code_scale(float amax) {
  const float s = amax / 448.0f;
  return s == 0.0f ? 1.0f : s;
}

MOE_DEVICE bool plain_scale(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

// Any width, stride and alignment: one CTA per row, three passes over the row
// (the second and third mostly from L1 / L2).
template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) row_norm_any_kernel(NormParams p) {
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

// The same without a mean, and with codes: one CTA per row.  HELD: the row stays in
// shared memory between its sum of squares and its results (22650 x 1641 bf16 codes
// 131 us, read again element by element 174; instructions, about 100 an element and
// warp, bound it); rows that it cannot hold are read again.  The results are
// formed a block of codes at a time by a warp each.
template <typename T, typename P, bool HELD>
__global__ void __launch_bounds__(kThreads) rms_any_kernel(NormParams p) {
  constexpr int kAhead = 8;  // elements of a thread on their way
  __shared__ float2 red[2][kWarps];
  extern __shared__ __align__(16) uint8_t staged[];
  T* held = reinterpret_cast<T*>(staged);
  const P* w = static_cast<const P*>(p.w);
  const int lane = threadIdx.x & 31;
  const int H = (int)p.H, blocks = (H + kCodeBlock - 1) / kCodeBlock;
  int phase = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + r * p.sx;
    const T* res = p.res ? static_cast<const T*>(p.res) + r * p.sres : nullptr;
    T* sum = p.sum ? static_cast<T*>(p.sum) + r * p.ssum : nullptr;
    T* y = p.y ? static_cast<T*>(p.y) + r * p.sy : nullptr;
    auto sum_of = [&](T a, T b) { return from_float<T>(to_float(a) + to_float(b)); };
    float q = 0.0f;
    for (int c0 = threadIdx.x; c0 < H; c0 += kAhead * kThreads) {
      T a[kAhead], b[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int c = c0 + i * kThreads;
        if (c < H) a[i] = x[c];
        if (c < H && res) b[i] = res[c];
      }
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int c = c0 + i * kThreads;
        if (c >= H) continue;
        const T h = res ? sum_of(a[i], b[i]) : a[i];
        if (sum) sum[c] = h;
        if (HELD) held[c] = h;
        q = fmaf(to_float(h), to_float(h), q);
      }
    }
    const float rstd = 1.0f / sqrtf(block_sum2(q, 0.0f, red[phase]).x / (float)p.H + p.eps);  // (and the row is there)
    phase ^= 1;
    for (int k = threadIdx.x >> 5; k < blocks; k += kWarps) {
      float v[kCodeBlock / 32], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < kCodeBlock / 32; i++) {
        const int c = k * kCodeBlock + i * 32 + lane;
        v[i] = 0.0f;
        if (c < H) {
          const T h = HELD ? held[c] : !res ? x[c] : sum ? sum[c] : sum_of(x[c], res[c]);
          v[i] = to_float(h) * rstd * (w ? to_float(w[c]) : 1.0f);
          if (y) y[c] = from_float<T>(v[i]);
        }
        amax = nan_max(amax, fabsf(v[i]));
      }
      if (!p.codes) continue;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) amax = nan_max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      const float scale = code_scale(amax), inv = 1.0f / scale;
      const bool plain = plain_scale(scale);
      uint8_t* codes = p.codes + r * p.H;
#pragma unroll
      for (int i = 0; i < kCodeBlock / 32; i++) {
        const int c = k * kCodeBlock + i * 32 + lane;
        if (c < H) codes[c] = (uint8_t)e4m3x2(plain ? div_by_scale(v[i], scale, inv) : v[i] / scale, 0.0f);
      }
      if (lane == 0) p.scales[r * (int64_t)blocks + k] = scale;
    }
    if (threadIdx.x == 0 && p.rstd) p.rstd[r] = rstd;
    __syncthreads();  // the row's place is written again
  }
}

// 16 bytes of a row as fp32.
template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
  T e[kN];
};

template <typename T>
MOE_DEVICE void load_vec(float (&out)[Vec<T>::kN], const T* p) {
  union {
    uint4 v;
    Vec<T> t;
  } u;
  u.v = *reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < Vec<T>::kN; i++) out[i] = to_float(u.t.e[i]);
}

// Parameters of the same columns: fp32 or the rows' type.
template <typename T, typename P>
MOE_DEVICE void load_params(float (&out)[Vec<T>::kN], const P* p) {
  constexpr int kPieces = Vec<T>::kN * (int)sizeof(P) / 16;  // 1, or 2 for fp32 beside 16-bit rows
#pragma unroll
  for (int k = 0; k < kPieces; k++) {
    float part[Vec<P>::kN];
    load_vec<P>(part, p + k * Vec<P>::kN);
#pragma unroll
    for (int i = 0; i < Vec<P>::kN; i++) out[k * Vec<P>::kN + i] = part[i];
  }
}

template <typename T>
MOE_DEVICE void unpack(float (&out)[Vec<T>::kN], uint4 raw) {
  union {
    uint4 v;
    Vec<T> t;
  } u;
  u.v = raw;
#pragma unroll
  for (int i = 0; i < Vec<T>::kN; i++) out[i] = to_float(u.t.e[i]);
}

template <typename T>
MOE_DEVICE uint4 pack(const float (&in)[Vec<T>::kN]) {
  union {
    uint4 v;
    Vec<T> t;
  } u;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; i++) u.t.e[i] = in[i];
  } else {  // two at a time
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(in[2 * i], in[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(in[2 * i], in[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    u.v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return u.v;
}

// SHIFTED kernels take rows that start anywhere as the aligned 16-byte pieces
// that hold them: `skip` elements of a row's first piece lie before it.  A team's
// rows lie a multiple of 16 bytes apart, so that its threads keep their columns.
// Element by element (the any kernels) 8000 x 1001 bf16 took 35 us forward and 49
// backward; as pieces it takes 15 and 22.  They need rows that start alike in
// every matrix; what does not is left to the any kernels.
// Bit k: element k of the piece whose first column is c0 belongs to the row.
template <int N>
MOE_DEVICE uint32_t piece_mask(int c0, int H) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < N; k++) m |= (c0 + k >= 0 && c0 + k < H ? 1u : 0u) << k;
  return m;
}

// A piece with zeros outside the row.
template <typename T>
MOE_DEVICE uint4 masked_piece(uint4 raw, uint32_t mask) {
  union {
    uint4 v;
    T e[Vec<T>::kN];
  } u;
  u.v = raw;
#pragma unroll
  for (int k = 0; k < Vec<T>::kN; k++)
    if (!(mask >> k & 1)) u.e[k] = from_float<T>(0.0f);
  return u.v;
}

// A piece with a neighbour's elements, if any, outside the row: they are part of
// the matrix but in its last rows (`cut`, see first_cut_row), where they are not read.
template <typename T, bool SHIFTED>
MOE_DEVICE uint4 load_piece(const T* p, uint32_t mask, bool cut) {
  constexpr int N = Vec<T>::kN;
  if (!SHIFTED || !cut || mask == (1u << N) - 1) return *reinterpret_cast<const uint4*>(p);
  union {
    uint4 v;
    T e[N];
  } u;
  u.v = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < N; k++)
    if (mask >> k & 1) u.e[k] = p[k];
  return u.v;
}

template <typename T, bool SHIFTED>
MOE_DEVICE void store_piece(T* p, uint4 raw, uint32_t mask) {
  constexpr int N = Vec<T>::kN;
  if (!SHIFTED || mask == (1u << N) - 1) {
    *reinterpret_cast<uint4*>(p) = raw;
    return;
  }
  union {
    uint4 v;
    T e[N];
  } u;
  u.v = raw;
#pragma unroll
  for (int k = 0; k < N; k++)
    if (mask >> k & 1) p[k] = u.e[k];
}

// Parameters of a piece's columns; p: of its first.
template <typename T, typename P, bool SHIFTED>
MOE_DEVICE void piece_params(float (&out)[Vec<T>::kN], const P* p, uint32_t mask) {
  if (SHIFTED) {
#pragma unroll
    for (int k = 0; k < Vec<T>::kN; k++)
      if (mask >> k & 1) out[k] = to_float(p[k]);
  } else {
    load_params<T, P>(out, p);
  }
}

// Codes of a row held as V pieces a thread (0 past its end).  A block is
// kCodeBlock / N consecutive pieces: those of neighbouring lanes, and of several v
// where a team is narrower than a block.
template <typename T, int V, int LANES>
MOE_DEVICE void store_codes(const NormParams& p, const float (&h)[V][Vec<T>::kN], int64_t r, int t, int team, int n) {
  constexpr int N = Vec<T>::kN, kPieces = kCodeBlock / N;  // pieces of a block
  constexpr int kLanes = LANES && LANES < kPieces ? LANES : kPieces;
  constexpr int kJoin = kPieces / kLanes < V ? kPieces / kLanes : V;  // a thread's pieces of one block
  const int64_t blocks = (p.H + kCodeBlock - 1) / kCodeBlock;
#pragma unroll
  for (int v0 = 0; v0 < V; v0 += kJoin) {
    float amax = 0.0f;
#pragma unroll
    for (int v = v0; v < v0 + kJoin; v++)
#pragma unroll
      for (int k = 0; k < N; k++) amax = nan_max(amax, fabsf(h[v][k]));
#pragma unroll
    for (int d = kLanes / 2; d >= 1; d >>= 1) amax = nan_max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const float scale = code_scale(amax), inv = 1.0f / scale;
    const bool plain = plain_scale(scale);
#pragma unroll
    for (int v = v0; v < v0 + kJoin; v++) {
      const int piece = v * team + t;
      if (piece >= n) continue;
      uint32_t w[N / 4];
#pragma unroll
      for (int i = 0; i < N / 4; i++) {
        float q[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
          q[k] = plain ? div_by_scale(h[v][4 * i + k], scale, inv) : h[v][4 * i + k] / scale;
        w[i] = e4m3x2(q[0], q[1]) | (uint32_t)e4m3x2(q[2], q[3]) << 16;
      }
      uint8_t* to = p.codes + r * p.H + (int64_t)piece * N;
      if constexpr (N == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(to) = w[0];
      if (piece % kPieces == 0) p.scales[r * blocks + piece / kPieces] = scale;
    }
  }
}

// rstd is rsqrtf's, within 2 ulp of the any kernels' 1 / sqrtf: a row's last bits
// depend on which kernel its alignment gives it.
// Rows of 16-byte vectors held in registers between the mean, the variance and
// the result, so that the row is read once, V vectors a thread.  LANES threads
// of a warp take a row; or (0) a CTA does, and its next row is on its way while
// it reduces and writes this one: two barriers a row would leave the memory idle
// (8192 x 7168 bf16 with a residual: 109 us without, 76 when it came in).  Teams of a warp
// have enough others to wait for: with a ring of their own 8192 x 7168 took 162.
template <typename T, typename P, int V, int LANES, int THREADS, bool SHIFTED, bool RMS, bool CODES>
__global__ void __launch_bounds__(THREADS, LANES ? 4 : 1024 / THREADS) row_norm_vec_kernel(NormParams p) {
  static_assert(!CODES || (RMS && !SHIFTED), "codes come of aligned rows without a mean");
  constexpr int N = Vec<T>::kN;
  constexpr bool kAhead = LANES == 0;
  // vectors past the end are computed with the rest (0, and the first weights) and
  // not stored, where registers allow: a few branches a row less (8192 x 7168 with a
  // residual 75.7 -> 73.4 us; 65536 x 1024, which spills, 47.8 -> 52.0)
  constexpr bool kStraight = LANES == 0 && !SHIFTED;
  __shared__ float2 red[2][THREADS / 32];
  const int team = LANES ? LANES : (int)blockDim.x, teams = LANES ? THREADS / LANES : 1;
  const int t = LANES ? threadIdx.x % LANES : threadIdx.x;
  // rows of block number n; SHIFTED: eight apart, so that its rows (and those of
  // every block that this CTA takes, the grid being a multiple of eight) start alike
  const int own = LANES ? threadIdx.x / LANES : 0;
  auto row_of = [&](int64_t n) { return SHIFTED ? ((n >> 3) * teams + own) * 8 + (n & 7) : n * teams + own; };
  const int64_t blocks = SHIFTED ? (p.rows + 8 * teams - 1) / (8 * teams) * 8 : (p.rows + teams - 1) / teams;
  const int skip = SHIFTED ? (int)((blockIdx.x & 7) * p.sx % N) : 0;
  const int nvec = ((int)p.H + skip + N - 1) / N, v_step = team * N;
  const int c0 = t * N - skip;  // this thread's first column
  uint32_t mask[V];             // of its pieces
#pragma unroll
  for (int v = 0; v < V; v++) mask[v] = SHIFTED ? piece_mask<N>(c0 + v * v_step, (int)p.H) : ~0u;
  const P* w = static_cast<const P*>(p.w) + (p.w ? c0 : 0);
  const P* b = static_cast<const P*>(p.b) + (p.b ? c0 : 0);
  extern __shared__ __align__(16) uint8_t staged[];  // SHIFTED: the parameters as the rows' pieces lie
  auto total = [&](float v, float2* r) {
    if (!LANES) return block_sum2(v, 0.0f, r).x;
#pragma unroll
    for (int d = LANES / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  uint4 x_raw[V], res_raw[V];
  bool edge = false;  // a piece of this thread holds elements outside the row
#pragma unroll
  for (int v = 0; v < V; v++) edge |= SHIFTED && mask[v] != (1u << N) - 1;
  auto fetch_x = [&](int64_t r, int n) {
    const T* x = static_cast<const T*>(p.x) + r * p.sx + c0;
#pragma unroll
    for (int v = 0; v < V; v++) {
      x_raw[v] = make_uint4(0, 0, 0, 0);
      if (v * team + t < n) x_raw[v] = load_piece<T, SHIFTED>(x + v * v_step, mask[v], r >= p.cut);
    }
  };
  auto fetch_res = [&](int64_t r, int v) {
    const T* res = static_cast<const T*>(p.res) + r * p.sres + c0 + v * v_step;
    return load_piece<T, SHIFTED>(res, mask[v], r >= p.cut);
  };
  auto fetch = [&](int64_t r) {
    fetch_x(r, nvec);
    if (p.res) {
#pragma unroll
      for (int v = 0; v < V; v++)
        if (v * team + t < nvec) res_raw[v] = fetch_res(r, v);
    }
  };
  if (kAhead && row_of(blockIdx.x) < p.rows) fetch(row_of(blockIdx.x));
  if (SHIFTED) {
    P* sw = reinterpret_cast<P*>(staged);
    P* sb = sw + nvec * N;
    for (int i = threadIdx.x; i < nvec * N; i += (int)blockDim.x) {
      const int c = i - skip;
      const bool in = c >= 0 && c < (int)p.H;
      sw[i] = in && p.w ? static_cast<const P*>(p.w)[c] : from_float<P>(0.0f);
      sb[i] = in && p.b ? static_cast<const P*>(p.b)[c] : from_float<P>(0.0f);
    }
    w = sw + t * N;
    b = sb + t * N;
    __syncthreads();
  }
  int phase = 0;
  for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
    // a team past the last row has no columns: its warp shuffles together
    const int64_t r = row_of(block), next = row_of(block + gridDim.x);
    if (SHIFTED && !LANES && r >= p.rows) break;
    const int n = r < p.rows ? nvec : 0;
    float h[V][N];
    if (!kAhead) fetch_x(r, n);
    if (SHIFTED && edge) {
#pragma unroll
      for (int v = 0; v < V; v++) x_raw[v] = masked_piece<T>(x_raw[v], mask[v]);
    }
#pragma unroll
    for (int v = 0; v < V; v++) unpack<T>(h[v], x_raw[v]);
    if (p.res) {
      T* sum = static_cast<T*>(p.sum) + (p.sum ? r * p.ssum + c0 : 0);
#pragma unroll
      for (int v = 0; v < V; v++) {
        if (v * team + t < n) {
          float a[N];
          const uint4 raw = kAhead ? res_raw[v] : fetch_res(r, v);
          unpack<T>(a, SHIFTED && edge ? masked_piece<T>(raw, mask[v]) : raw);
#pragma unroll
          for (int k = 0; k < N; k++) a[k] += h[v][k];
          const uint4 packed = pack<T>(a);  // the norm is that of the sum as stored
          unpack<T>(h[v], packed);
          if (p.sum) store_piece<T, SHIFTED>(sum + v * v_step, packed, mask[v]);
        }
      }
    }
    if (kAhead && next < p.rows) fetch(next);
    float mean = 0.0f;
    if (!RMS) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int k = 0; k < N; k++) s += h[v][k];  // 0 outside the row
      mean = total(s, red[0]) / (float)p.H;
    }
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
      const bool in = v * team + t < n;
      if (!kStraight && !in) continue;
      const float off = in ? mean : 0.0f;
#pragma unroll
      for (int k = 0; k < N; k++) {
        if (!RMS) h[v][k] -= off;
        if (SHIFTED) h[v][k] = mask[v] >> k & 1 ? h[v][k] : 0.0f;
        q = fmaf(h[v][k], h[v][k], q);
      }
    }
    const float rstd = rsqrtf(total(q, red[RMS ? phase : 1]) / (float)p.H + p.eps);
    if (RMS) phase ^= 1;  // one barrier a row: the sums of the row before may still be read
    T* y = static_cast<T*>(p.y) + (!RMS || p.y ? r * p.sy + c0 : 0);
#pragma unroll
    for (int v = 0; v < V; v++) {
      const bool in = v * team + t < n;
      if (!kStraight && !in) continue;
      float g[N], c[N];
#pragma unroll
      for (int k = 0; k < N; k++) g[k] = 1.0f, c[k] = 0.0f;
      if (p.w) load_params<T, P>(g, in ? w + v * v_step : static_cast<const P*>(p.w));
      if (!RMS && p.b) load_params<T, P>(c, in ? b + v * v_step : static_cast<const P*>(p.b));
#pragma unroll
      for (int k = 0; k < N; k++) {
        if (RMS) {
          g[k] = h[v][k] * rstd * g[k];
          if (CODES) h[v][k] = in ? g[k] : 0.0f;
        } else {
          g[k] = fmaf(h[v][k] * rstd, g[k], c[k]);
        }
      }
      if (in && (!RMS || p.y)) store_piece<T, SHIFTED>(y + v * v_step, pack<T>(g), mask[v]);
    }
    if constexpr (CODES) store_codes<T, V, LANES>(p, h, r, t, team, n);
    if (t == 0 && r < p.rows) {
      if (!RMS && p.mean) p.mean[r] = mean;
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

template <typename T, typename P, bool RMS>
__global__ void __launch_bounds__(kThreads) row_norm_bwd_rows_any_kernel(NormBwdParams p) {
  __shared__ float2 red[kWarps];
  const P* w = static_cast<const P*>(p.w);
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* gy = static_cast<const T*>(p.gy) + r * p.sgy;
    const T* h = static_cast<const T*>(p.h) + r * p.sh;
    const T* gsum = p.gsum ? static_cast<const T*>(p.gsum) + r * p.sgsum : nullptr;
    T* gx = static_cast<T*>(p.gx) + r * p.sgx;
    const float mean = RMS ? 0.0f : p.mean[r], rstd = p.rstd[r];
    float su = 0.0f, sx = 0.0f;
    for (int64_t c = threadIdx.x; c < p.H; c += kThreads) {
      const float u = to_float(gy[c]) * (w ? to_float(w[c]) : 1.0f);
      if (!RMS) su += u;
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
template <typename T, bool RMS>
__global__ void __launch_bounds__(kThreads) row_norm_bwd_cols_kernel(NormBwdParams p) {
  __shared__ float2 part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int64_t beg = blockIdx.y * p.rows_per_chunk, end = min64(beg + p.rows_per_chunk, p.rows);
  float aw = 0.0f, ab = 0.0f;
  if (c < p.H) {
    for (int64_t r = beg + warp; r < end; r += kWarps) {
      const float g = to_float(static_cast<const T*>(p.gy)[r * p.sgy + c]);
      const float xhat = (to_float(static_cast<const T*>(p.h)[r * p.sh + c]) - (RMS ? 0.0f : p.mean[r])) * p.rstd[r];
      aw = fmaf(g, xhat, aw);
      if (!RMS) ab += g;
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
    if (!RMS) p.pb[blockIdx.y * p.H + c] = s.y;
  }
}

// The first `bytes` of a piece, zeros behind them.
MOE_DEVICE void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Sums of two values over a team of `warps` warps, known to its threads; one
// barrier.  Halves of a warp reduce one value each.  `red`: a float2 per warp,
// not written again before the team's next barrier but one.
template <bool PART>
MOE_DEVICE float2 team_sum2(float a, float b, float2* red, int warp, int warps, int barrier, int threads) {
  if (PART) {  // `threads` lanes, a power of two: the teams of a warp at once
    for (int d = threads >> 1; d >= 1; d >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, d);
      b += __shfl_xor_sync(0xffffffffu, b, d);
    }
    return make_float2(a, b);
  }
  const int lane = threadIdx.x & 31;
  const bool low = lane < 16;
  auto halves = [&](float x, float y) {  // lanes 0-15: sum of x over the warp, 16-31: of y
    float v = (low ? x : y) + __shfl_xor_sync(0xffffffffu, low ? y : x, 16);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  float v = halves(a, b);
  if (warps > 1) {
    if ((lane & 15) == 0) reinterpret_cast<float*>(red + warp)[low ? 0 : 1] = v;
    __syncwarp();  // the barrier's form wants whole warps
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
    const float2 t = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    v = halves(t.x, t.y);
  }
  return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}

// Rows of 16-byte vectors: one pass that forms gx and a CTA's partial sums of
// gw and gb.  A team of threads takes a row, V vectors a thread, and keeps the
// sums of its columns in registers over the rows it meets; its next rows are on
// their way into a ring of 8 / V stages that is each thread's own, so that only the
// two sums of a row need a barrier.  Teams are a part of a warp (kPart), some
// warps of a CTA (kSome), or a cluster of CTAs (kCluster) for rows that the
// registers of one cannot hold.  What bounds it is the instructions a row takes:
// places in the ring are constants, addresses run along, vectors past the end are
// zeros in the ring and computed with the rest, and the weights stay in registers.
// Of a cluster's CTAs two share an SM, so that one works while the other waits for
// its cluster (1024 x 16384 fp32: 47 us, with one of 512 threads 52).
constexpr int kBwdBlock = 512, kClusterBlock = 256, kMaxCluster = 8;
enum Team { kPart, kSome, kCluster };
template <Team TEAM>
constexpr int kBlockOf = TEAM == kCluster ? kClusterBlock : kBwdBlock;
template <Team TEAM>
constexpr int kRing = kBlockOf<TEAM> * 16 * 3 * 8;  // eight vectors a thread of each of three matrices

MOE_DEVICE uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
MOE_DEVICE uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
  return r;
}

MOE_DEVICE void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of two values over a cluster: every warp leaves its sums in every CTA.
// `red`: a float2 per warp of the cluster, not written again before its next
// barrier but one.
MOE_DEVICE float2 cluster_sum2(float a, float b, float2* red) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, ctas = (int)cluster_size();
  const bool low = lane < 16;
  auto halves = [&](float x, float y) {
    float v = (low ? x : y) + __shfl_xor_sync(0xffffffffu, low ? y : x, 16);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  float v = halves(a, b);
  if ((lane & 15) < ctas) {
    const float* to = reinterpret_cast<const float*>(red + cluster_rank() * warps + (threadIdx.x >> 5)) + (low ? 0 : 1);
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(remote)
                 : "r"((uint32_t)__cvta_generic_to_shared(to)), "r"(lane & 15));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
  }
  cluster_barrier();
  float2 t = make_float2(0.0f, 0.0f);
  for (int i = lane; i < warps * ctas; i += 32) t.x += red[i].x, t.y += red[i].y;
  v = halves(t.x, t.y);
  return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}

template <typename T, typename P, Team TEAM, int V, bool SHIFTED, bool RMS>
__global__ void __launch_bounds__(kBlockOf<TEAM>, kBwdBlock / kBlockOf<TEAM>)
    row_norm_bwd_vec_kernel(NormBwdParams p, int team_threads) {
  constexpr int N = Vec<T>::kN, STAGES = 8 / V;
  constexpr bool PART = TEAM == kPart;
  // ring: [stage][matrix][vector of the thread][thread]
  constexpr int kVec = kBlockOf<TEAM> * 16, kMatrix = V * kVec, kStage = 3 * kMatrix;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 red[2][TEAM == kCluster ? kMaxCluster * kClusterBlock / 32 : 32];
  const int ctas = TEAM == kCluster ? (int)cluster_size() : 1, rank = TEAM == kCluster ? (int)cluster_rank() : 0;
  const int64_t unit = blockIdx.x / ctas, units = gridDim.x / ctas;  // CTA or cluster
  const int team = threadIdx.x / team_threads, teams = blockDim.x / team_threads;
  const int t = rank * (int)blockDim.x + threadIdx.x % team_threads;
  const int warp = t >> 5, warps = team_threads >> 5;
  const int64_t step = units * teams;
  const int64_t first = unit * teams + team;
  const int skip = SHIFTED ? (int)(first * p.sgy % N) : 0;
  const int nvec = ((int)p.H + skip + N - 1) / N, c0 = t * N - skip;  // this thread's first column
  const int rounds = first < p.rows ? (int)((p.rows - first + step - 1) / step) : 0;  // rows of this team
  // PART: teams of a part of a warp shuffle together: they go as many rounds as
  // the first, and their rounds past the last row are zeros in the ring
  const int loops = PART ? (int)((p.rows - (first - team) + step - 1) / step) : rounds;
  const float inv_h = 1.0f / (float)p.H;
  uint8_t* own = smem + threadIdx.x * 16;
  const uint32_t own_u32 = (uint32_t)__cvta_generic_to_shared(own);
  const int v_len = team_threads * ctas, v_step = v_len * N;
  bool in[V];
  uint32_t mask[V];  // of this thread's pieces
#pragma unroll
  for (int v = 0; v < V; v++) {
    in[v] = v * v_len + t < nvec;
    mask[v] = SHIFTED ? piece_mask<N>(c0 + v * v_step, (int)p.H) : ~0u;
    if (!in[v])
      for (int i = 0; i < 3 * STAGES; i++)
        *reinterpret_cast<uint4*>(own + i * kMatrix + v * kVec) = make_uint4(0, 0, 0, 0);
  }

  // where this thread's next copies come from, and where its results go
  const T* gy = static_cast<const T*>(p.gy) + first * p.sgy + c0;
  const T* h = static_cast<const T*>(p.h) + first * p.sh + c0;
  const T* gs = static_cast<const T*>(p.gsum) + (p.gsum ? first * p.sgsum + c0 : 0);
  T* gx = static_cast<T*>(p.gx) + first * p.sgx + c0;
  const int64_t gy_step = step * p.sgy, h_step = step * p.sh, gs_step = step * p.sgsum, gx_step = step * p.sgx;
  int to_fill = rounds;
  auto fill = [&](uint32_t dst) {
    if (to_fill > 0) {
#pragma unroll
      for (int v = 0; v < V; v++) {
        if (in[v]) {
          // the piece that ends a matrix may be short
          const int bytes = SHIFTED && to_fill == 1 ? min(16, ((int)p.H - c0 - v * v_step) * (int)sizeof(T)) : 16;
          cp_async16(dst + v * kVec, gy + v * v_step, bytes);
          cp_async16(dst + kMatrix + v * kVec, h + v * v_step, bytes);
          if (p.gsum) cp_async16(dst + 2 * kMatrix + v * kVec, gs + v * v_step, bytes);
        }
      }
      gy += gy_step;
      h += h_step;
      gs += gs_step;
    } else if (PART) {
#pragma unroll
      for (int i = 0; i < 3 * V; i++)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i * kVec), "r"(0) : "memory");
    }
    to_fill--;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

#pragma unroll
  for (int i = 0; i < STAGES - 1; i++) fill(own_u32 + i * kStage);
  float aw[V][N] = {}, ab[V][N] = {};
  const P* w = static_cast<const P*>(p.w) + (p.w ? c0 : 0);
  float wv[V][N];
#pragma unroll
  for (int v = 0; v < V; v++) {
#pragma unroll
    for (int k = 0; k < N; k++) wv[v][k] = 1.0f;
    if (p.w && in[v]) piece_params<T, P, SHIFTED>(wv[v], w + v * v_step, mask[v]);
  }
  // a row's mean and deviation are a lane's load for a whole batch of rows, a batch
  // ahead: loaded a row ahead, they were what each row waited for
  const int batch = PART ? team_threads : 32, lane = t & (batch - 1);
  float mean_now = 0.0f, rstd_now = 0.0f, mean_next = 0.0f, rstd_next = 0.0f;
  auto stats = [&](int round, float& m, float& d) {
    if (round < rounds) m = RMS ? 0.0f : p.mean[first + round * step], d = p.rstd[first + round * step];
  };
  stats(lane, mean_now, rstd_now);
  stats(batch + lane, mean_next, rstd_next);
  if (TEAM == kCluster) cluster_barrier();  // its CTAs have started
  int stage = 0, phase = 0;                 // stage: in bytes
  for (int round = 0; round < loops; round++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    fill(own_u32 + (stage == 0 ? (STAGES - 1) * kStage : stage - kStage));  // the stage of the row before
    const int place = round & (batch - 1);
    if (round > 0 && place == 0) {
      mean_now = mean_next;
      rstd_now = rstd_next;
      stats(round + batch + lane, mean_next, rstd_next);
    }
    const float mean = RMS ? 0.0f : __shfl_sync(0xffffffffu, mean_now, place, batch);
    const float rstd = __shfl_sync(0xffffffffu, rstd_now, place, batch);
    const uint8_t* at = own + stage;
    float su = 0.0f, sx = 0.0f;
    float u[V][N], xhat[V][N];
    auto staged = [&](int matrix, int v) {
      return *reinterpret_cast<const uint4*>(at + matrix * kMatrix + v * kVec);
    };
#pragma unroll
    for (int v = 0; v < V; v++) {
      unpack<T>(u[v], staged(0, v));
      unpack<T>(xhat[v], staged(1, v));
#pragma unroll
      for (int k = 0; k < N; k++) xhat[v][k] = RMS ? xhat[v][k] * rstd : (xhat[v][k] - mean) * rstd;
      if (SHIFTED && mask[v] != (1u << N) - 1) {  // a neighbour's elements
#pragma unroll
        for (int k = 0; k < N; k++)
          if (!(mask[v] >> k & 1)) u[v][k] = xhat[v][k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < N; k++) {
        aw[v][k] = fmaf(u[v][k], xhat[v][k], aw[v][k]);
        if (!RMS) ab[v][k] += u[v][k];
      }
#pragma unroll
      for (int k = 0; k < N; k++) {
        u[v][k] *= wv[v][k];
        if (!RMS) su += u[v][k];
        sx = fmaf(u[v][k], xhat[v][k], sx);
      }
    }
    const float2 sums = TEAM == kCluster ? cluster_sum2(su, sx, red[phase])
                                         : team_sum2<PART>(su, sx, red[phase] + team * warps, warp, warps, team + 1,
                                                           team_threads);
    const float mu = sums.x * inv_h, mx = sums.y * inv_h;
#pragma unroll
    for (int v = 0; v < V; v++) {
      float o[N];
      unpack<T>(o, p.gsum ? staged(2, v) : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int k = 0; k < N; k++) o[k] = fmaf(rstd, fmaf(-mx, xhat[v][k], RMS ? u[v][k] : u[v][k] - mu), o[k]);
      if (in[v] && (!PART || round < rounds)) store_piece<T, SHIFTED>(gx + v * v_step, pack<T>(o), mask[v]);
    }
    gx += gx_step;
    phase ^= 1;
    stage = stage == (STAGES - 1) * kStage ? 0 : stage + kStage;
  }
  if (!p.gw && !p.gb) return;

  // the CTA's partial sums: teams added up in order through the ring's memory
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int sum = 0; sum < (RMS ? 1 : 2); sum++) {
    float(&acc)[V][N] = sum ? ab : aw;
    if (SHIFTED && TEAM == kCluster) {
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int k = 0; k < N; k++)
          if (in[v] && mask[v] >> k & 1) (sum ? p.pb : p.pw)[unit * p.H + c0 + v * v_step + k] = acc[v][k];
      continue;
    }
    if (SHIFTED) {  // by column: the teams' pieces begin at different ones
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int k = 0; k < N; k++)
          if (in[v] && mask[v] >> k & 1) part[team * (int)p.H + c0 + v * v_step + k] = acc[v][k];
      __syncthreads();
      for (int c = threadIdx.x; c < (int)p.H; c += blockDim.x) {
        float s = part[c];
        for (int j = 1; j < teams; j++) s += part[j * (int)p.H + c];
        (sum ? p.pb : p.pw)[unit * p.H + c] = s;
      }
      continue;
    }
    if (teams > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int k = 0; k < N; k++) part[(v * N + k) * kBlockOf<TEAM> + threadIdx.x] = acc[v][k];
      __syncthreads();
      if (team == 0)
        for (int j = 1; j < teams; j++)
#pragma unroll
          for (int v = 0; v < V; v++)
#pragma unroll
            for (int k = 0; k < N; k++) acc[v][k] += part[(v * N + k) * kBlockOf<TEAM> + j * team_threads + t];
    }
    float* out = (sum ? p.pb : p.pw) + unit * p.H + t * N;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (team == 0 && in[v])
#pragma unroll
        for (int k = 0; k < N; k += 4)
          *reinterpret_cast<float4*>(out + v * v_step + k) =
              make_float4(acc[v][k], acc[v][k + 1], acc[v][k + 2], acc[v][k + 3]);
  }
}

// Adds the chunks' partial sums up: 32 columns a CTA, each warp every 16th chunk
// (so that a thread's loads are all on their way at once), the warps in order.
constexpr int kFinishWarps = 16, kFinishLoads = 10;

template <bool RMS>
__global__ void __launch_bounds__(kFinishWarps * 32) row_norm_bwd_finish_kernel(NormBwdParams p) {
  __shared__ float2 part[kFinishWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float2 s = make_float2(0.0f, 0.0f);
  if (c < p.H) {
    for (int64_t k0 = warp; k0 < p.chunks; k0 += kFinishWarps * kFinishLoads) {
      float2 v[kFinishLoads];
#pragma unroll
      for (int i = 0; i < kFinishLoads; i++) {
        const int64_t k = k0 + i * kFinishWarps;
        v[i] = k < p.chunks ? make_float2(p.pw[k * p.H + c], RMS ? 0.0f : p.pb[k * p.H + c]) : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int i = 0; i < kFinishLoads; i++) s.x += v[i].x, s.y += v[i].y;
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.H) {
    for (int i = 1; i < kFinishWarps; i++) s.x += part[i][lane].x, s.y += part[i][lane].y;
    if (p.gw) p.gw[c] = s.x;
    if (!RMS && p.gb) p.gb[c] = s.y;
  }
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows that start on 16 bytes and hold whole 16-byte vectors.
bool vector_rows(const void* p, int64_t stride, int64_t rows, int bytes) {
  return aligned16(p) && (rows <= 1 || stride * bytes % 16 == 0);
}

// Rows that start on pieces' elements alike: what the SHIFTED kernels take.
bool alike(const void* p, int64_t stride, int64_t other, int64_t rows, int n) {
  return !p || (aligned16(p) && (rows <= 1 || stride % n == other % n));
}

// CTAs that keep a team's rows a multiple of 16 bytes apart, unless each team has one row.
int64_t shifted_grid(int64_t grid, int64_t blocks) {
  if (blocks <= 8) return blocks;
  return grid >= blocks ? blocks : grid < 8 ? 8 : grid / 8 * 8;
}

constexpr int kMaxStaged = 200 * 1024;  // bytes of parameters a CTA stages at the most

template <typename T, typename P, bool RMS, bool CODES, bool SHIFTED, int LANES, int THREADS, int V = 4>
cudaError_t run_vec(const NormParams& p, cudaStream_t st) {
  const int n = 16 / (int)sizeof(T), pieces = (int)(p.H + (SHIFTED ? n - 1 : 0) + n - 1) / n;
  const int block = LANES ? THREADS : ((pieces + V - 1) / V + 31) / 32 * 32;
  const int teams = LANES ? THREADS / (LANES + !LANES) : 1, group = SHIFTED ? 8 : 1;
  const int64_t blocks = (p.rows + group * teams - 1) / (group * teams) * group;
  const int64_t cap = (int64_t)device_sm_count() * ((LANES ? 2048 : 1024) / block);
  const int64_t grid = blocks < cap ? blocks : cap < group ? group : cap / group * group;
  const int smem = SHIFTED ? pieces * n * (int)sizeof(P) * 2 : 0;
  if (SHIFTED) {
    static PerDeviceOnce once;
    cudaError_t e = once.run([] {
      return cudaFuncSetAttribute(row_norm_vec_kernel<T, P, V, LANES, THREADS, SHIFTED, RMS, CODES>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStaged);
    });
    if (e != cudaSuccess) return e;
  }
  row_norm_vec_kernel<T, P, V, LANES, THREADS, SHIFTED, RMS, CODES><<<(unsigned)grid, block, smem, st>>>(p);
  return cudaGetLastError();
}

// Up to 128 pieces a part of a warp takes a row, so that the narrowest rows leave
// no lanes idle (65536 x 128 bf16: 19 us with a warp a row, 8.7 so); above, the
// warps that hold it at two pieces a thread, which leaves registers for the next
// row.  Four pieces a thread (8192 x 7168: 157 us, against 76 then) and a warp with
// eight (4096 x 2048: 11.8, against 10.3 then) are slower; only rows past 2048 pieces
// need four.  Four 16-bit pieces beside masks and shifted addresses do not fit the 64
// registers of four CTAs an SM: the unaligned kernels of a part of a warp spill 60
// to 64 bytes a thread (8000 x 1001 bf16: 15.3 us), those of 1024 threads 236 to 260
// on aligned rows and 424 to 464 on others.
template <typename T, typename P, bool RMS, bool CODES, bool SHIFTED>
cudaError_t run_pieces(const NormParams& p, int64_t pieces, cudaStream_t st) {
  if (pieces <= 16) return run_vec<T, P, RMS, CODES, SHIFTED, 4, 256>(p, st);
  if (pieces <= 32) return run_vec<T, P, RMS, CODES, SHIFTED, 8, 256>(p, st);
  if (pieces <= 64) return run_vec<T, P, RMS, CODES, SHIFTED, 16, 256>(p, st);
  if (pieces <= 128) return run_vec<T, P, RMS, CODES, SHIFTED, 32, 256>(p, st);
  if (pieces <= 1024) return run_vec<T, P, RMS, CODES, SHIFTED, 0, 512, 2>(p, st);
  if (pieces <= 2048) return run_vec<T, P, RMS, CODES, SHIFTED, 0, 1024, 2>(p, st);
  return run_vec<T, P, RMS, CODES, SHIFTED, 0, 1024, 4>(p, st);
}

template <typename T, typename P>
cudaError_t run_rms_any(const NormParams& p, cudaStream_t st) {
  const int64_t bytes = p.H * (int64_t)sizeof(T);
  if (bytes > kMaxStaged) {
    rms_any_kernel<T, P, false><<<row_grid(p.rows), kThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(rms_any_kernel<T, P, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStaged);
  });
  if (e != cudaSuccess) return e;
  rms_any_kernel<T, P, true><<<row_grid(p.rows), kThreads, (size_t)bytes, st>>>(p);
  return cudaGetLastError();
}

template <typename T, typename P, bool RMS>
cudaError_t run_forward(NormParams p, cudaStream_t st) {
  const int b = sizeof(T), n = 16 / b;
  const int64_t pieces = (p.H + n - 1) / n;
  const bool vec = p.H * b % 16 == 0 && vector_rows(p.x, p.sx, p.rows, b) && vector_rows(p.res, p.sres, p.rows, b) &&
                   vector_rows(p.sum, p.ssum, p.rows, b) && vector_rows(p.y, p.sy, p.rows, b) && aligned16(p.w) &&
                   aligned16(p.b);
  const bool shifted = aligned16(p.x) && alike(p.res, p.sres, p.sx, p.rows, n) &&
                       alike(p.sum, p.ssum, p.sx, p.rows, n) && alike(p.y, p.sy, p.sx, p.rows, n);
  if (RMS && p.codes) {
    // whole pieces of codes: as wide as a row's pieces are long
    if (vec && pieces <= 4096 && (reinterpret_cast<uintptr_t>(p.codes) & (n - 1)) == 0)
      return run_pieces<T, P, RMS, RMS, false>(p, pieces, st);
    return run_rms_any<T, P>(p, st);
  }
  if (vec && pieces <= 4096)
    return run_pieces<T, P, RMS, false, false>(p, pieces, st);
  if (shifted && pieces < 4096 && (pieces + 1) * n * (int64_t)sizeof(P) * 2 <= kMaxStaged) {
    p.cut = first_cut_row(p.rows, p.sx, n);
    if (p.res) p.cut = std::min(p.cut, first_cut_row(p.rows, p.sres, n));
    return run_pieces<T, P, RMS, false, true>(p, pieces + 1, st);  // a row may touch one more
  }
  if constexpr (RMS) return run_rms_any<T, P>(p, st);
  row_norm_any_kernel<T, P><<<row_grid(p.rows), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// Partial sums of `chunks` units, after the kernel on `chunks` x `ctas` CTAs of them.
template <typename T, typename P, bool RMS, Team TEAM, int V, bool SHIFTED>
cudaError_t run_bwd_units(NormBwdParams p, int64_t chunks, int ctas, int block, int team, cudaStream_t st) {
  static_assert(kRing<TEAM> >= kBlockOf<TEAM> * 16 / (int)sizeof(T) * 4 * V, "the partial sums fit the ring");
  p.chunks = chunks;
  p.pb = p.pw + p.chunks * p.H;
  cudaLaunchAttribute cluster = {};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)ctas;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(chunks * ctas));
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = kRing<TEAM>;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, row_norm_bwd_vec_kernel<T, P, TEAM, V, SHIFTED, RMS>, p, team);
  if (e != cudaSuccess) return e;
  if (p.gw || p.gb) row_norm_bwd_finish_kernel<RMS><<<(unsigned)((p.H + 31) / 32), kFinishWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, typename P, bool RMS, Team TEAM, int V, bool SHIFTED>
cudaError_t allow_ring() {
  static PerDeviceOnce once;
  return once.run([] {
    return cudaFuncSetAttribute(row_norm_bwd_vec_kernel<T, P, TEAM, V, SHIFTED, RMS>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kRing<TEAM>);
  });
}

template <typename T, typename P, bool RMS, Team TEAM, int V, bool SHIFTED>
cudaError_t run_bwd_teams(const NormBwdParams& p, int64_t pieces, cudaStream_t st) {
  cudaError_t e = allow_ring<T, P, RMS, TEAM, V, SHIFTED>();
  if (e != cudaSuccess) return e;
  constexpr bool kParts = TEAM == kPart;
  const int want = (int)(pieces + V - 1) / V;
  const int team = !kParts ? (want + 31) / 32 * 32 : want <= 4 ? 4 : want <= 8 ? 8 : 16, whole = kParts ? 32 / team : 1;
  int teams = kBwdBlock / team;  // (teams of several warps: at most eight, named barriers 1 to 8)
  while (teams > whole && p.rows < (int64_t)teams * device_sm_count()) teams -= whole;  // whole warps
  const int64_t blocks = (p.rows + teams - 1) / teams, sms = device_sm_count();
  int64_t chunks = blocks < sms ? blocks : sms;
  if (chunks > kMaxChunks) chunks = kMaxChunks;
  if (SHIFTED) chunks = shifted_grid(chunks, blocks);
  return run_bwd_units<T, P, RMS, TEAM, V, SHIFTED>(p, chunks, 1, team * teams, team, st);
}

template <typename T, typename P, bool RMS, int V, bool SHIFTED>
cudaError_t run_bwd_clusters(const NormBwdParams& p, int64_t pieces, cudaStream_t st) {
  cudaError_t e = allow_ring<T, P, RMS, kCluster, V, SHIFTED>();
  if (e != cudaSuccess) return e;
  // as few as hold a row, a power of two or not (3000 x 9000 bf16: three 63 us, four
  // 74; unaligned 2048 x 16383: five 90, eight 126)
  const int least = (int)((pieces + V * kClusterBlock - 1) / (V * kClusterBlock)), ctas = least < 2 ? 2 : least;
  const int want = (int)(pieces + ctas - 1) / ctas, block = ((want + V - 1) / V + 31) / 32 * 32;
  // as many clusters as run at once: the GPU's parts need not be whole clusters
  static int at_once[PerDeviceOnce::kMaxDevices][kMaxCluster + 1];
  static PerDeviceOnce once;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run([&] {
    cudaError_t r = cudaSuccess;
    for (int i = 2; i <= kMaxCluster && r == cudaSuccess; i++) {
      cudaLaunchAttribute cluster = {};
      cluster.id = cudaLaunchAttributeClusterDimension;
      cluster.val.clusterDim.x = (unsigned)i;
      cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)i);
      cfg.blockDim = dim3(kClusterBlock);
      cfg.dynamicSmemBytes = kRing<kCluster>;
      cfg.attrs = &cluster;
      cfg.numAttrs = 1;
      r = cudaOccupancyMaxActiveClusters(&at_once[dev][i], row_norm_bwd_vec_kernel<T, P, kCluster, V, SHIFTED, RMS>, &cfg);
    }
    return r;
  });
  if (e != cudaSuccess) return e;
  int64_t chunks = at_once[dev][ctas] < 1 ? 1 : at_once[dev][ctas];
  if (chunks > kMaxChunks) chunks = kMaxChunks;
  if (chunks > p.rows) chunks = p.rows;
  if (SHIFTED) chunks = shifted_grid(chunks, p.rows);
  return run_bwd_units<T, P, RMS, kCluster, V, SHIFTED>(p, chunks, ctas, block, block, st);
}

// Up to 32 pieces teams are a part of a warp (65536 x 128 bf16: 21 us, with a warp
// a row 31), up to 1024 some warps at two pieces a thread.  Above, what registers
// can hold beside the columns' sums decides: fp32 rows go on with four pieces a
// thread (2048 x 8192: 37 us; clusters 60), 16-bit rows would spill (2048 x 16384:
// 97 us) and take clusters (64).
// Vectors that a thread's registers hold beside the columns' sums:
template <typename T>
constexpr int kMostVecs = 16 / Vec<T>::kN;

template <typename T, typename P, bool RMS, bool SHIFTED>
cudaError_t run_bwd_pieces(const NormBwdParams& p, int64_t pieces, cudaStream_t st) {
  if (pieces <= 32) return run_bwd_teams<T, P, RMS, kPart, 2, SHIFTED>(p, pieces, st);
  if (pieces <= 2 * kBwdBlock) return run_bwd_teams<T, P, RMS, kSome, 2, SHIFTED>(p, pieces, st);
  if constexpr (kMostVecs<T> > 2)
    if (pieces <= kMostVecs<T> * kBwdBlock) return run_bwd_teams<T, P, RMS, kSome, kMostVecs<T>, SHIFTED>(p, pieces, st);
  return run_bwd_clusters<T, P, RMS, kMostVecs<T>, SHIFTED>(p, pieces, st);
}

template <typename T, typename P, bool RMS>
cudaError_t run_backward(NormBwdParams p, cudaStream_t st) {
  const int b = sizeof(T), n = 16 / b;
  const int64_t pieces = (p.H + n - 1) / n;
  const bool vec = p.H * b % 16 == 0 && vector_rows(p.gy, p.sgy, p.rows, b) && vector_rows(p.h, p.sh, p.rows, b) &&
                   vector_rows(p.gsum, p.sgsum, p.rows, b) && vector_rows(p.gx, p.sgx, p.rows, b) && aligned16(p.w);
  const bool shifted = aligned16(p.gy) && alike(p.h, p.sh, p.sgy, p.rows, n) &&
                       alike(p.gsum, p.sgsum, p.sgy, p.rows, n) && alike(p.gx, p.sgx, p.sgy, p.rows, n);
  constexpr int64_t kMost = kMaxCluster * kMostVecs<T> * kClusterBlock;
  if (p.rows > 0 && vec && pieces <= kMost) return run_bwd_pieces<T, P, RMS, false>(p, pieces, st);
  if (p.rows > 0 && shifted && pieces < kMost) return run_bwd_pieces<T, P, RMS, true>(p, pieces + 1, st);  // one more
  p.chunks = bwd_chunks(p.rows);
  p.rows_per_chunk = (p.rows + p.chunks - 1) / p.chunks;
  p.pb = p.pw + p.chunks * p.H;
  if (p.gw || p.gb) {
    row_norm_bwd_cols_kernel<T, RMS><<<dim3((unsigned)((p.H + 31) / 32), (unsigned)p.chunks), kThreads, 0, st>>>(p);
    row_norm_bwd_finish_kernel<RMS><<<(unsigned)((p.H + 31) / 32), kFinishWarps * 32, 0, st>>>(p);
  }
  if (p.rows > 0) row_norm_bwd_rows_any_kernel<T, P, RMS><<<row_grid(p.rows), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

}  // namespace moe
