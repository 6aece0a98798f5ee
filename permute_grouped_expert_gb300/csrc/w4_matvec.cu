// w4_matvec.cu -- matrix-vector products with 4-bit weights and group scales:
// one matrix for a few tokens, or one matrix per expert over dispatched rows;
// and the quantizer that makes such weights.
//
//   y[m][n] = act( sum_k (q[n][k] - z[n][k / group]) scale[n][k / group] x[m][k] )
//
// The products are m16n8k16 tensor-core products of 16 weight rows with 8
// tokens.  A nibble becomes a 16-bit float without a conversion: placed in the
// top mantissa bits of a number whose exponent is 2^4 it reads 16 + q, and
// 16 + z is taken off exactly, so both operands are exact and a group's sum
// is rounded in fp32 only; its scale is applied to that sum in fp32.  A sum over
// k may take k in any order, so a lane's eight nibbles of one 32-bit word form
// the pairs (i, i + 4) that two masks give at once, and the token values are
// paired the same way.
//
// A CTA takes 16 output features (with SwiGLU the up and the gate rows of 16)
// and its warps share the groups of K; partial sums meet in shared memory in
// warp order.
#include "block_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokStride = 20;  // floats between tokens of a partial tile: conflict-free fragment stores

struct W4Params {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  int64_t N, Kd, G, zero_bytes;
  const void* x;
  int64_t sx;
  const void* addend;
  int64_t sadd;
  void* y;
  int64_t sy;
  int64_t M;  // tokens, without experts
  // one matrix per expert
  const int32_t* counts;
  const int32_t* offsets;
  int E;
  int64_t cap;
};

template <typename T>
struct Pair;  // how 4-bit codes become pairs of T

template <>
struct Pair<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x41804180u, kMask = 0x00780078u;
  static constexpr int kShift = 3;  // bits below a nibble in the mantissa
  static MOE_DEVICE uint32_t sub(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
  }
  static MOE_DEVICE void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

template <>
struct Pair<__half> {
  static constexpr uint32_t kMagic = 0x4C004C00u, kMask = 0x03C003C0u;
  static constexpr int kShift = 6;
  static MOE_DEVICE uint32_t sub(uint32_t a, uint32_t b) {
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
  }
  static MOE_DEVICE void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// Codes (i, i + 4) of a word as two T's, less 16 + z: exactly q - z.
template <typename T>
MOE_DEVICE uint32_t code_pair(uint32_t w, int i, uint32_t zz) {
  const int s = Pair<T>::kShift - 4 * i;
  const uint32_t v = s >= 0 ? w << s : w >> -s;
  return Pair<T>::sub((v & Pair<T>::kMask) | Pair<T>::kMagic, zz);
}

template <typename T>
MOE_DEVICE uint32_t zero_pair(uint32_t z) {
  return Pair<T>::kMagic | z << Pair<T>::kShift | z << (16 + Pair<T>::kShift);
}

// The a-th expert with rows below the capacity, or -1; every thread calls it.
MOE_DEVICE int nth_active_expert(const W4Params& p, int a) {
  __shared__ unsigned words[32];
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.E; base += kThreads) {
    const int e = base + threadIdx.x;
    const bool on = e < p.E && p.counts[e] > 0 && p.offsets[e] < p.cap;
    const unsigned m = __ballot_sync(0xffffffffu, on);
    if (lane == 0) words[e >> 5] = m;
  }
  __syncthreads();
  const int nwords = (p.E + 31) >> 5;
  for (int i = 0; i < nwords; i++) {
    const unsigned m = words[i];
    const int n = __popc(m);
    if (a < n) return i * 32 + (int)__fns(m, 0, a + 1);
    a -= n;
  }
  return -1;
}

// GROUP: elements a scale; NT: tiles of 8 tokens a pass; RT: 2 with SwiGLU (up, gate)
template <typename T, int GROUP, int NT, int RT>
__global__ void __launch_bounds__(kThreads) w4_matvec_kernel(W4Params p) {
  constexpr int LK = GROUP / 4;  // k values a lane takes of a group, for each of its two rows
  constexpr int W = LK / 8;      // 32-bit words they fill
  __shared__ float red[kWarps][RT][NT * 8][kTokStride];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, c = lane & 3;
  const int64_t n_out = RT == 2 ? p.N / 2 : p.N;
  const int64_t n0 = (int64_t)blockIdx.x * 16;

  int64_t first = 0, M = p.M, e = 0;
  if (p.counts) {
    const int a = nth_active_expert(p, blockIdx.y);
    if (a < 0) return;
    e = a;
    first = p.offsets[a];
    M = min64(first + p.counts[a], p.cap) - first;
  }
  const uint8_t* codes = p.codes + e * p.N * (p.Kd / 2);
  const T* scales = static_cast<const T*>(p.scales) + e * p.N * p.G;
  const uint8_t* zeros = p.zeros ? p.zeros + e * p.N * p.zero_bytes : nullptr;
  const T* x = static_cast<const T*>(p.x) + first * p.sx;

  int64_t row[RT][2];
#pragma unroll
  for (int rt = 0; rt < RT; rt++)
#pragma unroll
    for (int h = 0; h < 2; h++) row[rt][h] = min64(n0 + gr + 8 * h, n_out - 1) + rt * n_out;  // past the end: unused

  for (int64_t t0 = 0; t0 < M; t0 += 8 * NT) {
    float acc[RT][NT][4] = {};
    for (int64_t g = warp; g < p.G; g += kWarps) {
      const int64_t k = g * GROUP + c * LK;
      const bool in = k < p.Kd;  // the last group may be short by whole lanes
      uint32_t w[RT][2][W];
      float s[RT][2];
      uint32_t zz[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; rt++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(codes + (row[rt][h] * p.Kd + k) / 2);
#pragma unroll
          for (int j = 0; j < W; j++) w[rt][h][j] = in ? src[j] : 0u;
          s[rt][h] = to_float(scales[row[rt][h] * p.G + g]);
          const uint32_t z = zeros ? zeros[row[rt][h] * p.zero_bytes + g / 2] >> (4 * (g & 1)) & 15u : 8u;
          zz[rt][h] = zero_pair<T>(z);
        }
      float part[RT][NT][4] = {};
#pragma unroll
      for (int j = 0; j < W; j++) {
        uint32_t a[RT][2][4];
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            // fragment order: row gr, row gr + 8, then both again at the next pair
            a[rt][i >> 1][(i & 1) * 2] = code_pair<T>(w[rt][0][j], i, zz[rt][0]);
            a[rt][i >> 1][(i & 1) * 2 + 1] = code_pair<T>(w[rt][1][j], i, zz[rt][1]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          if (nt > 0 && t0 + nt * 8 >= M) break;  // the same for the whole CTA
          const int64_t tok = t0 + nt * 8 + gr;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (in && tok < M) v = *reinterpret_cast<const uint4*>(x + tok * p.sx + k + j * 8);
          const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
          const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
          for (int rt = 0; rt < RT; rt++) {
            Pair<T>::mma(part[rt][nt], a[rt][0], b0, b1);
            Pair<T>::mma(part[rt][nt], a[rt][1], b2, b3);
          }
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; rt++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int i = 0; i < 4; i++) acc[rt][nt][i] = fmaf(s[rt][i >> 1], part[rt][nt][i], acc[rt][nt][i]);
    }

#pragma unroll
    for (int rt = 0; rt < RT; rt++)
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int i = 0; i < 4; i++) red[warp][rt][nt * 8 + 2 * c + (i & 1)][gr + 8 * (i >> 1)] = acc[rt][nt][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += kThreads) {
      const int r = i & 15, tt = i >> 4;
      const int64_t tok = t0 + tt, n = n0 + r;
      if (tok >= M || n >= n_out) continue;
      float v[RT];
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
        v[rt] = red[0][rt][tt][r];
#pragma unroll
        for (int k = 1; k < kWarps; k++) v[rt] += red[k][rt][tt][r];
      }
      float o = v[0];
      if (RT == 2) o = v[RT - 1] / (1.0f + expf(-v[RT - 1])) * v[0];
      if (p.addend) o += to_float(static_cast<const T*>(p.addend)[(first + tok) * p.sadd + n]);
      static_cast<T*>(p.y)[(first + tok) * p.sy + n] = from_float<T>(o);
    }
    __syncthreads();
  }
}

// One warp per row and pair of groups (the two zero points of a byte).
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_w4_kernel(const T* w, int64_t R, int64_t Kd, int group, int64_t G,
                                                               uint8_t* codes, T* scales, uint8_t* zeros) {
  const int lane = threadIdx.x & 31;
  const int64_t pairs = (G + 1) / 2, items = R * pairs;
  for (int64_t it = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * kWarps) {
    const int64_t r = it / pairs, g0 = it % pairs * 2;
    uint32_t zbyte = 0;
    for (int64_t g = g0; g < g0 + 2 && g < G; g++) {
      const T* src = w + r * Kd + g * group;
      const int n = (int)min64(group, Kd - g * group);
      float lo = 0.0f, hi = 0.0f;
      for (int k = lane; k < n; k += 32) {
        const float v = to_float(src[k]);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
      }
      lo = -warp_max(-lo);
      hi = warp_max(hi);
      const float span = zeros ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
      T st = from_float<T>(span);
      if (to_float(st) == 0.0f) st = from_float<T>(1.0f);
      const float s = to_float(st);
      const float z = zeros ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f) : 8.0f;
      if (lane == 0) scales[r * G + g] = st;
      zbyte |= (uint32_t)z << (4 * (g - g0));
      for (int k = 2 * lane; k < n; k += 64) {
        uint32_t b = 0;
        for (int i = 0; i < 2; i++) {
          const float q = fminf(fmaxf(rintf(__fdiv_rn(to_float(src[k + i]), s)) + z, 0.0f), 15.0f);
          b |= (uint32_t)q << (4 * i);
        }
        codes[(r * Kd + g * group + k) / 2] = (uint8_t)b;
      }
    }
    if (zeros && lane == 0) zeros[r * pairs + g0 / 2] = (uint8_t)zbyte;
  }
}

template <typename T, int GROUP, int NT>
void run_rt(const W4Params& p, bool swiglu, dim3 grid, cudaStream_t st) {
  if (swiglu)
    w4_matvec_kernel<T, GROUP, NT, 2><<<grid, kThreads, 0, st>>>(p);
  else
    w4_matvec_kernel<T, GROUP, NT, 1><<<grid, kThreads, 0, st>>>(p);
}

template <typename T, int GROUP>
void run_nt(const W4Params& p, int64_t tokens, bool swiglu, dim3 grid, cudaStream_t st) {
  if (tokens <= 8)
    run_rt<T, GROUP, 1>(p, swiglu, grid, st);
  else if (tokens <= 16)
    run_rt<T, GROUP, 2>(p, swiglu, grid, st);
  else
    run_rt<T, GROUP, 4>(p, swiglu, grid, st);
}

template <typename T>
void run_group(const W4Params& p, int group, int64_t tokens, bool swiglu, dim3 grid, cudaStream_t st) {
  switch (group) {
    case 32: run_nt<T, 32>(p, tokens, swiglu, grid, st); break;
    case 64: run_nt<T, 64>(p, tokens, swiglu, grid, st); break;
    default: run_nt<T, 128>(p, tokens, swiglu, grid, st); break;
  }
}

W4Params base_params(const moe_w4& w, const moe_rows& x, const moe_rows& y) {
  W4Params p = {};
  p.codes = static_cast<const uint8_t*>(w.codes);
  p.scales = w.scales;
  p.zeros = static_cast<const uint8_t*>(w.zeros);
  p.N = w.N;
  p.Kd = w.Kd;
  p.G = (w.Kd + w.group - 1) / w.group;
  p.zero_bytes = (p.G + 1) / 2;
  p.x = x.data;
  p.sx = x.stride;
  p.y = y.data;
  p.sy = y.stride;
  return p;
}

// tokens: a bound on the rows of one matrix
cudaError_t run(const moe_w4& w, const W4Params& p, int64_t tokens, int64_t matrices, int32_t activation,
                cudaStream_t st) {
  const bool swiglu = activation == MOE_W4_SWIGLU;
  const int64_t n_out = swiglu ? w.N / 2 : w.N;
  const dim3 grid((unsigned)((n_out + 15) / 16), (unsigned)matrices);
  if (w.dtype == MOE_ELEM_BF16)
    run_group<__nv_bfloat16>(p, w.group, tokens, swiglu, grid, st);
  else
    run_group<__half>(p, w.group, tokens, swiglu, grid, st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_w4_matvec(const moe_w4& w, int64_t M, const moe_rows& x, int32_t activation,
                             const moe_rows* addend, const moe_rows& y, cudaStream_t st) {
  W4Params p = base_params(w, x, y);
  p.M = M;
  if (addend) p.addend = addend->data, p.sadd = addend->stride;
  return run(w, p, M, 1, activation, st);
}

cudaError_t launch_grouped_w4_matvec(const moe_handle_dev& h, const moe_shape& s, const moe_layout& l, const moe_w4& w,
                                     const moe_rows& x, int32_t activation, const moe_rows& y, cudaStream_t st) {
  W4Params p = base_params(w, x, y);
  p.counts = h.tokens_per_expert;
  p.offsets = h.padded_offsets;
  p.E = (int)s.E;
  p.cap = l.capacity;
  const int64_t routes = s.T * s.K;
  // a token's routes go to different experts, so an expert has at most T rows
  return run(w, p, s.T, routes < s.E ? routes : s.E, activation, st);
}

cudaError_t launch_quantize_w4_rows(const void* w, int64_t R, int64_t Kd, int32_t group, int32_t dtype, void* codes,
                                    void* scales, void* zeros, cudaStream_t st) {
  const int64_t G = (Kd + group - 1) / group, items = R * ((G + 1) / 2);
  const int64_t cap = (int64_t)device_sm_count() * (2048 / kThreads), blocks = (items + kWarps - 1) / kWarps;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  if (dtype == MOE_ELEM_BF16)
    quantize_w4_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(
        static_cast<const __nv_bfloat16*>(w), R, Kd, group, G, static_cast<uint8_t*>(codes),
        static_cast<__nv_bfloat16*>(scales), static_cast<uint8_t*>(zeros));
  else
    quantize_w4_kernel<__half><<<grid, kThreads, 0, st>>>(static_cast<const __half*>(w), R, Kd, group, G,
                                                          static_cast<uint8_t*>(codes), static_cast<__half*>(scales),
                                                          static_cast<uint8_t*>(zeros));
  return cudaGetLastError();
}

}  // namespace moe
