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
  uint32_t magic;  // Pair<T>::kMagic: as a run-time value it stays in a register, and mask-and-set is one instruction
  bool every;  // blockIdx.y is the expert; else it counts the experts that have rows
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
    asm(
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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// Codes (i, i + 4) of a word as two T's, less 16 + z: exactly q - z.
template <typename T>
MOE_DEVICE uint32_t code_pair(uint32_t w, int i, uint32_t magic, uint32_t zz) {
  const int s = Pair<T>::kShift - 4 * i;
  const uint32_t v = s >= 0 ? w << s : w >> -s;
  uint32_t b;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(v), "n"(Pair<T>::kMask), "r"(magic));  // (v & mask) | magic
  return Pair<T>::sub(b, zz);
}

template <typename T>
MOE_DEVICE uint32_t zero_pair(uint32_t z) {
  return Pair<T>::kMagic | z << Pair<T>::kShift | z << (16 + Pair<T>::kShift);
}

template <typename T>
MOE_DEVICE float scale_bits(uint16_t b) {
  return to_float(*reinterpret_cast<T*>(&b));
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

// A warp's tile of codes for one step: 32 weight rows x 128 k (64 bytes a row)
// in shared memory, 16-byte chunks exchanged by row so that the fragment reads
// of every group size touch each bank once.
constexpr int kStepK = 128;
constexpr int kRowBytes = kStepK / 2;
constexpr int kWarpRows = 32;
constexpr int kStageBytes = kWarpRows * kRowBytes;
constexpr int kStages = 6;

MOE_DEVICE int chunk_at(int row, int chunk) {
  return row * kRowBytes + ((chunk ^ ((row >> 1 & 1) << 1 | (row >> 2 & 1))) << 4);
}

MOE_DEVICE void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
MOE_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEVICE void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// GROUP: elements a scale; NT: tiles of 8 tokens a pass.  wk warps of a CTA
// share the K steps of the same 32 weight rows: neighbouring rows, or with
// SwiGLU the up and the gate rows of 16 features.
template <typename T, int GROUP, int NT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 2) w4_matvec_kernel(W4Params p, int wk) {
  constexpr int U = kStepK / GROUP;                    // groups a step
  constexpr int W = GROUP / 32;                        // 32-bit code words a lane takes of a group and row
  constexpr int kFeatures = SWIGLU ? 16 : kWarpRows;   // output features of a warp's rows
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int gr = lane >> 2, c = lane & 3;
  const int blocks = kWarps / wk;  // row blocks of a CTA
  const int64_t n_out = SWIGLU ? p.N / 2 : p.N;
  const int64_t cta_n0 = (int64_t)blockIdx.x * blocks * kFeatures;
  const int64_t n0 = cta_n0 + (warp / wk) * kFeatures;
  const int split = warp % wk;

  int64_t first = 0, M = p.M, e = 0;
  if (p.counts) {
    e = p.every ? (int)blockIdx.y : nth_active_expert(p, blockIdx.y);
    if (e < 0) return;
    first = p.offsets[e];
    M = min64(first + p.counts[e], p.cap) - first;
    if (M <= 0) return;
  }
  const uint8_t* codes = p.codes + e * p.N * (p.Kd / 2);
  const uint16_t* scales = static_cast<const uint16_t*>(p.scales) + e * p.N * p.G;
  const uint8_t* zeros = p.zeros ? p.zeros + e * p.N * p.zero_bytes : nullptr;
  const T* x = static_cast<const T*>(p.x) + first * p.sx;

  // Row r of the warp's tile is weight row n0 + r, with SwiGLU row n0 + r of the
  // up half and n0 + r - 16 of the gate half; rows past the end are read again
  // and not stored.  Lane (gr, c) copies chunk c of rows gr, gr + 8, ... and
  // holds the products of the same rows: offsets from the tile's first row.
  const int64_t last = n_out - 1 - n0;
  uint32_t rel[4];
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const int r = SWIGLU ? (q & 1) * 8 + gr : q * 8 + gr;
    rel[q] = (uint32_t)min64(r, last);
  }
  const uint32_t row_bytes = (uint32_t)(p.Kd / 2), G = (uint32_t)p.G, zero_bytes = (uint32_t)p.zero_bytes;
  const uint8_t* codes_at[2];
  const uint16_t* scales_at[2];
  const uint8_t* zeros_at[2];
#pragma unroll
  for (int rt = 0; rt < 2; rt++) {
    const int64_t r0 = n0 + (SWIGLU && rt ? n_out : 0);
    codes_at[rt] = codes + r0 * row_bytes;
    scales_at[rt] = scales + r0 * G;
    zeros_at[rt] = zeros ? zeros + r0 * zero_bytes : nullptr;
  }

  const uint32_t magic = p.magic;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  const uint32_t ring_u32 = (uint32_t)__cvta_generic_to_shared(ring);
  const int steps = (int)((p.Kd + kStepK - 1) / kStepK);
  const int mine = n0 < n_out && split < steps ? (steps - split + wk - 1) / wk : 0;

  auto fill = [&](int it, int stage) {
    if (it < mine) {
      const int step = split + it * wk;
      const bool in = (int64_t)step * kStepK + c * 32 < p.Kd;  // Kd is a multiple of 32, a chunk 32 elements
      const uint32_t dst = ring_u32 + stage * kStageBytes;
#pragma unroll
      for (int q = 0; q < 4; q++)
        cp_async16(dst + chunk_at(q * 8 + gr, c),
                   codes_at[q >> 1] + (in ? rel[q] * row_bytes + (uint32_t)(step * kRowBytes + c * 16) : 0u), in);
    }
    cp_async_commit();
  };

  for (int64_t t0 = 0; t0 < M; t0 += 8 * NT) {
    float acc[2][NT][4] = {};
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) fill(i, i);
    int stage = 0, free_stage = kStages - 1;
    for (int it = 0; it < mine; it++) {
      const int step = split + it * wk;
      // scales and zero points of this step, while its codes arrive
      uint16_t sc[4][U];
      uint8_t zp[4][U];
#pragma unroll
      for (int q = 0; q < 4; q++)
#pragma unroll
        for (int u = 0; u < U; u++) {
          const uint32_t g = step * U + u;
          sc[q][u] = g < G ? scales_at[q >> 1][rel[q] * G + g] : (uint16_t)0;
          zp[q][u] = zeros && g < G ? zeros_at[q >> 1][rel[q] * zero_bytes + g / 2] : (uint8_t)0x88;
        }
      cp_async_wait<kStages - 2>();
      __syncwarp();
      fill(it + kStages - 1, free_stage);  // the stage every lane has left
      const uint8_t* tile = ring + stage * kStageBytes;
      free_stage = stage;
      stage = stage + 1 == kStages ? 0 : stage + 1;
#pragma unroll
      for (int u = 0; u < U; u++) {
        uint32_t w[4][W], zz[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int r = q * 8 + gr;
          if (W == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(tile + chunk_at(r, c));
            w[q][0] = v.x, w[q][1 % W] = v.y, w[q][2 % W] = v.z, w[q][3 % W] = v.w;
          } else if (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(tile + chunk_at(r, 2 * u + (c >> 1)) + (c & 1) * 8);
            w[q][0] = v.x, w[q][1 % W] = v.y;
          } else {
            w[q][0] = *reinterpret_cast<const uint32_t*>(tile + chunk_at(r, u) + c * 4);
          }
          zz[q] = zero_pair<T>(zp[q][u] >> (4 * ((step * U + u) & 1)) & 15u);
        }
        const int k = (step * U + u) * GROUP + c * (GROUP / 4);
        float part[2][NT][4] = {};
#pragma unroll
        for (int j = 0; j < W; j++) {
          uint32_t a[2][2][4];
#pragma unroll
          for (int rt = 0; rt < 2; rt++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
              // fragment order: row gr, row gr + 8, then both again at the next pair
              a[rt][i >> 1][(i & 1) * 2] = code_pair<T>(w[2 * rt][j], i, magic, zz[2 * rt]);
              a[rt][i >> 1][(i & 1) * 2 + 1] = code_pair<T>(w[2 * rt + 1][j], i, magic, zz[2 * rt + 1]);
            }
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            if (nt > 0 && t0 + nt * 8 >= M) break;  // the same for the whole CTA
            const int64_t tok = t0 + nt * 8 + gr;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (k < p.Kd && tok < M) v = *reinterpret_cast<const uint4*>(x + tok * p.sx + k + j * 8);
            const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
            const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
            for (int rt = 0; rt < 2; rt++) {
              Pair<T>::mma(part[rt][nt], a[rt][0], b0, b1);
              Pair<T>::mma(part[rt][nt], a[rt][1], b2, b3);
            }
          }
        }
#pragma unroll
        for (int rt = 0; rt < 2; rt++)
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int i = 0; i < 4; i++)
              acc[rt][nt][i] = fmaf(scale_bits<T>(sc[2 * rt + (i >> 1)][u]), part[rt][nt][i], acc[rt][nt][i]);
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // partial tiles through the warps' rings: [tile][token][row]
    constexpr int kTile = NT * 8 * kTokStride;
    static_assert(2 * kTile * (int)sizeof(float) <= kStages * kStageBytes, "a partial tile fits the ring");
    float* red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int rt = 0; rt < 2; rt++)
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          red[rt * kTile + (nt * 8 + 2 * c + (i & 1)) * kTokStride + gr + 8 * (i >> 1)] = acc[rt][nt][i];
    __syncthreads();
    const int features = blocks * kFeatures;
    const int toks = (int)min64(M - t0, 8 * NT);
    for (int i = threadIdx.x; i < features * toks; i += kThreads) {
      const int f = i % features, tt = i / features, r = f % kFeatures;
      const int64_t n = cta_n0 + f, tok = t0 + tt;
      if (n >= n_out) continue;
      const float* base = reinterpret_cast<const float*>(smem + (f / kFeatures) * wk * (kStages * kStageBytes));
      auto total = [&](int rt) {
        const float* at = base + rt * kTile + tt * kTokStride + (r & 15);
        float v = at[0];
        for (int k = 1; k < wk; k++) v += at[k * (kStages * kStageBytes / 4)];
        return v;
      };
      float o;
      if (SWIGLU) {
        const float gate = total(1);
        o = gate / (1.0f + expf(-gate)) * total(0);
      } else {
        o = total(r >> 4);
      }
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

template <typename T, int GROUP, int NT, bool SWIGLU>
cudaError_t launch(const W4Params& p, int wk, dim3 grid, cudaStream_t st) {
  constexpr int kSmem = kWarps * kStages * kStageBytes;
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(w4_matvec_kernel<T, GROUP, NT, SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem);
  });
  if (e != cudaSuccess) return e;
  w4_matvec_kernel<T, GROUP, NT, SWIGLU><<<grid, kThreads, kSmem, st>>>(p, wk);
  return cudaGetLastError();
}

template <typename T, int GROUP, int NT>
cudaError_t run_act(const W4Params& p, bool swiglu, int wk, dim3 grid, cudaStream_t st) {
  return swiglu ? launch<T, GROUP, NT, true>(p, wk, grid, st) : launch<T, GROUP, NT, false>(p, wk, grid, st);
}

template <typename T, int GROUP>
cudaError_t run_nt(const W4Params& p, int64_t tokens, bool swiglu, int wk, dim3 grid, cudaStream_t st) {
  if (tokens <= 8) return run_act<T, GROUP, 1>(p, swiglu, wk, grid, st);
  if (tokens <= 16) return run_act<T, GROUP, 2>(p, swiglu, wk, grid, st);
  return run_act<T, GROUP, 4>(p, swiglu, wk, grid, st);
}

template <typename T>
cudaError_t run_group(const W4Params& p, int group, int64_t tokens, bool swiglu, int wk, dim3 grid, cudaStream_t st) {
  switch (group) {
    case 32: return run_nt<T, 32>(p, tokens, swiglu, wk, grid, st);
    case 64: return run_nt<T, 64>(p, tokens, swiglu, wk, grid, st);
    default: return run_nt<T, 128>(p, tokens, swiglu, wk, grid, st);
  }
}

W4Params base_params(const moe_w4& w, const moe_rows& x, const moe_rows& y) {
  W4Params p = {};
  p.codes = static_cast<const uint8_t*>(w.codes);
  p.scales = w.scales;
  p.zeros = static_cast<const uint8_t*>(w.zeros);
  p.magic = w.dtype == MOE_ELEM_BF16 ? Pair<__nv_bfloat16>::kMagic : Pair<__half>::kMagic;
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

// tokens: the rows a matrix is expected to meet; matrices: those that have rows
cudaError_t run(const moe_w4& w, const W4Params& p, int64_t tokens, int64_t matrices, int32_t activation,
                cudaStream_t st) {
  const bool swiglu = activation == MOE_W4_SWIGLU;
  const int64_t blocks = (w.N + kWarpRows - 1) / kWarpRows;  // row blocks of a matrix
  const int64_t want = (int64_t)device_sm_count() * 2 * kWarps;  // warps that fill the device
  int wk = 1;
  while (wk < kWarps && blocks * matrices * wk < want) wk *= 2;
  const dim3 grid((unsigned)((blocks * wk + kWarps - 1) / kWarps), (unsigned)matrices);
  return w.dtype == MOE_ELEM_BF16 ? run_group<__nv_bfloat16>(p, w.group, tokens, swiglu, wk, grid, st)
                                  : run_group<__half>(p, w.group, tokens, swiglu, wk, grid, st);
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
  p.every = routes >= s.E;
  // a token's routes go to different experts, so an expert has at most T rows
  const int64_t mean_rows = (routes + s.E - 1) / s.E;
  return run(w, p, s.T <= 8 ? s.T : mean_rows <= 12 ? 16 : s.T, routes < s.E ? routes : s.E, activation, st);
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
