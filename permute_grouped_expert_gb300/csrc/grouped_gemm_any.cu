// grouped_gemm_any.cu -- products grouped by expert for rows and matrices of any
// size, stride and alignment: element loads into shared memory, register-operand
// tensor products (mma.sync m16n8k16, fp32 sums), masked element stores.
//
// A CTA takes 64 x 64 output tiles in turn and runs along the contraction 32 at a
// time, its next operands on their way in registers meanwhile.  Loads bound it:
// 32 two-byte loads a thread for 64 x 64 x 32 products.
#include "block_common.cuh"
#include "grouped_gemm.cuh"

namespace moe {

namespace {

constexpr int kThreads = 128, TILE = 64, BK = 32, LD = BK + 8;  // LD: fragments without bank conflicts
constexpr int kMaxE = 1024;

template <typename T>
MOE_DEVICE void mma_16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]);
template <>
MOE_DEVICE void mma_16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <>
MOE_DEVICE void mma_16816<__half>(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// A TILE x BK operand in registers: 16-bit patterns, zeros outside [mn] x [k].
// KMAJOR: element (i, k) at src[i * ld + k], else at src[k * ld + i].
template <bool KMAJOR>
MOE_DEVICE void fetch(uint16_t (&v)[TILE * BK / kThreads], const uint16_t* src, int64_t ld, int64_t mn, int64_t k) {
#pragma unroll
  for (int j = 0; j < TILE * BK / kThreads; j++) {
    const int at = threadIdx.x + j * kThreads;
    const int i = KMAJOR ? at / BK : at % TILE, c = KMAJOR ? at % BK : at / TILE;
    v[j] = 0;
    if (i < mn && c < k) v[j] = src[KMAJOR ? i * ld + c : c * ld + i];
  }
}

template <bool KMAJOR>
MOE_DEVICE void put(uint16_t (*dst)[LD], const uint16_t (&v)[TILE * BK / kThreads]) {
#pragma unroll
  for (int j = 0; j < TILE * BK / kThreads; j++) {
    const int at = threadIdx.x + j * kThreads;
    dst[KMAJOR ? at / BK : at % TILE][KMAJOR ? at % BK : at / TILE] = v[j];
  }
}

template <typename T, typename OUT, GemmDir DIR>
__global__ void __launch_bounds__(kThreads) grouped_gemm_any_kernel(GroupedGemm p) {
  __shared__ uint16_t s_a[TILE][LD], s_b[TILE][LD];
  __shared__ int s_prefix[kMaxE + 1];  // row tiles of the experts before
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = (int)p.E;
  auto seg = [&](int e, int64_t& beg, int64_t& end) { gemm_segment(p.offsets, p.counts, p.cap, e, beg, end); };
  int64_t total;
  const int64_t nt = ((DIR == kForward ? p.N : p.Kd) + TILE - 1) / TILE;
  const int64_t mt = (p.N + TILE - 1) / TILE;  // kWeight
  if (DIR == kWeight) {
    total = E * mt * nt;
  } else {
    if (warp == 0) {
      int base = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int m = 0;
        if (e < E) {
          int64_t b, n;
          seg(e, b, n);
          m = n > b ? (int)((n - b + TILE - 1) / TILE) : 0;
        }
        int incl = m;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        if (e < E) s_prefix[e] = base + incl - m;
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) s_prefix[E] = base;
    }
    __syncthreads();
    total = s_prefix[E] * nt;
  }
  const uint16_t* pa = static_cast<const uint16_t*>(p.a);
  const uint16_t* pb = static_cast<const uint16_t*>(p.b);
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    int e;
    int64_t m0, n0 = (t % nt) * TILE, beg, end, m, n, k;  // sizes of the tile and of the contraction
    const uint16_t *a, *b;
    if (DIR == kWeight) {
      e = (int)(t / (mt * nt));
      m0 = t / nt % mt * TILE;
      seg(e, beg, end);
      a = pa + beg * p.sa + m0;
      b = pb + beg * p.sb + n0;
      m = p.N - m0;
      n = p.Kd - n0;
      k = max64(end - beg, 0);
    } else {
      const int mtile = (int)(t / nt);
      e = expert_of_row(s_prefix, E, mtile);
      m0 = (int64_t)(mtile - s_prefix[e]) * TILE;
      seg(e, beg, end);
      a = pa + (beg + m0) * p.sa;
      const uint16_t* w = pb + (int64_t)e * p.N * p.Kd;
      b = DIR == kForward ? w + n0 * p.Kd : w + n0;
      m = end - beg - m0;
      n = (DIR == kForward ? p.N : p.Kd) - n0;
      k = DIR == kForward ? p.Kd : p.N;
    }
    constexpr bool kA = DIR != kWeight, kB = DIR == kForward;
    const int64_t lda = p.sa, ldb = DIR == kWeight ? p.sb : p.Kd;
    const int64_t step_a = kA ? BK : BK * lda, step_b = kB ? BK : BK * ldb;
    float acc[2][4][4] = {};
    uint16_t va[TILE * BK / kThreads], vb[TILE * BK / kThreads];
    const int wm = (warp >> 1) * 32, wn = (warp & 1) * 32, g = lane >> 2, q = (lane & 3) * 2;
    fetch<kA>(va, a, lda, m, k);
    fetch<kB>(vb, b, ldb, n, k);
    for (int64_t k0 = 0; k0 < k; k0 += BK) {
      __syncthreads();
      put<kA>(s_a, va);
      put<kB>(s_b, vb);
      __syncthreads();
      a += step_a;
      b += step_b;
      if (k0 + BK < k) {
        fetch<kA>(va, a, lda, m, k - k0 - BK);
        fetch<kB>(vb, b, ldb, n, k - k0 - BK);
      }
#pragma unroll
      for (int ks = 0; ks < BK; ks += 16) {
        uint32_t fa[2][4], fb[4][2];
        auto word = [&](const uint16_t* s) { return *reinterpret_cast<const uint32_t*>(s); };
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int r = wm + i * 16 + g;
          fa[i][0] = word(&s_a[r][ks + q]);
          fa[i][1] = word(&s_a[r + 8][ks + q]);
          fa[i][2] = word(&s_a[r][ks + q + 8]);
          fa[i][3] = word(&s_a[r + 8][ks + q + 8]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
          fb[j][0] = word(&s_b[wn + j * 8 + g][ks + q]);
          fb[j][1] = word(&s_b[wn + j * 8 + g][ks + q + 8]);
        }
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) mma_16816<T>(acc[i][j], fa[i], fb[j]);
      }
    }
    OUT* out = static_cast<OUT*>(p.out) +
               (DIR == kWeight ? (int64_t)e * p.N * p.Kd + m0 * p.Kd : (beg + m0) * p.sout) + n0;
    const int64_t ldo = DIR == kWeight ? p.Kd : p.sout;
    const float* add = DIR == kWeight && p.addend ? p.addend + (int64_t)e * p.N * p.Kd + m0 * p.Kd + n0 : nullptr;
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int x = 0; x < 4; x++) {
          const int r = wm + i * 16 + g + (x >> 1) * 8, c = wn + j * 8 + q + (x & 1);
          if (r >= m || c >= n) continue;
          const float v = add ? acc[i][j][x] + add[r * ldo + c] : acc[i][j][x];
          out[r * ldo + c] = from_float<OUT>(v);
        }
  }
}

template <typename T>
cudaError_t run(GemmDir dir, const GroupedGemm& g, cudaStream_t st) {
  const int64_t most = (int64_t)device_sm_count() * 8;
  const int64_t nt = ((dir == kForward ? g.N : g.Kd) + TILE - 1) / TILE;
  const int64_t rt = dir == kWeight ? g.E * ((g.N + TILE - 1) / TILE) : g.cap / TILE + g.E;
  const unsigned grid = (unsigned)(rt * nt < most ? rt * nt : most);
  if (dir == kForward)
    grouped_gemm_any_kernel<T, T, kForward><<<grid, kThreads, 0, st>>>(g);
  else if (dir == kData)
    grouped_gemm_any_kernel<T, T, kData><<<grid, kThreads, 0, st>>>(g);
  else if (g.out_dtype == MOE_ELEM_F32)
    grouped_gemm_any_kernel<T, float, kWeight><<<grid, kThreads, 0, st>>>(g);
  else
    grouped_gemm_any_kernel<T, T, kWeight><<<grid, kThreads, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_gemm_any(GemmDir dir, const GroupedGemm& g, cudaStream_t st) {
  return g.dtype == MOE_ELEM_BF16 ? run<__nv_bfloat16>(dir, g, st) : run<__half>(dir, g, st);
}

}  // namespace moe
