// w4_matvec.cu -- entry of the 4-bit matrix-vector products (w4_matvec.cuh) and
// the quantizer that makes such weights.
#include "w4_matvec.cuh"

namespace moe {

namespace w4 {
extern template cudaError_t run<__nv_bfloat16, true>(const Params&, int, int64_t, int64_t, cudaStream_t);
extern template cudaError_t run<__nv_bfloat16, false>(const Params&, int, int64_t, int64_t, cudaStream_t);
extern template cudaError_t run<__half, true>(const Params&, int, int64_t, int64_t, cudaStream_t);
extern template cudaError_t run<__half, false>(const Params&, int, int64_t, int64_t, cudaStream_t);
}  // namespace w4

namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantWarps = kQuantThreads / 32;

// One warp per row and pair of groups (the two zero points of a byte).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_w4_kernel(const T* w, int64_t R, int64_t Kd, int group, int64_t G,
                                                               uint8_t* codes, T* scales, uint8_t* zeros) {
  const int lane = threadIdx.x & 31;
  const int64_t pairs = (G + 1) / 2, items = R * pairs;
  for (int64_t it = (int64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * kQuantWarps) {
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

w4::Params params(const moe_w4& w, int64_t matrices, const moe_rows& x, int32_t activation, const moe_rows& y) {
  w4::Params p = {};
  p.codes = static_cast<const uint8_t*>(w.codes);
  p.scales = static_cast<const uint16_t*>(w.scales);
  p.zeros = static_cast<const uint8_t*>(w.zeros);
  p.N = w.N;
  p.Kd = w.Kd;
  p.G = (w.Kd + w.group - 1) / w.group;
  p.zero_bytes = (p.G + 1) / 2;
  p.swiglu = activation == MOE_W4_SWIGLU;
  p.n_out = p.swiglu ? w.N / 2 : w.N;
  p.gate = p.swiglu ? w.N / 2 : 16;
  p.x = x.data;
  p.sx = x.stride;
  p.y = y.data;
  p.sy = y.stride;
  p.matrices = matrices;
  return p;
}

cudaError_t run(const moe_w4& w, const w4::Params& p, int64_t tokens, int64_t matrices, cudaStream_t st) {
  const bool bf16 = w.dtype == MOE_ELEM_BF16;
  // eight groups of scales are 16 aligned bytes, their zero points 4 (64 tokens through
  // 256 experts of 4096 x 7168: 626 us, as pieces that may straddle 664)
  if (p.G % 8 == 0)
    return bf16 ? w4::run<__nv_bfloat16, true>(p, w.group, tokens, matrices, st)
                : w4::run<__half, true>(p, w.group, tokens, matrices, st);
  return bf16 ? w4::run<__nv_bfloat16, false>(p, w.group, tokens, matrices, st)
              : w4::run<__half, false>(p, w.group, tokens, matrices, st);
}

}  // namespace

cudaError_t launch_w4_matvec(const moe_w4& w, int64_t M, const moe_rows& x, int32_t activation,
                             const moe_rows* addend, const moe_rows& y, cudaStream_t st) {
  w4::Params p = params(w, 1, x, activation, y);
  p.M = M;
  if (addend) p.addend = addend->data, p.sadd = addend->stride;
  return run(w, p, M, 1, st);
}

cudaError_t launch_grouped_w4_matvec(const moe_handle_dev& h, const moe_shape& s, const moe_layout& l, const moe_w4& w,
                                     const moe_rows& x, int32_t activation, const moe_rows& y, cudaStream_t st) {
  w4::Params p = params(w, s.E, x, activation, y);
  p.counts = h.tokens_per_expert;
  p.offsets = h.padded_offsets;
  p.status = h.status;
  p.E = (int)s.E;
  p.cap = l.capacity;
  const int64_t routes = s.T * s.K;
  p.every = routes >= s.E;
  // a pass holds twice the mean rows of an expert: few experts need a second
  const int64_t mean_rows = (routes + s.E - 1) / s.E;
  return run(w, p, s.T < 2 * mean_rows ? s.T : 2 * mean_rows, routes < s.E ? routes : s.E, st);
}

cudaError_t launch_quantize_w4_rows(const void* w, int64_t R, int64_t Kd, int32_t group, int32_t dtype, void* codes,
                                    void* scales, void* zeros, cudaStream_t st) {
  const int64_t G = (Kd + group - 1) / group, items = R * ((G + 1) / 2);
  const int64_t cap = (int64_t)device_sm_count() * (2048 / kQuantThreads), blocks = (items + kQuantWarps - 1) / kQuantWarps;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  if (dtype == MOE_ELEM_BF16)
    quantize_w4_kernel<__nv_bfloat16><<<grid, kQuantThreads, 0, st>>>(
        static_cast<const __nv_bfloat16*>(w), R, Kd, group, G, static_cast<uint8_t*>(codes),
        static_cast<__nv_bfloat16*>(scales), static_cast<uint8_t*>(zeros));
  else
    quantize_w4_kernel<__half><<<grid, kQuantThreads, 0, st>>>(static_cast<const __half*>(w), R, Kd, group, G,
                                                          static_cast<uint8_t*>(codes), static_cast<__half*>(scales),
                                                          static_cast<uint8_t*>(zeros));
  return cudaGetLastError();
}

}  // namespace moe
