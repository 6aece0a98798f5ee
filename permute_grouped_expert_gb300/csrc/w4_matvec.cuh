// w4_matvec.cuh -- matrix-vector products with 4-bit weights and group scales:
// one matrix for a few tokens, or one matrix per expert over dispatched rows.
//
//   y[m][n] = act( sum_k (q[n][k] - z[n][k / group]) scale[n][k / group] x[m][k] )
//
// The products are m16n8k16 tensor-core products of 16 weight rows with 8
// tokens, f16 operands and fp32 sums.  What bounds them is not the tensor cores
// but the instructions that make operands of nibbles, so a nibble is used where
// it lies: masked out of a word at bits 0-3 of a half it reads as the
// subnormal q 2^-24, at bits 4-7 as q 2^-20, both exact, which is five
// instructions for a word of eight codes.  The factor 16 between them, and the
// order that two masks give (codes i and i + 4 of a word form a pair), are put
// on the tokens' side once: the CTA stages the tokens in fragment order, each
// 128 elements of a token multiplied by the power of two that brings their
// largest to [2^14, 2^15).  An element keeps all its bits down to 2^-24 of the
// largest, and below that errs by 2^-35 of it.  With f that factor,
//   sum (q - z) x = (sum q 2^-24 f x - z sum 2^-24 f x) 2^24 / f
// whose second sum is staged with the tokens; a group's difference is scaled
// and added up in fp32.  Codes thus enter uncentred, and the tensor cores may cut
// where fp32 rounds: the error is relative to sum |q x|, not sum |(q - z) x|, a
// few 1e-7 of it.  It moves 3 to 5 bf16 outputs in 10000 by a step (2048
// elements, groups of 128) and their error to 64 bits, 0.0017, in no digit.  A token with an
// infinity or a NaN gives outputs that are not finite.
//
// A warp takes 32 weight rows (with SwiGLU the up and the gate rows of 16
// features) whose codes stream through its own ring in shared memory.  Where
// rows are few the CTAs of a cluster share the K steps of the same rows, so that
// each stages its part of the tokens only, and then the warps of a CTA; partial
// sums meet in (distributed) shared memory in a fixed order.
//
// Device times on one GB300, bf16 tokens and groups of 128 (share of the HBM
// floor, the weights' bytes at a copy's 6793 GB/s):
//   one token, 4096 x 7168 SwiGLU      10.6 us, 20 %   8192 x 8192   11.6 us, 44 %
//              32768 x 8192            30.4 us, 67 %
//   16 / 32 tokens, 8192 x 8192        18.6 / 31.6 us  32 tokens, 32768 x 8192   89 us, 23 %
//   64 tokens top-8 through 256 experts of 4096 x 7168 SwiGLU   625 us, 80 %
// Few rows are bound by the launch, the staging and one pass of the ring (a copy of
// the same 15 MB takes 6.4 us); long streams of few tokens by HBM; from 16 tokens
// on by the chains of operand reads and products, which keep the tensor cores 40 %
// busy with the 16 warps an SM that registers allow.
#pragma once

#include "block_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace w4 {

constexpr int kMaxCluster = 8;
constexpr int kTokStride = 20;  // floats between tokens of a partial tile: conflict-free fragment stores

struct Params {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  int64_t N, Kd, G, zero_bytes;
  int64_t n_out;      // output features
  int64_t gate;       // rows from a tile's first 16 rows to its second: N / 2 with SwiGLU, else 16
  bool swiglu;
  const void* x;
  int64_t sx;
  const void* addend;
  int64_t sadd;
  void* y;
  int64_t sy;
  int64_t M;          // tokens, without experts
  int64_t matrices;   // that codes, scales and zeros hold
  // one matrix per expert
  const int32_t* counts;
  const int32_t* offsets;
  int32_t* status;  // of the handle
  int E;
  bool every;  // blockIdx.y is the expert; else it counts the experts that have rows
  int64_t cap;
};

MOE_DEVICE void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with sums that start at zero.
MOE_DEVICE void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// The integer 0..15 as a float.
MOE_DEVICE float small_float(uint32_t v) { return __uint_as_float(0x4B000000u | v) - 8388608.0f; }

template <typename T>
MOE_DEVICE float scale_bits(uint16_t b) {
  return to_float(*reinterpret_cast<T*>(&b));
}

// The a-th expert with rows below the capacity, or -1; every thread calls it.
MOE_DEVICE int nth_active_expert(const Params& p, int a) {
  __shared__ unsigned words[32];
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.E; base += (int)blockDim.x) {
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

// How a CTA shares an SM.  ALIGNED: eight groups of any row are 16 aligned
// bytes of scales and 4 of zero points.  Scales and zero points stream with the
// codes, eight groups of the 32 rows at a time, as the aligned pieces that hold
// them (two at the most), into slots enough for the steps in flight.  The rest
// holds staged tokens: per step and token 128 f16 and, for each group, the sum
// of what they hold and the factor that undoes their scaling.
template <int GROUP, int NT, int WARPS, int KSPLIT, bool ALIGNED>
struct Plan {
  static constexpr int kGroups = kStepK / GROUP;  // groups of a step
  static constexpr int kWarps = WARPS, kThreads = 32 * kWarps;
  static constexpr int kRowBlocks = WARPS / KSPLIT;  // tiles of 32 rows of a CTA; KSPLIT warps share the steps of one
  static constexpr int kCtas = WARPS == 8 ? (NT == 1 ? 3 : 2) : 1;  // CTAs of an SM
  static constexpr int kStages = kCtas == 3 ? 3 : 4;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kScalePitch = ALIGNED ? 16 : 32, kZeroPitch = ALIGNED ? 4 : 8;
  static constexpr int kSlotBytes = kWarpRows * (kScalePitch + kZeroPitch);
  static constexpr int kSlotSteps = 8 / kGroups;
  static constexpr int kSlots = (kStages - 1 + kSlotSteps - 1) / kSlotSteps + 1;
  static constexpr int kWarpBytes = kRingBytes + kSlots * kSlotBytes;
  static constexpr int kSmemBytes = 228 * 1024 / kCtas / 128 * 128 - 1024 - 128;  // less what the system and statics take
  static constexpr int kTokenBytes = kSmemBytes - kWarps * kWarpBytes;
  // steps of `toks` tokens that fit
  static __host__ __device__ int chunk(int toks) {
    return kTokenBytes / (toks * kStepK * 2 + (toks + 1) / 2 * 2 * kGroups * 8);
  }
  static_assert(kTokenBytes >= 8 * NT * (kStepK * 2 + kGroups * 8), "a pass of any size makes progress");
  // a warp's partial tiles, [2][token][row], take its ring's place
  static constexpr int kTile = NT * 8 * kTokStride;
  static_assert(2 * kTile * (int)sizeof(float) <= kRingBytes, "partial tiles fit the ring");
};

MOE_DEVICE int chunk_at(int row, int chunk) {
  return row * kRowBytes + ((chunk ^ ((row >> 1 & 1) << 1 | (row >> 2 & 1))) << 4);
}

MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of the piece, zeros behind them.
MOE_DEVICE void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MOE_DEVICE void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MOE_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEVICE void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where lane-of-quad c of a token finds the tokens' 16 bytes for code word j of
// a step, from the step's and token's 256 bytes: the words of odd tokens change
// places in pairs, so that a quarter-warp's read of two tokens meets every bank
// once.
MOE_DEVICE int frag_at(int tok, int j, int c) { return (j ^ (tok & 1)) * 4 + c; }

// Stages steps [s0, s1) of `toks` tokens (x: the first of them).  Half a warp
// takes a token's step, eight elements a lane.  frag: 16 bytes at
// (step * toks + token) * 16 + frag_at: the pairs (0, 4), (1, 5) / 16, (2, 6),
// (3, 7) / 16 of the eight k of that code word.  aux: {sum, factor} at
// (step * groups + group) * even(toks) + token.
template <typename T, int GROUP, int kThreads>
MOE_DEVICE void stage_tokens(const T* x, int64_t sx, int64_t Kd, int toks, int s0, int s1, uint4* frag, float2* aux) {
  constexpr int U = kStepK / GROUP;
  constexpr int kBatch = 4;  // units a half-warp has in flight
  constexpr int kHalves = kThreads / 16;
  const int k8 = threadIdx.x & 15;
  const int j = GROUP == 128 ? k8 & 3 : GROUP == 64 ? (k8 >> 3) * 2 + (k8 & 1) : k8 >> 2;
  const int c = GROUP == 128 ? k8 >> 2 : GROUP == 64 ? k8 >> 1 & 3 : k8 & 3;
  const int even = (toks + 1) & ~1;
  const int rounds = ((s1 - s0) * toks + kHalves - 1) / kHalves;
  const int ds = kHalves / toks, dt = kHalves % toks;  // one round further
  int s = (threadIdx.x >> 4) / toks, tok = (threadIdx.x >> 4) % toks;
  for (int first = 0; first < rounds; first += kBatch) {  // every lane stays: shuffles below
    union {
      uint4 v;
      T e[8];
    } in[kBatch];
    int ss = s, tt = tok;
#pragma unroll
    for (int b = 0; b < kBatch; b++) {
      const int64_t k = (int64_t)(s0 + ss) * kStepK + k8 * 8;
      in[b].v = make_uint4(0, 0, 0, 0);
      if (s0 + ss < s1 && k < Kd) in[b].v = *reinterpret_cast<const uint4*>(x + tt * sx + k);
      ss += ds;
      tt += dt;
      if (tt >= toks) tt -= toks, ss++;
    }
#pragma unroll
    for (int b = 0; b < kBatch; b++) {
      if (first + b >= rounds) break;  // the same for the whole CTA
      float f[8], top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        f[i] = to_float(in[b].e[i]);
        top = fmaxf(top, fabsf(f[i]));
      }
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      // 2^(14 - E) for top in [2^E, 2^(E+1)); E held where both it and its inverse are
      // normal (below 2^-100 every bf16, a multiple of 2^-133, is still exact in f16)
      const int E = top > 0.0f ? min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127) : 14;
      const float up = __uint_as_float((uint32_t)(127 + 14 - E) << 23);
      const float up16 = up * 0.0625f;
      __half2 h[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float m = i & 1 ? up16 : up;
        h[i] = __floats2half2_rn(f[i] * m, f[i + 4] * m);
      }
      // of the scaled elements: a sum of large ones of one sign would leave fp32's range
      auto two = [&](int i) { return fmaf(f[i + 1], up, f[i] * up); };
      float sum = (two(0) + two(2)) + (two(4) + two(6));
#pragma unroll
      for (int d = GROUP / 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (s0 + s < s1) {
        frag[(s * toks + tok) * 16 + frag_at(tok, j, c)] = *reinterpret_cast<uint4*>(h);
        if (k8 % (GROUP / 8) == 0)
          aux[(s * U + k8 / (GROUP / 8)) * even + tok] =
              make_float2(sum * 0x1p-24f, __uint_as_float((uint32_t)(127 + 12 - 14 + E) << 23));
      }
      s += ds;
      tok += dt;
      if (tok >= toks) tok -= toks, s++;
    }
  }
}

MOE_DEVICE void cluster_barrier() {
  __syncwarp();  // lanes leave the loops before it at different rounds; the aligned form wants the whole warp
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The float at this CTA's shared address `at`, read from the CTA of this rank.
MOE_DEVICE float ld_cluster(const float* at, int rank) {
  uint32_t a;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// GROUP: elements a scale; NT: tiles of 8 tokens a pass.  A warp holds 32
// weight rows: neighbouring rows, or with SwiGLU the up and the gate rows of 16
// features.  The K steps of a row are shared by the ck CTAs of a cluster, a
// run of steps each.
template <typename T, int GROUP, int NT, int WARPS, int KSPLIT, bool ALIGNED>
__global__ void __launch_bounds__(Plan<GROUP, NT, WARPS, KSPLIT, ALIGNED>::kThreads,
                                  Plan<GROUP, NT, WARPS, KSPLIT, ALIGNED>::kCtas)
    matvec_kernel(Params p, int ck) {
  using P = Plan<GROUP, NT, WARPS, KSPLIT, ALIGNED>;
  constexpr int U = P::kGroups;
  constexpr int W = GROUP / 32;  // 32-bit code words a lane takes of a group and row
  constexpr int kWarps = P::kWarps, kThreads = P::kThreads, kStages = P::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int gr = lane >> 2, c = lane & 3;
  const int log_features = p.swiglu ? 4 : 5;  // output features of a warp's rows
  const int rank = blockIdx.x % ck;           // clusters lie along x
  const int64_t cta_n0 = (int64_t)(blockIdx.x / ck) * P::kRowBlocks << log_features;
  const int64_t n0 = cta_n0 + ((int64_t)(warp % P::kRowBlocks) << log_features);

  int64_t first = 0, M = p.M, e = 0;
  if (p.counts) {
    // (a shuffle tells the compiler that the expert is the whole warp's)
    e = __shfl_sync(0xffffffffu, p.every ? (int)blockIdx.y : nth_active_expert(p, blockIdx.y), 0);
    if (e < 0) return;
    first = p.offsets[e];
    M = min64(first + p.counts[e], p.cap) - first;
    // (a handle that no preprocess wrote may hold anything: rows stay within [0, cap))
    if (M <= 0 || !MOE_IN_BOUNDS(71, first, p.cap, p.status) || first < 0) return;
  }
  const T* x = static_cast<const T*>(p.x) + first * p.sx;

  uint8_t* ring = smem + warp * P::kRingBytes;
  uint8_t* slots = smem + kWarps * P::kRingBytes + warp * P::kSlots * P::kSlotBytes;
  uint4* frag = reinterpret_cast<uint4*>(smem + kWarps * P::kWarpBytes);
  const uint32_t ring_u32 = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t slots_u32 = (uint32_t)__cvta_generic_to_shared(slots);
  const int all_steps = (int)((p.Kd + kStepK - 1) / kStepK), run = (all_steps + ck - 1) / ck;
  const int begin = min(rank * run, all_steps), end = min(begin + run, all_steps);  // this CTA's steps
  const int part = (run + KSPLIT - 1) / KSPLIT;
  const int my_begin = min(begin + warp / P::kRowBlocks * part, end);               // this warp's
  const int mine = n0 < p.n_out ? min(my_begin + part, end) : my_begin;

  // Row r of the warp's tile is weight row n0 + r below 16, n0 + gate + r - 16
  // from there.  Lane (gr, c) copies chunk c of rows gr + 8 q and holds the
  // products of the same rows.  A row past the last output reads another (its
  // products are not stored).  Addresses are a base of the whole warp, which
  // moves with the steps, and a lane's 32-bit offset.
  const uint32_t row_bytes = (uint32_t)(p.Kd / 2), G = (uint32_t)p.G, zero_bytes = (uint32_t)p.zero_bytes;
  const int last = (int)min64(15, p.n_out - 1 - n0);                        // of the tile's first 16 rows
  const int last16 = p.swiglu ? last : (int)min64(15, p.n_out - 17 - n0);  // of the second, below 0 if there is none
  const int64_t row0 = e * p.N + n0, row16 = row0 + (last16 < 0 ? 0 : p.gate);
  const uint8_t* codes_at[2] = {p.codes + row0 * row_bytes, p.codes + row16 * row_bytes};
  uint32_t code_to[4];
#pragma unroll
  for (int q = 0; q < 4; q++)
    code_to[q] = (uint32_t)max(min((q & 1) * 8 + gr, q < 2 ? last : last16), 0) * row_bytes + c * 16;
  const int at0 = chunk_at(gr, c);  // rows gr + 8 q lie 8 q rows further

  auto fill_codes = [&](int step, int stage) {
    // Kd is a multiple of 32, a chunk 32 elements; what a chunk past the end holds meets zeros
    if (step < mine && c * 32 < (int)p.Kd - step * kStepK) {
      const uint32_t dst = ring_u32 + stage * kStageBytes + at0;
#pragma unroll
      for (int q = 0; q < 4; q++)
        cp_async16(dst + q * 8 * kRowBytes, codes_at[q >> 1] + (int64_t)step * kRowBytes + code_to[q]);
    }
  };
  // the eight groups that begin with this step's, where it is the first to need them
  auto fill_scales = [&](int step) {
    if (step >= mine || (step != my_begin && step * U % 8 != 0)) return;
    // this lane's row
    const int64_t row = lane < 16 ? row0 + min(lane, max(last, 0)) : row16 + max(min(lane & 15, last16), 0);
    const int64_t scale_row = row * G, zero_row = row * zero_bytes;
    const uint32_t g0 = step * U & ~7;
    const uint32_t to = slots_u32 + (g0 >> 3) % P::kSlots * P::kSlotBytes + lane * P::kScalePitch;
    const uint32_t zto =
        slots_u32 + (g0 >> 3) % P::kSlots * P::kSlotBytes + kWarpRows * P::kScalePitch + lane * P::kZeroPitch;
    if (ALIGNED) {
      cp_async16(to, p.scales + scale_row + g0, 16);
      if (p.zeros) cp_async4(zto, p.zeros + zero_row + (g0 >> 1), 4);
    } else {
      // aligned pieces; the last of the array may be short
      const int64_t at = (scale_row + g0) * 2, total = p.matrices * p.N * p.G * 2;
      const int off = (int)(at & 15);
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.scales) + (at - off);
      cp_async16(to, src, (int)min64(16, total - (at - off)));
      if (off && g0 + (16 - off) / 2 < G) cp_async16(to + 16, src + 16, (int)min64(16, total - (at - off) - 16));
      if (p.zeros) {
        const int64_t zat = zero_row + (g0 >> 1), ztotal = p.matrices * p.N * p.zero_bytes;
        const int zoff = (int)(zat & 3);
        const uint8_t* zsrc = p.zeros + (zat - zoff);
        cp_async4(zto, zsrc, (int)min64(4, ztotal - (zat - zoff)));
        if (zoff && (g0 >> 1) + 4 - zoff < zero_bytes)
          cp_async4(zto + 4, zsrc + 4, (int)min64(4, ztotal - (zat - zoff) - 4));
      }
    }
  };
  // Where a lane's rows find their scales and zero points in a slot: rows 8
  // apart start at the same place of an aligned piece.
  int scale_to[2], zero_to[2];
#pragma unroll
  for (int rt = 0; rt < 2; rt++) {
    const int64_t r = (rt ? row16 : row0) + gr;
    scale_to[rt] = (gr + 16 * rt) * P::kScalePitch + (ALIGNED ? 0 : (int)(r * p.G * 2 & 15));
    zero_to[rt] = kWarpRows * P::kScalePitch + (gr + 16 * rt) * P::kZeroPitch +
                  (ALIGNED ? 0 : (int)(r * p.zero_bytes & 3));
  }

  for (int64_t t0 = 0; t0 < M; t0 += 8 * NT) {
    const int toks = (int)min64(M - t0, 8 * NT), even = (toks + 1) & ~1;
    const int chunk = min(P::chunk(toks), run);
    float2* aux = reinterpret_cast<float2*>(frag + chunk * toks * 16);
    float acc[2][NT][4] = {};
    // the first scales belong to the first group of copies
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) fill_scales(my_begin + i);
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) {
      fill_codes(my_begin + i, i);
      cp_async_commit();
    }
    // a lane's tokens in a staged step: words of even and of odd index, see frag_at
    uint32_t tok_to[NT][2], sum_to[NT];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const int tok = min(nt * 8 + gr, toks - 1);  // columns past the last token are not stored
      tok_to[nt][0] = tok * 256 + frag_at(tok, 0, c) * 16;
      tok_to[nt][1] = tok * 256 + frag_at(tok, 1, c) * 16;
      sum_to[nt] = min(nt * 8 + 2 * c, even - 2) * 8;
    }
    int stage = 0, free_stage = kStages - 1;
    for (int s0 = begin; s0 < end; s0 += chunk) {
      const int s1 = min(s0 + chunk, end);
      if (s0 > begin) __syncthreads();  // the last chunk has been read
      stage_tokens<T, GROUP, kThreads>(x + t0 * p.sx, p.sx, p.Kd, toks, s0, s1, frag, aux);
      __syncthreads();
      // (with KSPLIT the launch sees to it that one chunk holds all of the CTA's steps)
      const int from = KSPLIT == 1 ? s0 : my_begin;
      const uint8_t* tokens = reinterpret_cast<const uint8_t*>(frag) + (from - s0) * toks * 256;
      const uint8_t* sums = reinterpret_cast<const uint8_t*>(aux) + (from - s0) * U * even * 8;
      for (int step = from; step < min(s1, mine); step++) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        fill_codes(step + kStages - 1, free_stage);  // the stage every lane has left
        fill_scales(step + kStages - 1);
        cp_async_commit();
        __syncwarp();  // lanes may have copied less than others; the products want the whole warp
        const uint8_t* tile = ring + stage * kStageBytes;
        free_stage = stage;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const uint8_t* slot = slots + (step * U >> 3) % P::kSlots * P::kSlotBytes;
#pragma unroll
        for (int u = 0; u < U; u++) {
          uint32_t w[4][W];
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const uint8_t* t = tile + q * 8 * kRowBytes;
            if (W == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(t + at0);
              w[q][0] = v.x, w[q][1 % W] = v.y, w[q][2 % W] = v.z, w[q][3 % W] = v.w;
            } else if (W == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(t + chunk_at(gr, 2 * u + (c >> 1)) + (c & 1) * 8);
              w[q][0] = v.x, w[q][1 % W] = v.y;
            } else {
              w[q][0] = *reinterpret_cast<const uint32_t*>(t + chunk_at(gr, u) + c * 4);
            }
          }
          float part[2][NT][4];
#pragma unroll
          for (int j = 0; j < W; j++) {
            // fragment order: row gr, row gr + 8, then both again at the next pair
            uint32_t a[2][2][4];
#pragma unroll
            for (int rt = 0; rt < 2; rt++)
#pragma unroll
              for (int h = 0; h < 2; h++) {
                const uint32_t v = w[2 * rt + h][j], v8 = v >> 8;
                a[rt][0][h] = v & 0x000F000Fu;
                a[rt][0][2 + h] = v & 0x00F000F0u;
                a[rt][1][h] = v8 & 0x000F000Fu;
                a[rt][1][2 + h] = v8 & 0x00F000F0u;
              }
            const int word = u * W + j;
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              if (nt > 0 && nt * 8 >= toks) break;  // the same for the whole CTA
              const uint4 b = *reinterpret_cast<const uint4*>(tokens + tok_to[nt][word & 1] + (word & 2) * 64);
#pragma unroll
              for (int rt = 0; rt < 2; rt++) {
                if (j == 0)
                  mma_f16_first(part[rt][nt], a[rt][0], b.x, b.y);
                else
                  mma_f16(part[rt][nt], a[rt][0], b.x, b.y);
                mma_f16(part[rt][nt], a[rt][1], b.z, b.w);
              }
            }
          }
          const int g = (step * U + u) & 7;
          float s[4], z[4];
#pragma unroll
          for (int q = 0; q < 4; q++) {
            s[q] = scale_bits<T>(*reinterpret_cast<const uint16_t*>(slot + scale_to[q >> 1] +
                                                                    (q & 1) * 8 * P::kScalePitch + g * 2));
            // a group past the end: its place in the slot was not filled
            if (!ALIGNED && U > 1 && step * U + u >= (int)G) s[q] = 0.0f;
            z[q] = 8.0f;
          }
          if (p.zeros)
#pragma unroll
            for (int q = 0; q < 4; q++)
              z[q] = small_float(slot[zero_to[q >> 1] + (q & 1) * 8 * P::kZeroPitch + (g >> 1)] >> (4 * (g & 1)) & 15u);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            if (nt > 0 && nt * 8 >= toks) break;
            // {sum, factor} of tokens 2 c and 2 c + 1
            const float4 xs = *reinterpret_cast<const float4*>(sums + u * even * 8 + sum_to[nt]);
#pragma unroll
            for (int rt = 0; rt < 2; rt++)
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int q = 2 * rt + (i >> 1);
                const float v = fmaf(-z[q], i & 1 ? xs.z : xs.x, part[rt][nt][i]) * (i & 1 ? xs.w : xs.y);
                acc[rt][nt][i] = fmaf(s[q], v, acc[rt][nt][i]);
              }
          }
        }
        tokens += toks * 256;
        sums += U * even * 8;
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    float* red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int rt = 0; rt < 2; rt++)
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          red[rt * P::kTile + (nt * 8 + 2 * c + (i & 1)) * kTokStride + gr + 8 * (i >> 1)] =
              acc[rt][nt][i] * 0x1p12f;  // with the staged factor 2^12 / f: 2^24 / f
    // every CTA of the cluster finishes a share of the outputs
    const int features = P::kRowBlocks << log_features, log_cta = 31 - __clz(features);
    if (ck > 1)
      cluster_barrier();
    else
      __syncthreads();
    for (int i = rank * kThreads + threadIdx.x; i < features * toks; i += ck * kThreads) {
      const int f = i & (features - 1), tt = i >> log_cta, r = f & ((1 << log_features) - 1);
      const int64_t n = cta_n0 + f, tok = t0 + tt;
      if (n >= p.n_out) continue;
      const float* base = reinterpret_cast<const float*>(smem + (f >> log_features) * P::kRingBytes);
      auto total = [&](int rt) {
        const float* at = base + rt * P::kTile + tt * kTokStride + (r & 15);
        constexpr int kNext = P::kRowBlocks * P::kRingBytes / 4;  // to the next part of K
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < KSPLIT; k++) {
          if (ck == 1) {
            v += at[k * kNext];
          } else {
            float part[kMaxCluster];
#pragma unroll
            for (int q = 0; q < kMaxCluster; q++)  // in flight together
              if (q < ck) part[q] = ld_cluster(at + k * kNext, q);
#pragma unroll
            for (int q = 0; q < kMaxCluster; q++)
              if (q < ck) v += part[q];
          }
        }
        return v;
      };
      float o;
      if (p.swiglu) {
        const float gate = total(1);
        o = gate / (1.0f + expf(-gate)) * total(0);
      } else {
        o = total(r >> 4);
      }
      if (p.addend) o += to_float(static_cast<const T*>(p.addend)[(first + tok) * p.sadd + n]);
      static_cast<T*>(p.y)[(first + tok) * p.sy + n] = from_float<T>(o);
    }
    if (ck > 1)
      cluster_barrier();  // nobody leaves, or fills its ring again, while it is read
    else
      __syncthreads();
  }
}

// One kernel with its launch shape for a problem.
template <typename T, int GROUP, int NT, int WARPS, int KSPLIT, bool ALIGNED>
struct Launch {
  using P = Plan<GROUP, NT, WARPS, KSPLIT, ALIGNED>;
  cudaLaunchAttribute cluster = {};
  cudaLaunchConfig_t cfg = {};
  int ck = 1;        // CTAs that share a row's K
  int64_t cost = 0;  // length of the longest chain of steps

  // Clusters of each size that run at once, per device: a cluster stays within
  // one group of SMs, so that some sizes leave SMs empty.
  cudaError_t at_once(const int** out) {
    static PerDeviceOnce once;
    static int table[PerDeviceOnce::kMaxDevices][kMaxCluster + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once.run([&] {
      cudaError_t r = cudaFuncSetAttribute(matvec_kernel<T, GROUP, NT, WARPS, KSPLIT, ALIGNED>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmemBytes);
      cfg.numAttrs = 1;
      for (int k = 1; k <= kMaxCluster && r == cudaSuccess; k++) {
        cluster.val.clusterDim.x = (unsigned)k;
        cfg.gridDim = dim3((unsigned)k);
        r = cudaOccupancyMaxActiveClusters(&table[dev][k], matvec_kernel<T, GROUP, NT, WARPS, KSPLIT, ALIGNED>, &cfg);
      }
      return r;
    });
    *out = table[dev];
    return e;
  }

  cudaError_t plan(const Params& p, int64_t matrices) {
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.blockDim = dim3(P::kThreads);
    cfg.dynamicSmemBytes = P::kSmemBytes;
    cfg.attrs = &cluster;
    const int* slots;
    cudaError_t e = at_once(&slots);
    if (e != cudaSuccess) return e;
    // In twentieths of a step's time on a full SM: a step on an SM with that many
    // CTAs, each of which stages its tokens, and what a CTA spends around its steps.
    // Fitted to measured times; over 16 shapes (1 to 64 tokens, 1024 to 32768 rows, one
    // matrix to 256) against every kernel and cluster size: within 2 % of the fastest
    // but for 32 tokens of 2048 x 7168 (19.0 us, fastest 17.6), 13 of 1024 x 2048 (7.2,
    // 6.4) and one of 4096 x 7168 with SwiGLU (10.7, 9.9).
    constexpr int64_t kAround = 8 * 20, kAlone = NT == 1 ? 8 : 13;  // (few warps do not speed up in proportion)
    const int64_t rows = kWarpRows * P::kRowBlocks;
    const int64_t ctas = (p.N + rows - 1) / rows, sms = device_sm_count();
    const int64_t steps = (p.Kd + kStepK - 1) / kStepK;
    for (int k = 1; k <= kMaxCluster && k <= steps; k++) {
      const int64_t run = (steps + k - 1) / k;
      if (slots[k] < 1 || (KSPLIT > 1 && run > P::chunk(8 * NT))) continue;
      const int64_t clusters = ctas * matrices, waves = (clusters + slots[k] - 1) / slots[k];
      const int64_t on_sm = waves > 1 ? P::kCtas : (clusters * k + sms - 1) / sms;
      const int64_t step = (20 * on_sm / P::kCtas > kAlone ? 20 * on_sm / P::kCtas : kAlone) + (NT > 1 ? 3 * on_sm : 0);
      const int64_t c = waves * ((run + KSPLIT - 1) / KSPLIT * step + kAround);
      if (cost == 0 || c < cost) cost = c, ck = k;
    }
    if (cost == 0) cost = INT64_MAX;  // no way to run it
    cluster.val.clusterDim.x = (unsigned)ck;
    cfg.gridDim = dim3((unsigned)(ctas * ck), (unsigned)matrices);
    cfg.numAttrs = ck > 1 ? 1 : 0;
    return cudaSuccess;
  }

  cudaError_t run(const Params& p, cudaStream_t st) {
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, matvec_kernel<T, GROUP, NT, WARPS, KSPLIT, ALIGNED>, p, ck);
  }
};

// CTAs of 8 warps, several an SM, are the rule (64 tokens through 256 experts
// 625 us; 852 with 16 warps that share the steps).  CTAs of 16 warps stage more
// than eight tokens once for 512 weight rows where there are rows enough (32 tokens,
// 32768 x 8192: 89 us, 8 warps 102); where there are few CTAs, 16 warps halve the
// steps of each tile (13 tokens, 4099 x 8224: 18.6 us, 8 warps 21.7).  Each side at
// its best cluster size; the plan's cost decides.
template <typename T, int GROUP, int NT, bool ALIGNED>
cudaError_t launch(const Params& p, int64_t matrices, cudaStream_t st) {
  Launch<T, GROUP, NT, 8, 1, ALIGNED> small;
  cudaError_t e = small.plan(p, matrices);
  if (e != cudaSuccess) return e;
  Launch<T, GROUP, NT, 16, 2, ALIGNED> split;
  e = split.plan(p, matrices);
  if (e != cudaSuccess) return e;
  if constexpr (NT > 1) {
    Launch<T, GROUP, NT, 16, 1, ALIGNED> large;
    e = large.plan(p, matrices);
    if (e != cudaSuccess) return e;
    if (large.cost <= small.cost && large.cost <= split.cost) return large.run(p, st);
  }
  return split.cost < small.cost ? split.run(p, st) : small.run(p, st);
}

template <typename T, bool ALIGNED, int GROUP>
cudaError_t run_tokens(const Params& p, int64_t tokens, int64_t matrices, cudaStream_t st) {
  if (tokens <= 8) return launch<T, GROUP, 1, ALIGNED>(p, matrices, st);
  if (tokens <= 16) return launch<T, GROUP, 2, ALIGNED>(p, matrices, st);
  return launch<T, GROUP, 4, ALIGNED>(p, matrices, st);
}

// tokens: the rows a matrix is expected to meet; matrices: those that have rows.
// Instantiated in one translation unit per type and alignment.
template <typename T, bool ALIGNED>
cudaError_t run(const Params& p, int group, int64_t tokens, int64_t matrices, cudaStream_t st) {
  switch (group) {
    case 32: return run_tokens<T, ALIGNED, 32>(p, tokens, matrices, st);
    case 64: return run_tokens<T, ALIGNED, 64>(p, tokens, matrices, st);
    default: return run_tokens<T, ALIGNED, 128>(p, tokens, matrices, st);
  }
}

}  // namespace w4

}  // namespace moe
