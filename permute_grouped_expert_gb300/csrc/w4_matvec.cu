// w4_matvec.cu -- matrix-vector products with 4-bit weights and group scales:
// one matrix for a few tokens, or one matrix per expert over dispatched rows;
// and the quantizer that makes such weights.
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
// and added up in fp32.  A token with an infinity or a NaN gives NaN.
//
// A warp takes 32 weight rows (with SwiGLU the up and the gate rows of 16
// features) whose codes stream through its own ring in shared memory.  Where
// rows are few the CTAs of a cluster share the K steps of the same rows, so that
// each stages its part of the tokens only, and then the warps of a CTA; partial
// sums meet in (distributed) shared memory in a fixed order.
#include "block_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantWarps = kQuantThreads / 32;
constexpr int kMaxCluster = 8;
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
  bool vector_scales, vector_zeros;  // eight groups of any row are one aligned 16-byte / 4-byte piece
  // one matrix per expert
  const int32_t* counts;
  const int32_t* offsets;
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
MOE_DEVICE int nth_active_expert(const W4Params& p, int a) {
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
// Scales and zero points stream with the codes, eight groups of the 32 rows at
// a time (16 and 4 bytes a row), into slots enough for the steps in flight.
constexpr int kSlotBytes = kWarpRows * (16 + 4);
__host__ __device__ constexpr int scale_slots(int group) { return group == 128 ? 2 : 4; }
// Staged tokens: per step and token 128 f16 and, for each group, the sum of
// what they hold and the factor that undoes their scaling.
// How a CTA shares an SM (host and device).
template <int GROUP, int NT>
struct Plan {
  static constexpr int kWarps = NT == 1 ? 8 : 16, kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 1 ? 3 : 1;  // CTAs of an SM
  static constexpr int kStages = NT == 1 ? 3 : 5;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kSlots = scale_slots(GROUP);
  static constexpr int kSmemBytes = 228 * 1024 / kCtas / 128 * 128 - 1024 - 128;  // less what the system and statics take
  static constexpr int kTokenBytes = kSmemBytes - kWarps * (kRingBytes + kSlots * kSlotBytes);
  // steps of `toks` tokens that fit
  static MOE_DEVICE int chunk(int toks) {
    return kTokenBytes / (toks * kStepK * 2 + (toks + 1) / 2 * 2 * (kStepK / GROUP) * 8);
  }
  static_assert(kTokenBytes >= 8 * NT * (kStepK * 2 + kStepK / GROUP * 8), "a pass makes progress");
};

MOE_DEVICE int chunk_at(int row, int chunk) {
  return row * kRowBytes + ((chunk ^ ((row >> 1 & 1) << 1 | (row >> 2 & 1))) << 4);
}

MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
MOE_DEVICE void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
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
      // 2^(14 - E) for top in [2^E, 2^(E+1)); E held where both it and its inverse are normal
      const int E = top > 0.0f ? min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127) : 14;
      const float up = __uint_as_float((uint32_t)(127 + 14 - E) << 23);
      const float up16 = up * 0.0625f;
      __half2 h[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float m = i & 1 ? up16 : up;
        h[i] = __floats2half2_rn(f[i] * m, f[i + 4] * m);
      }
      float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
      for (int d = GROUP / 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (s0 + s < s1) {
        frag[(s * toks + tok) * 16 + frag_at(tok, j, c)] = *reinterpret_cast<uint4*>(h);
        if (k8 % (GROUP / 8) == 0)
          aux[(s * U + k8 / (GROUP / 8)) * even + tok] =
              make_float2(sum * (up * 0x1p-24f), __uint_as_float((uint32_t)(127 + 12 - 14 + E) << 23));
      }
      s += ds;
      tok += dt;
      if (tok >= toks) tok -= toks, s++;
    }
  }
}

MOE_DEVICE void cluster_barrier() {
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
template <typename T, int GROUP, int NT, bool SWIGLU>
__global__ void __launch_bounds__(Plan<GROUP, NT>::kThreads, Plan<GROUP, NT>::kCtas) w4_matvec_kernel(W4Params p, int ck) {
  constexpr int U = kStepK / GROUP;                    // groups a step
  constexpr int W = GROUP / 32;                        // 32-bit code words a lane takes of a group and row
  constexpr int kFeatures = SWIGLU ? 16 : kWarpRows;   // output features of a warp's rows
  using P = Plan<GROUP, NT>;
  constexpr int kWarps = P::kWarps, kThreads = P::kThreads, kSlots = P::kSlots, kStages = P::kStages, kRingBytes = P::kRingBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int gr = lane >> 2, c = lane & 3;
  const int64_t n_out = SWIGLU ? p.N / 2 : p.N;
  const int rank = blockIdx.x % ck;  // clusters lie along x
  const int64_t cta_n0 = (int64_t)(blockIdx.x / ck) * kWarps * kFeatures;
  const int64_t n0 = cta_n0 + warp * kFeatures;

  int64_t first = 0, M = p.M, e = 0;
  if (p.counts) {
    // (a shuffle tells the compiler that the expert is the whole warp's)
    e = __shfl_sync(0xffffffffu, p.every ? (int)blockIdx.y : nth_active_expert(p, blockIdx.y), 0);
    if (e < 0) return;
    first = p.offsets[e];
    M = min64(first + p.counts[e], p.cap) - first;
    if (M <= 0) return;
  }
  const uint8_t* codes = p.codes + e * p.N * (p.Kd / 2);
  const uint16_t* scales = static_cast<const uint16_t*>(p.scales) + e * p.N * p.G;
  const uint8_t* zeros = p.zeros ? p.zeros + e * p.N * p.zero_bytes : nullptr;
  const T* x = static_cast<const T*>(p.x) + first * p.sx;

  uint8_t* ring = smem + warp * kRingBytes;
  uint8_t* slots = smem + kWarps * kRingBytes + warp * kSlots * kSlotBytes;
  uint4* frag = reinterpret_cast<uint4*>(smem + kWarps * (kRingBytes + kSlots * kSlotBytes));
  const uint32_t ring_u32 = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t slots_u32 = (uint32_t)__cvta_generic_to_shared(slots);
  const int all_steps = (int)((p.Kd + kStepK - 1) / kStepK), run = (all_steps + ck - 1) / ck;
  const int begin = min(rank * run, all_steps), end = min(begin + run, all_steps);  // this CTA's steps
  const int mine = n0 < n_out ? end : begin;                                      // this warp's end

  // Row r of the warp's tile is weight row n0 + r, with SwiGLU row n0 + r of the
  // up half and n0 + r - 16 of the gate half.  Lane (gr, c) copies chunk c of
  // rows gr + 8 q and holds the products of the same rows.  A row past the last
  // (its products are not stored) reads the last.  Addresses are a base of the
  // whole warp, which moves with the steps, and a lane's 32-bit offset.
  const uint32_t row_bytes = (uint32_t)(p.Kd / 2), G = (uint32_t)p.G, zero_bytes = (uint32_t)p.zero_bytes;
  const uint8_t* codes_at[2];
  const uint16_t* scales_at[2];
  const uint8_t* zeros_at[2];
#pragma unroll
  for (int rt = 0; rt < 2; rt++) {
    const int64_t r0 = n0 + (SWIGLU && rt ? n_out : 0);
    codes_at[rt] = codes + r0 * row_bytes;
    scales_at[rt] = scales + r0 * G;
    zeros_at[rt] = zeros + r0 * zero_bytes;
  }
  uint32_t code_to[4];
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const uint32_t r = (uint32_t)min64(SWIGLU ? (q & 1) * 8 + gr : q * 8 + gr, max64(n_out - 1 - n0, 0));
    code_to[q] = r * row_bytes + c * 16;
  }
  // this lane's row of scales and zero points
  const uint32_t srow = (uint32_t)min64(SWIGLU ? lane & 15 : lane, max64(n_out - 1 - n0, 0));
  const uint16_t* scale_src = scales_at[SWIGLU ? lane >> 4 : 0] + srow * G;
  const uint8_t* zero_src = zeros_at[SWIGLU ? lane >> 4 : 0] + srow * zero_bytes;
  const int at0 = chunk_at(gr, c);  // rows gr + 8 q lie 8 q rows further

  auto fill = [&](int step, int stage) {
    if (step < mine) {
      // Kd is a multiple of 32, a chunk 32 elements; what a chunk past the end holds meets zeros
      if (c * 32 < (int)p.Kd - step * kStepK) {
        const uint32_t dst = ring_u32 + stage * kStageBytes + at0;
#pragma unroll
        for (int q = 0; q < 4; q++)
          cp_async16(dst + q * 8 * kRowBytes, codes_at[SWIGLU ? q >> 1 : 0] + (int64_t)step * kRowBytes + code_to[q]);
      }
      if (step == begin || step * U % 8 == 0) {
        const uint32_t g0 = step * U & ~7, slot = (g0 >> 3) % kSlots * kSlotBytes;
        if (p.vector_scales) {
          cp_async16(slots_u32 + slot + lane * 16, scale_src + g0);
        } else {
          uint16_t* to = reinterpret_cast<uint16_t*>(slots + slot + lane * 16);
          for (int i = 0; i < 8; i++) to[i] = g0 + i < G ? scale_src[g0 + i] : (uint16_t)0;
        }
        if (zeros) {
          if (p.vector_zeros) {
            cp_async4(slots_u32 + slot + kWarpRows * 16 + lane * 4, zero_src + (g0 >> 1));
          } else {
            uint8_t* to = slots + slot + kWarpRows * 16 + lane * 4;
            for (int i = 0; i < 4; i++) to[i] = (g0 >> 1) + i < zero_bytes ? zero_src[(g0 >> 1) + i] : (uint8_t)0;
          }
        }
      }
    }
    cp_async_commit();
  };

  for (int64_t t0 = 0; t0 < M; t0 += 8 * NT) {
    const int toks = (int)min64(M - t0, 8 * NT), even = (toks + 1) & ~1;
    const int chunk = min(P::chunk(toks), run);
    float2* aux = reinterpret_cast<float2*>(frag + chunk * toks * 16);
    float acc[2][NT][4] = {};
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) fill(begin + i, i);
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
      const uint8_t* tokens = reinterpret_cast<const uint8_t*>(frag);
      const uint8_t* sums = reinterpret_cast<const uint8_t*>(aux);
      for (int step = s0; step < min(s1, mine); step++) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        fill(step + kStages - 1, free_stage);  // the stage every lane has left
        const uint8_t* tile = ring + stage * kStageBytes;
        free_stage = stage;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const uint8_t* slot = slots + (step * U >> 3) % kSlots * kSlotBytes;
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int g = (step * U + u) & 7;
          float s[4], z[4];
#pragma unroll
          for (int q = 0; q < 4; q++) {
            s[q] = scale_bits<T>(*reinterpret_cast<const uint16_t*>(slot + (gr + 8 * q) * 16 + g * 2));
            z[q] = 8.0f;
          }
          if (zeros)
#pragma unroll
            for (int q = 0; q < 4; q++)
              z[q] = small_float(slot[kWarpRows * 16 + (gr + 8 * q) * 4 + (g >> 1)] >> (4 * (g & 1)) & 15u);
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

    // partial tiles through the warps' rings: [tile][token][row]
    constexpr int kTile = NT * 8 * kTokStride;
    static_assert(2 * kTile * (int)sizeof(float) <= kRingBytes, "a partial tile fits the ring");
    float* red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int rt = 0; rt < 2; rt++)
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          red[rt * kTile + (nt * 8 + 2 * c + (i & 1)) * kTokStride + gr + 8 * (i >> 1)] =
              acc[rt][nt][i] * 0x1p12f;  // with the staged factor 2^12 / f: 2^24 / f
    // every CTA of the cluster finishes a share of the outputs
    constexpr int kCtaFeatures = kWarps * kFeatures;
    if (ck > 1)
      cluster_barrier();
    else
      __syncthreads();
    for (int i = rank * kThreads + threadIdx.x; i < kCtaFeatures * toks; i += ck * kThreads) {
      const int f = i % kCtaFeatures, tt = i / kCtaFeatures, r = f % kFeatures;
      const int64_t n = cta_n0 + f, tok = t0 + tt;
      if (n >= n_out) continue;
      const float* base = reinterpret_cast<const float*>(smem + (f / kFeatures) * kRingBytes);
      auto total = [&](int rt) {
        const float* at = base + rt * kTile + tt * kTokStride + (r & 15);
        float part[kMaxCluster], v = 0.0f;
#pragma unroll
        for (int q = 0; q < kMaxCluster; q++)  // in flight together
          if (q < ck) part[q] = ck > 1 ? ld_cluster(at, q) : *at;
#pragma unroll
        for (int q = 0; q < kMaxCluster; q++)
          if (q < ck) v += part[q];
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
    if (ck > 1)
      cluster_barrier();  // nobody leaves, or fills its ring again, while it is read
    else
      __syncthreads();
  }
}

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

template <typename T, int GROUP, int NT, bool SWIGLU>
cudaError_t launch(const W4Params& p, int64_t matrices, cudaStream_t st) {
  using P = Plan<GROUP, NT>;
  cudaLaunchAttribute cluster = {};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kSmemBytes;
  cfg.attrs = &cluster;

  // clusters of each size that run at once: a cluster stays within one group of
  // SMs, so that some sizes leave SMs empty
  static PerDeviceOnce once;
  static int at_once[PerDeviceOnce::kMaxDevices][kMaxCluster + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run([&] {
    cudaError_t r = cudaFuncSetAttribute(w4_matvec_kernel<T, GROUP, NT, SWIGLU>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmemBytes);
    cfg.numAttrs = 1;
    for (int k = 1; k <= kMaxCluster && r == cudaSuccess; k++) {
      cluster.val.clusterDim.x = (unsigned)k;
      cfg.gridDim = dim3((unsigned)k);
      r = cudaOccupancyMaxActiveClusters(&at_once[dev][k], w4_matvec_kernel<T, GROUP, NT, SWIGLU>, &cfg);
    }
    return r;
  });
  if (e != cudaSuccess) return e;
  // CTAs that share a row's K: as many as shorten the longest chain of steps,
  // counting what a CTA spends around its steps as kOverhead of them
  constexpr int64_t kOverhead = 8;
  const int64_t ctas = (p.N + kWarpRows * P::kWarps - 1) / (kWarpRows * P::kWarps), steps = (p.Kd + kStepK - 1) / kStepK;
  int ck = 1;
  int64_t best = 0;
  for (int k = 1; k <= kMaxCluster && k <= steps; k++) {
    if (at_once[dev][k] < 1) continue;
    const int64_t cost =
        (ctas * matrices + at_once[dev][k] - 1) / at_once[dev][k] * ((steps + k - 1) / k + kOverhead);
    if (k == 1 || cost < best) best = cost, ck = k;
  }
  cluster.val.clusterDim.x = (unsigned)ck;
  cfg.gridDim = dim3((unsigned)(ctas * ck), (unsigned)matrices);
  cfg.stream = st;
  cfg.numAttrs = ck > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, w4_matvec_kernel<T, GROUP, NT, SWIGLU>, p, ck);
}

template <typename T, int GROUP, int NT>
cudaError_t run_act(const W4Params& p, bool swiglu, int64_t matrices, cudaStream_t st) {
  return swiglu ? launch<T, GROUP, NT, true>(p, matrices, st) : launch<T, GROUP, NT, false>(p, matrices, st);
}

template <typename T, int GROUP>
cudaError_t run_nt(const W4Params& p, int64_t tokens, bool swiglu, int64_t matrices, cudaStream_t st) {
  if (tokens <= 8) return run_act<T, GROUP, 1>(p, swiglu, matrices, st);
  if (tokens <= 16) return run_act<T, GROUP, 2>(p, swiglu, matrices, st);
  return run_act<T, GROUP, 4>(p, swiglu, matrices, st);
}

template <typename T>
cudaError_t run_group(const W4Params& p, int group, int64_t tokens, bool swiglu, int64_t matrices, cudaStream_t st) {
  switch (group) {
    case 32: return run_nt<T, 32>(p, tokens, swiglu, matrices, st);
    case 64: return run_nt<T, 64>(p, tokens, swiglu, matrices, st);
    default: return run_nt<T, 128>(p, tokens, swiglu, matrices, st);
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
  p.vector_scales = p.G % 8 == 0 && (reinterpret_cast<uintptr_t>(w.scales) & 15) == 0;
  p.vector_zeros = p.zero_bytes % 4 == 0 && (reinterpret_cast<uintptr_t>(w.zeros) & 3) == 0;
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
  return w.dtype == MOE_ELEM_BF16 ? run_group<__nv_bfloat16>(p, w.group, tokens, swiglu, matrices, st)
                                  : run_group<__half>(p, w.group, tokens, swiglu, matrices, st);
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
  // a pass holds twice the mean rows of an expert: few experts need a second
  const int64_t mean_rows = (routes + s.E - 1) / s.E;
  return run(w, p, s.T < 2 * mean_rows ? s.T : 2 * mean_rows, routes < s.E ? routes : s.E, activation, st);
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
