// router.cu -- top-k router of the MoE layer (logits -> routing map and
// probabilities) and the gradient of its logits.
//
// A group of L lanes takes a token, V neighbouring experts a lane (E <= V L), so
// that a warp works on 32 / L tokens at once.  The selection looks for a
// threshold that exactly K scores reach: it guesses one from the scores' mean and
// deviation, shrinks an interval by the counts, and stops at the first count
// that is K.  Where scores are equal no threshold may have that count; the
// interval then closes on one value by bisection of its bit pattern, everything
// above it is chosen and the lowest experts among those equal to it fill the
// rest.  Ids come out ascending.  Scores and sums are fp32 in a fixed order.
//
// The bytes are few (65536 x 256 fp32 logits: 10 us of HBM); what bounds both
// directions is instructions, and of the forward pass those of the pipe that
// compares: about 600 a warp for 256 experts, four to five counts among them.
// Hence no sort, no selection one by one, and one pass for the common case of
// finite logits.  Device times on one GB300:
//   65536 x 256 fp32 top-8 44 us, top-36 with the softmax over all 58 us;
//   65536 x 64 bf16 21 us; 16384 x 1024 top-32 32 us; 64 x 256 3.8 us
//   with a bias 65536 x 256 top-8 51 us, by sigmoids 64, softmax over all 54
//   gradient 65536 x 256 top-8 27 us (softmax over all 31), 8192 x 256 4.1 us
// The bias reads the chosen logits (softmax over all: the row) a second time.
// The gradient of 65536 tokens is bound by latency, 57 % of cycles without a warp
// that can issue: ids, the logits they point to, two sums, the row, a token after
// the other.
#include <cmath>
#include <type_traits>

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
  int renorm, format;
  bool vector_in, vector_out;  // rows of logits / of a sparse map are whole aligned vectors
  float scale;
  float quantile, spacing;  // of a standard normal sample of E, at the K-th largest
  const void* logits;
  const float* bias;
  void* map;
  float* probs;
  int32_t* status;
};

// Unsigned key in the order of the floats, and the float of a key.
MOE_DEVICE uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
MOE_DEVICE float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// exp(l - top) for l <= top, 1 where l is top (both may be infinite: the minimum
// drops a NaN).  What is below 2^-126 of the largest is 0.  The rounding of the
// product makes the relative error grow with the distance, to (top - l) 2^-24 and
// 2 ulp; expf would hold 2 ulp at several times the instructions.  Over the cases'
// logits the weights' error to 64 bits is 7e-8, that of a plain fp32 form 6e-8.
MOE_DEVICE float exp_below(float l, float top) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fminf(l - top, 0.0f) * 1.4426950408889634f));
  return e;
}

// sigmoid(l) * exp(-m) for m = min(largest l, 0): the common factor keeps the
// ratio of two sigmoids when both are far below the smallest float.  The quotients
// here are approximate ones, 2 ulp for these divisors of 1 to 2 (and for the sums
// of at most 1024 weights that they are divided by): they weigh, and do not choose.
MOE_DEVICE float sigmoid_scaled(float l, float m) {
  return __fdividef(l >= 0.0f ? 1.0f : expf(l - m), 1.0f + expf(-fabsf(l)));
}

// 1 - sigmoid(l)
MOE_DEVICE float sigmoid_rest(float l) {
  const float e = expf(-fabsf(l));
  return __fdividef(l < 0.0f ? 1.0f : e, 1.0f + e);
}

// Over the L lanes of a group.
template <int L>
MOE_DEVICE int group_add(int v) {
  if (L == 32) return __reduce_add_sync(kAll, v);
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <int L>
MOE_DEVICE float group_add(float v) {
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <int L>
MOE_DEVICE float group_max(float v) {
  if (L == 32) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
  }
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
// Two sums over the group; halves of a warp add one value each.
template <int L>
MOE_DEVICE void group_add2(float& a, float& b) {
  if (L == 32) {
    const bool lower = (threadIdx.x & 16) == 0;
    float v = (lower ? a : b) + __shfl_xor_sync(kAll, lower ? b : a, 16);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    a = __shfl_sync(kAll, v, 0);
    b = __shfl_sync(kAll, v, 16);
  } else {
    a = group_add<L>(a);
    b = group_add<L>(b);
  }
}
// Sum over the lanes of the group below this one.
template <int L>
MOE_DEVICE int group_below(int v) {
  const int lane = threadIdx.x % L;
  int s = v;
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    const int up = __shfl_up_sync(kAll, s, d, L);
    if (lane >= d) s += up;
  }
  return s - v;
}

// V values of a row as V / N vectors of N neighbours, the first at e0 and each
// `gap` after the one before; -inf past the row's end.
template <typename T, int V>
MOE_DEVICE void load_scores(float (&l)[V], const T* row, int e0, int gap, int E, bool vector) {
  constexpr int N = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < V; j += N) {
    const int e = e0 + j / N * gap;
    if (vector) {
      union {
        uint4 v;
        T e[N];
      } u;
      if (e < E) u.v = *reinterpret_cast<const uint4*>(row + e);
#pragma unroll
      for (int i = 0; i < N; i++) l[j + i] = e < E ? to_float(u.e[i]) : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < N; i++) l[j + i] = e + i < E ? to_float(row[e + i]) : -INFINITY;
    }
  }
}

// Counts in the low bits of a float: one comparison and one addition a score, of
// which only the comparison takes the pipe that bounds the kernel.
template <int V>
MOE_DEVICE int count_from(const float (&s)[V], float v) {
  float n[2] = {8388608.0f, 0.0f};  // 2^23
#pragma unroll
  for (int j = 0; j < V; j++) {
    float one;
    asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(one) : "f"(s[j]), "f"(v));
    n[j & 1] += one;
  }
  return __float_as_int(n[0] + n[1]) & 0x7fffff;
}

template <int V>
MOE_DEVICE uint32_t bits_from(const float (&s)[V], float v) {
  uint32_t on = 0;
#pragma unroll
  for (int j = 0; j < V; j++) on |= s[j] >= v ? 1u << j : 0u;
  return on;
}

// The score that the chosen reach, in `lo`; true where more than K scores of a
// token of the warp reach it, and `on` then tells every token's chosen: bit j,
// expert e0 + j.  `live` scores are above -inf; `low` and `top` are the smallest
// and the largest of them (+inf and -inf if there is none).
// `guess` is where the K-th score would be, and `step` how far a score is from
// the next there, if the scores were a normal sample: the first guess then
// counts K but for a few, and a step by the difference mostly lands on K.
// Whatever they are, the interval bounds the search.
template <int V, int L>
MOE_DEVICE bool select_top(const float (&s)[V], int K, int live, float low, float top, float guess, float step,
                           float& lo, uint32_t& on) {
  // counts: n_lo >= K scores reach lo, n_hi < K reach hi (hi is the top, and n_hi
  // 0, until there is a count below K); the choice is exact once a count is K
  lo = low;
  float hi = top;
  int n_lo = live, n_hi = 0;
  bool exact = live <= K, found = exact;
  // a token's lanes agree; other tokens of the warp go on
  auto all_found = [&] { return L == 32 ? found : (bool)__all_sync(kAll, found); };
  float mid = K == 1 ? top : fminf(guess, top);
  for (int it = 0; it < 12 && !all_found(); it++) {
    if (!(mid > lo && mid <= hi) || it > 4) {
      // the place of the K-th score if those between the ends were spread evenly
      const float part = __fdividef((float)(K - n_hi) + 0.5f, (float)(n_lo - n_hi + 1));
      mid = hi - (hi - lo) * fminf(fmaxf(part, 0.0625f), 0.9375f);
    }
    const int n = group_add<L>(count_from<V>(s, mid));
    if ((L == 32 || !found) && mid > lo && mid <= hi) {
      if (n >= K)
        lo = mid, n_lo = n, exact = n == K;
      else
        hi = mid, n_hi = n;
      found = exact || lo == top;  // (equal to the top, and not all of them fit)
    }
    mid += (float)(n - K) * step;
  }
  if (!all_found()) {  // equal, infinite or very uneven scores
    uint32_t klo = key_of(lo), khi = key_of(hi) + (n_hi == 0);
    if (found) khi = klo + 1;
    while (__any_sync(kAll, khi - klo > 1)) {
      const uint32_t kmid = klo + (khi - klo) / 2;
      const int n = group_add<L>(count_from<V>(s, of_key(kmid)));
      if (khi - klo <= 1) continue;
      if (n >= K)
        klo = kmid, n_lo = n;
      else
        khi = kmid;
    }
    if (!found) lo = of_key(klo), exact = n_lo == K;
  }
  if (L == 32 ? exact : (bool)__all_sync(kAll, exact)) return false;
  on = bits_from<V>(s, lo);
  uint32_t above = 0;
#pragma unroll
  for (int j = 0; j < V; j++) above |= s[j] > lo ? 1u << j : 0u;
  uint32_t equal = on & ~above;
  int room = K - group_add<L>(__popc(above)) - group_below<L>(__popc(equal));
  if (!exact) {
    for (; equal && room > 0; room--) {
      above |= equal & -equal;
      equal &= equal - 1;
    }
    on = above;
  }
  return true;
}

// BIAS: there is a bias; what it needs would cost the others registers (65536 x 64
// bf16 22.2 us with one kernel for both, 21.3 so).
template <typename T, int V, int L, int SCORE, bool BIAS>
__global__ void __launch_bounds__(kThreads, V == 8 ? 5 : V == 16 ? 3 : 2) router_topk_kernel(RouterParams p) {
  constexpr int kTokens = 32 / L;                     // tokens of a warp
  constexpr int kChosen = V * L < 128 ? V * L : 128;  // K at the most
  constexpr bool kSoftmax = SCORE == MOE_SCORE_SOFTMAX;
  // a token's chosen: expert and logit, later weight
  __shared__ uint2 chosen_of[kWarps][kTokens][kChosen];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = lane % L, e0 = at * V;
  uint2* chosen = chosen_of[warp][lane / L];
  const bool divide = kSoftmax || p.renorm;

  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTokens; t0 < p.T;
       t0 += (int64_t)gridDim.x * kWarps * kTokens) {
    const int64_t t = t0 + lane / L;
    const bool real = t < p.T;
    const T* row = static_cast<const T*>(p.logits) + (real ? t : t0) * p.stride;
    float s[V];
    load_scores<T, V>(s, row, e0, 16 / sizeof(T), p.E, p.vector_in);
    if (BIAS) {  // the choice: a quotient rounded correctly, so that near ties fall as in plain fp32
#pragma unroll
      for (int j = 0; j < V; j++)
        if (s[j] > -INFINITY)  // (false past the end of the row)
          s[j] = (kSoftmax ? s[j] : __fdiv_rn(1.0f, 1.0f + expf(-s[j]))) + p.bias[e0 + j];
    }
    // a lane's experts as if all of them were finite, which the squares tell
    float low = s[0], top = s[0], sum = 0.0f, squares = 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++) {
      low = fminf(low, s[j]);
      top = fmaxf(top, s[j]);
      sum += s[j];
      squares = fmaf(s[j], s[j], squares);
    }
    if (e0 >= p.E) low = INFINITY, sum = squares = 0.0f;
    int live = p.E;
    if (__any_sync(kAll, !(squares < INFINITY))) {  // some are masked, past the end, infinite or NaN
      bool bad = false;
      low = INFINITY;
      top = -INFINITY;
      live = 0;
      sum = squares = 0.0f;
#pragma unroll
      for (int j = 0; j < V; j++) {
        bad |= s[j] != s[j];
        const bool in = s[j] > -INFINITY;
        s[j] = in ? s[j] : -INFINITY;  // NaN: masked
        live += in;
        low = fminf(low, in ? s[j] : INFINITY);
        top = fmaxf(top, s[j]);
        sum += in ? s[j] : 0.0f;
        squares = fmaf(in ? s[j] : 0.0f, in ? s[j] : 0.0f, squares);
      }
      if (bad && p.status) atomicOr(p.status, MOE_DEV_ERR_NAN_LOGIT);
      live = group_add<L>(live);
    }
    low = -group_max<L>(-low);
    top = group_max<L>(top);
    group_add2<L>(sum, squares);
    const float mean = __fdividef(sum, (float)live);
    const float dev = sqrtf(fmaxf(__fdividef(squares, (float)live) - mean * mean, 0.0f));
    float lo;
    uint32_t on = 0;
    const bool ties =
        select_top<V, L>(s, p.K, live, low, top, mean + dev * p.quantile, dev * p.spacing, lo, on);
    // `bits`: the chosen are marked in `on`
    const bool bits = V != 8 || ties || p.format == MOE_ROUTING_SPARSE_BOOL;
    if (bits && !ties) on = bits_from<V>(s, lo);

    // the chosen ids in ascending order through shared memory, and the logits
    // beside them where this lane still has them
    const int first = group_below<L>(bits ? __popc(on) : count_from<V>(s, lo)), count = min(live, p.K);
    const bool staged = V == 8 && !BIAS;
    int slot = first;
    if (!bits) {
      uint32_t to = (uint32_t)__cvta_generic_to_shared(chosen + first);
#pragma unroll
      for (int j = 0; j < V; j++)
        asm volatile(
            "{\n.reg .pred on;\n"
            "setp.ge.f32 on, %2, %3;\n"
            "@on st.shared.v2.b32 [%0], {%1, %2};\n"
            "@on add.u32 %0, %0, 8;\n}"
            : "+r"(to)
            : "r"(e0 + j), "f"(s[j]), "f"(lo)
            : "memory");
    } else if (V == 8) {
#pragma unroll
      for (int j = 0; j < V; j++)
        if (on >> j & 1) chosen[slot++] = make_uint2(e0 + j, __float_as_uint(s[j]));
    } else {
      for (uint32_t left = on; left; left &= left - 1) chosen[slot++].x = e0 + __ffs(left) - 1;
    }
    __syncwarp();

    // weights, L of the chosen at a time; the largest logit that takes part is
    // `top` itself, and looked for where the scores are not the logits
    float z = 0.0f;
    if (!BIAS) {
      if (kSoftmax && !p.renorm) {  // every live expert takes part in the sum
#pragma unroll
        for (int j = 0; j < V; j++) z += exp_below(s[j], top);
      }
    } else {
      top = -INFINITY;
      if (kSoftmax && !p.renorm) {
        // the bias takes part in the choice alone: an expert that it masks stays in the sum
        load_scores<T, V>(s, row, e0, 16 / sizeof(T), p.E, p.vector_in);
#pragma unroll
        for (int j = 0; j < V; j++) {
          s[j] = s[j] == s[j] ? s[j] : -INFINITY;
          top = fmaxf(top, s[j]);
        }
      } else {
        for (int k = at; k < count; k += L) top = fmaxf(top, to_float(row[chosen[k].x]));
      }
      top = group_max<L>(top);
      if (kSoftmax && !p.renorm) {
#pragma unroll
        for (int j = 0; j < V; j++) z += exp_below(s[j], top);
      }
    }
    const float m = p.renorm ? fminf(top, 0.0f) : 0.0f;
    for (int k = at; k < count; k += L) {
      const uint2 c = chosen[k];
      const float l = staged ? __uint_as_float(c.y) : to_float(row[c.x]);
      const float w = kSoftmax ? exp_below(l, top) : sigmoid_scaled(l, m);
      chosen[k].y = __float_as_uint(w);
      if (p.renorm) z += w;
    }
    if (divide) z = group_add<L>(z);
    const float f = divide ? __fdividef(p.scale, z) : p.scale;  // (z is 0 where nothing is chosen)
    if (p.format == MOE_ROUTING_DENSE_I16) {
      if (real) {
        for (int k = at; k < p.K; k += L) {
          const uint2 c = chosen[k];
          const bool in = k < count;
          static_cast<int16_t*>(p.map)[t * p.K + k] = (int16_t)(in ? (int)c.x : -1);
          p.probs[t * p.K + k] = in ? __uint_as_float(c.y) * f : 0.0f;
        }
      }
    } else {
      __syncwarp();
      slot = first;
#pragma unroll
      for (int j = 0; j < V; j++) s[j] = on >> j & 1 ? __uint_as_float(chosen[slot++].y) * f : 0.0f;
      if (real) {
        uint8_t* map = static_cast<uint8_t*>(p.map) + t * p.E;
        float* probs = p.probs + t * p.E;
        if (p.vector_out) {
#pragma unroll
          for (int j = 0; j < V; j += 8) {
            if (e0 + j >= p.E) continue;
            uint2 b = make_uint2(0, 0);
#pragma unroll
            for (int i = 0; i < 4; i++) {
              b.x |= (on >> (j + i) & 1) << (8 * i);
              b.y |= (on >> (j + 4 + i) & 1) << (8 * i);
            }
            *reinterpret_cast<uint2*>(map + e0 + j) = b;
#pragma unroll
            for (int i = 0; i < 8; i += 4)
              *reinterpret_cast<float4*>(probs + e0 + j + i) =
                  make_float4(s[j + i], s[j + i + 1], s[j + i + 2], s[j + i + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; j++) {
            if (e0 + j >= p.E) continue;
            map[e0 + j] = on >> j & 1;
            probs[e0 + j] = s[j];
          }
        }
      }
    }
    __syncwarp();  // before the next token's chosen
  }
}

struct RouterBwdParams {
  int64_t T, stride, gstride;
  int E, K;
  int renorm, format;
  bool vector_in, vector_out, vector_map;
  float scale;
  const void *logits, *map;
  const float* gp;
  void* gl;
};

// Gradient where only the chosen take part: a lane takes one of them (or a few),
// and the row goes out through shared memory, zeros but for theirs.  Of the
// logits, and of a sparse map's gradients, only those of the chosen are read
// (16384 x 1024 top-32 fp32: 20 us; as a pass over the row, which the kernel
// below makes for the plain softmax, 66).
template <typename T, int V, int L, int SCORE, bool SPARSE>
__global__ void __launch_bounds__(kThreads, V == 8 ? (SPARSE ? 5 : 4) : 2) router_bwd_chosen_kernel(RouterBwdParams p) {
  constexpr int kTokens = 32 / L, N = 16 / sizeof(T), kVecs = V / N;
  constexpr int kEach = SPARSE || V == 8 ? V : 128 / L;  // chosen of a lane at the most
  constexpr bool kSoftmax = SCORE == MOE_SCORE_SOFTMAX;
  __shared__ uint4 staged[kWarps][kTokens * L * kVecs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % L;
  uint4* vecs = staged[warp] + lane / L * (L * kVecs);  // this token's row
  T* grow = reinterpret_cast<T*>(vecs);
  int16_t* ids = reinterpret_cast<int16_t*>(vecs);  // before the row

  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTokens; t0 < p.T;
       t0 += (int64_t)gridDim.x * kWarps * kTokens) {
    const int64_t t = t0 + lane / L;
    const bool real = t < p.T;
    const T* row = static_cast<const T*>(p.logits) + (real ? t : t0) * p.stride;
    int count = real ? p.K : 0;
    if (SPARSE) {  // the chosen ids in ascending order
      const uint8_t* map = static_cast<const uint8_t*>(p.map) + (real ? t : t0) * p.E;
      const int e0 = at * V;
      uint32_t on = 0;
      if (p.vector_map) {
#pragma unroll
        for (int j = 0; j < V; j += 8) {
          if (e0 + j >= p.E) continue;
          const uint2 b = *reinterpret_cast<const uint2*>(map + e0 + j);
#pragma unroll
          for (int i = 0; i < 8; i++) on |= (uint32_t)(((i < 4 ? b.x : b.y) >> (8 * (i & 3)) & 0xffu) != 0) << (j + i);
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; j++)
          if (e0 + j < p.E) on |= (uint32_t)(map[e0 + j] != 0) << j;
      }
      count = group_add<L>(__popc(on));
      int slot = group_below<L>(__popc(on));
      for (; on; on &= on - 1) ids[slot++] = (int16_t)(e0 + __ffs(on) - 1);
      if (!real) count = 0;
      __syncwarp();
    }
    int e[kEach];
    float l[kEach], g[kEach], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      if (i * L >= count) break;
      const int k = at + i * L;
      e[i] = -1;
      if (k < count) e[i] = SPARSE ? ids[k] : static_cast<const int16_t*>(p.map)[t * p.K + k];
      if (e[i] >= p.E) e[i] = -1;
      g[i] = e[i] >= 0 ? p.gp[SPARSE ? t * p.E + e[i] : t * p.K + k] : 0.0f;
      l[i] = e[i] >= 0 ? to_float(row[e[i]]) : -INFINITY;
      if (!(l[i] > -INFINITY)) e[i] = -1, l[i] = -INFINITY, g[i] = 0.0f;  // masked or NaN
      top = fmaxf(top, l[i]);
    }
    if (SPARSE) __syncwarp();  // the ids are read
#pragma unroll
    for (int j = 0; j < kVecs; j++) vecs[j * L + at] = make_uint4(0, 0, 0, 0);
    if (kSoftmax || p.renorm) top = group_max<L>(top);
    const float m = p.renorm ? fminf(top, 0.0f) : 0.0f;
    float n[kEach], z = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      if (i * L >= count) break;
      n[i] = e[i] < 0 ? 0.0f : kSoftmax ? exp_below(l[i], top) : sigmoid_scaled(l[i], m);
      z += n[i];
      dot = fmaf(g[i], n[i], dot);
    }
    float inv = p.scale;
    if (p.renorm) {
      group_add2<L>(z, dot);
      const float r = z > 0.0f ? __fdividef(1.0f, z) : 0.0f;
      inv *= r;
      dot *= r;
    } else {
      dot = 0.0f;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      if (i * L >= count) break;
      float v = n[i] * inv * (g[i] - dot);
      if (!kSoftmax) v *= sigmoid_rest(l[i]);
      if (e[i] >= 0 && n[i] != 0.0f) grow[e[i]] = from_float<T>(v);
    }
    __syncwarp();
    if (real) {
      T* out = static_cast<T*>(p.gl) + t * p.gstride;
      if (p.vector_out) {
#pragma unroll
        for (int j = 0; j < kVecs; j++)
          if ((j * L + at) * N < p.E) reinterpret_cast<uint4*>(out)[j * L + at] = vecs[j * L + at];
      } else {
        for (int i = at; i < p.E; i += L) out[i] = grow[i];
      }
    }
    __syncwarp();  // before the next token's row
  }
}

// Gradient of the plain softmax, where every expert takes part.  A lane takes 16
// bytes of a row at every L-th place, so that loads and stores are whole lines.
template <typename T, int V, int L>
__global__ void __launch_bounds__(kThreads, V == 32 ? 2 : 1) router_bwd_all_kernel(RouterBwdParams p) {
  constexpr int kTokens = 32 / L, N = 16 / sizeof(T);
  __shared__ uint4 staged[kWarps][kTokens * V * L / 4];  // dense maps: gradients by expert
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % L;
  uint4* token = staged[warp] + lane / L * L * (V / 4);
  float* row_g = reinterpret_cast<float*>(token);
  auto expert = [&](int j) { return (j / N * L + at) * N + j % N; };

  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTokens; t0 < p.T;
       t0 += (int64_t)gridDim.x * kWarps * kTokens) {
    const int64_t t = t0 + lane / L;
    const bool real = t < p.T;
    float l[V], g[V];
    load_scores<T, V>(l, static_cast<const T*>(p.logits) + (real ? t : t0) * p.stride, at * N, L * N, p.E, p.vector_in);
    if (p.format == MOE_ROUTING_DENSE_I16) {
#pragma unroll
      for (int j = 0; j < V / 4; j++) token[j * L + at] = make_uint4(0, 0, 0, 0);
      __syncwarp();
      if (real) {
        for (int k = at; k < p.K; k += L) {
          const int e = static_cast<const int16_t*>(p.map)[t * p.K + k];
          if (e >= 0 && e < p.E) row_g[e] = p.gp[t * p.K + k];
        }
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(row_g + expert(j));
        g[j] = v.x, g[j + 1] = v.y, g[j + 2] = v.z, g[j + 3] = v.w;
      }
      __syncwarp();
    } else {
      const uint8_t* map = static_cast<const uint8_t*>(p.map) + (real ? t : t0) * p.E;
      const float* gp = p.gp + (real ? t : t0) * p.E;
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const int e = expert(j);
        if (p.vector_map && e < p.E) {
          const uint32_t b = *reinterpret_cast<const uint32_t*>(map + e);
          const float4 v = *reinterpret_cast<const float4*>(gp + e);
          g[j] = b & 0xffu ? v.x : 0.0f;
          g[j + 1] = b >> 8 & 0xffu ? v.y : 0.0f;
          g[j + 2] = b >> 16 & 0xffu ? v.z : 0.0f;
          g[j + 3] = b >> 24 ? v.w : 0.0f;
        } else {
#pragma unroll
          for (int i = 0; i < 4; i++) g[j + i] = e + i < p.E && map[e + i] != 0 ? gp[e + i] : 0.0f;
        }
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; j++) top = fmaxf(top, l[j]);
    top = group_max<L>(top);
    // l: the weight each expert takes part with, 0 where it is masked, NaN or past
    // the row's end; z its sum; dot = sum of g n
    float z = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const bool in = l[j] > -INFINITY;
      const float n = exp_below(l[j], top);
      l[j] = in ? n : 0.0f;
      g[j] = in ? g[j] : 0.0f;
      z += l[j];
      dot = fmaf(g[j], l[j], dot);
    }
    group_add2<L>(z, dot);
    const float r = z > 0.0f ? __fdividef(1.0f, z) : 0.0f, inv = p.scale * r;
    dot *= r;
#pragma unroll
    for (int j = 0; j < V; j++) g[j] = l[j] != 0.0f ? l[j] * inv * (g[j] - dot) : 0.0f;
    if (!real) continue;
    T* out = static_cast<T*>(p.gl) + t * p.gstride;
#pragma unroll
    for (int j = 0; j < V; j += N) {
      const int e = expert(j);
      if (p.vector_out) {
        union {
          uint4 v;
          T e[N];
        } u;
#pragma unroll
        for (int i = 0; i < N; i++) u.e[i] = from_float<T>(g[j + i]);
        if (e < p.E) *reinterpret_cast<uint4*>(out + e) = u.v;
      } else {
#pragma unroll
        for (int i = 0; i < N; i++)
          if (e + i < p.E) out[e + i] = from_float<T>(g[j + i]);
      }
    }
  }
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int L>
unsigned token_grid(int64_t T) {
  const int64_t per_block = kWarps * (32 / L);
  const int64_t blocks = (T + per_block - 1) / per_block, cap = (int64_t)device_sm_count() * (2048 / kThreads);
  return (unsigned)(blocks < cap ? blocks : cap);
}

// Eight experts a lane and as few lanes a token as hold them, up to a warp; more
// experts a lane beyond 256.  (A warp a token, whatever E: 65536 x 16 47 us, so 7.6;
// eight experts are two fp32 vectors or one 16-bit vector of a lane.)
#define MOE_ROUTER_SHAPE(RUN)         \
  do {                                \
    if (p.E <= 8) RUN(8, 1);          \
    else if (p.E <= 16) RUN(8, 2);    \
    else if (p.E <= 32) RUN(8, 4);    \
    else if (p.E <= 64) RUN(8, 8);    \
    else if (p.E <= 128) RUN(8, 16);  \
    else if (p.E <= 256) RUN(8, 32);  \
    else if (p.E <= 512) RUN(16, 32); \
    else RUN(32, 32);                 \
  } while (0)

template <typename T, int SCORE>
void run_topk(const RouterParams& p, cudaStream_t st) {
#define RUN(V, L) router_topk_kernel<T, V, L, SCORE, true><<<token_grid<L>(p.T), kThreads, 0, st>>>(p)
  if (p.bias) {
    MOE_ROUTER_SHAPE(RUN);
    return;
  }
#undef RUN
#define RUN(V, L) router_topk_kernel<T, V, L, SCORE, false><<<token_grid<L>(p.T), kThreads, 0, st>>>(p)
  MOE_ROUTER_SHAPE(RUN);
#undef RUN
}

template <typename T, int SCORE>
void run_bwd(const RouterBwdParams& p, cudaStream_t st) {
#define RUN(V, L) router_bwd_all_kernel<T, V, L><<<token_grid<L>(p.T), kThreads, 0, st>>>(p)
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
    if (!p.renorm) {
      MOE_ROUTER_SHAPE(RUN);
      return;
    }
  }
#undef RUN
#define RUN(V, L) router_bwd_chosen_kernel<T, V, L, SCORE, true><<<token_grid<L>(p.T), kThreads, 0, st>>>(p)
  if (p.format == MOE_ROUTING_SPARSE_BOOL) {
    MOE_ROUTER_SHAPE(RUN);
    return;
  }
#undef RUN
#define RUN(V, L) router_bwd_chosen_kernel<T, V, L, SCORE, false><<<token_grid<L>(p.T), kThreads, 0, st>>>(p)
  MOE_ROUTER_SHAPE(RUN);
#undef RUN
}

template <int SCORE, typename Params>
void run_score(int32_t dtype, const Params& p, cudaStream_t st) {
  constexpr bool kBackward = std::is_same<Params, RouterBwdParams>::value;
  auto run = [&](auto zero) {
    using T = decltype(zero);
    if constexpr (kBackward)
      run_bwd<T, SCORE>(p, st);
    else
      run_topk<T, SCORE>(p, st);
  };
  switch (dtype) {
    case MOE_ELEM_F32: run(0.0f); break;
    case MOE_ELEM_BF16: run(__nv_bfloat16()); break;
    default: run(__half()); break;
  }
}

template <typename Params>
cudaError_t run_dtype(const moe_router& r, const Params& p, cudaStream_t st) {
  if (r.score == MOE_SCORE_SOFTMAX)
    run_score<MOE_SCORE_SOFTMAX>(r.logits_dtype, p, st);
  else
    run_score<MOE_SCORE_SIGMOID>(r.logits_dtype, p, st);
  return cudaGetLastError();
}

int elem_bytes(int32_t dtype) { return dtype == MOE_ELEM_F32 ? 4 : 2; }

// Rows of E elements that are whole 16-byte vectors.
bool vector_rows(const moe_rows& m, int64_t E, int bytes) {
  return E * bytes % 16 == 0 && E % 8 == 0 && m.stride * bytes % 16 == 0 && aligned(m.data, 16);
}

}  // namespace

cudaError_t launch_router_topk(const moe_router& r, const moe_rows& logits, const float* bias, int32_t format,
                               void* map, float* probs, int32_t* status, cudaStream_t st) {
  RouterParams p = {};
  p.T = r.T;
  p.E = (int)r.E;
  p.K = (int)r.K;
  p.renorm = r.renormalize != 0;
  p.scale = r.scale;
  p.format = format;
  p.logits = logits.data;
  p.stride = logits.stride;
  p.bias = bias;
  p.map = map;
  p.probs = probs;
  p.status = status;
  // the upper tail's quantile by the rational approximation 26.2.23 of Abramowitz
  // and Stegun's handbook
  const float tail = (float)r.K / (float)(r.E + 1), side = tail <= 0.5f ? tail : 1.0f - tail;
  const float q = std::sqrt(-2.0f * std::log(side));
  const float x = q - (2.515517f + q * (0.802853f + q * 0.010328f)) /
                          (1.0f + q * (1.432788f + q * (0.189269f + q * 0.001308f)));
  p.quantile = tail <= 0.5f ? x : -x;
  p.spacing = std::exp(0.5f * x * x) * 2.5066283f / (float)r.E;  // 1 / (E density)
  p.vector_in = vector_rows(logits, r.E, elem_bytes(r.logits_dtype));
  p.vector_out = r.E % 8 == 0 && aligned(map, 8) && aligned(probs, 16);
  return run_dtype(r, p, st);
}

cudaError_t launch_router_topk_backward(const moe_router& r, const moe_rows& logits, int32_t format, const void* map,
                                        const float* grad_probs, const moe_rows& grad_logits, cudaStream_t st) {
  RouterBwdParams p = {};
  p.T = r.T;
  p.E = (int)r.E;
  p.K = (int)r.K;
  p.renorm = r.renormalize != 0;
  p.scale = r.scale;
  p.format = format;
  p.logits = logits.data;
  p.stride = logits.stride;
  p.map = map;
  p.gp = grad_probs;
  p.gl = grad_logits.data;
  p.gstride = grad_logits.stride;
  const int b = elem_bytes(r.logits_dtype);
  p.vector_in = vector_rows(logits, r.E, b);
  p.vector_out = vector_rows(grad_logits, r.E, b);
  p.vector_map = r.E % 8 == 0 && aligned(map, 8) && aligned(grad_probs, 16);
  return run_dtype(r, p, st);
}

}  // namespace moe
