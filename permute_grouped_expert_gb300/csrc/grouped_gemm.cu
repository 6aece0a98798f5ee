// grouped_gemm.cu -- products grouped by expert on the tensor cores of pairs of
// SMs (2-CTA clusters, tcgen05 cta_group::2, operands by TMA, sums in TMEM).
//
//   kForward  y[r]  = W x[r]            kData  gx[r] = W^T gy[r]
//   kWeight   gW    = sum gy[r] x[r]^T (+ addend)
//
// Rows' products put the expert's matrix on the M side of the MMA and its rows on
// the N side: a tile is 256 features (128 a CTA) by up to 256 rows, and an expert's
// last rows cost what they are, in steps of 32, where rows as M would be filled up
// to 256.  kData reads W as it lies, its features contiguous (an M-major operand),
// so that no transposed copy exists.  The weights' gradient has 256 x 256 tiles of
// the matrix and runs along the expert's rows, both operands with M and N
// contiguous; rows that are not the expert's (they may hold anything, NaN too) are
// never read: the copies of an expert's last rows end with them, zeros in front.
//
// Per CTA, warp-specialised (rank 0 leads the pair):
//   warps 0, 3  TMA producers of its half of the first and of the second operand, 64 of
//               the contraction a stage: one copy each (a thread issues a copy in about 120
//               cycles, whatever its bytes; four of 8 KB a stage were what the weights'
//               gradient waited for)
//   warp 1      TMEM; on the leader one elected lane issues the MMAs (PIECES: on the
//               other CTA one tells the leader of the stages that were filled there)
//   warp 2      on the leader: claims tiles and hands their numbers to both CTAs
//   warps 4..   epilogue of this CTA's 128 features, beside the next tile's MMAs
//   PIECES: the last eight warps bring operands into place
// Every wait is bounded (MOE_DEV_ERR_TIMEOUT, then a clean exit); those that a whole
// tile may take go on as long as its stages do.
//
// Device times on one GB300, beside the floor by a copy's 6796 GB/s or 1880 TFLOP/s
// and what bounds them:
//   1 token, 8 of 256 experts, 7168 x 2048 bf16       42 us,  82 %  launch, HBM
//   64 tokens, the same                              950 us, 101 %  HBM
//   8192 tokens, 256 experts, 4096 x 7168, uneven   3.4 ms,  72 %  HBM and MMAs, not together
//     its weights' gradient in bf16 / fp32           4.0 / 5.8 ms, 61 / 79 %; added to itself 20.7 ms
//   4096 tokens, 64 experts, 2048 x 2048             210 us,  70 %  copies into shared memory
//     its weights' gradient in fp32                  266 us,  74 %  stores beside the copies
//       added to itself                              730 us,  49 %  reads of the old one
//   8192 x 8192 x 8192 over 8 experts                700 us,  84 %  MMAs (power), last tiles
//     its weights' gradient in bf16 / fp32           720 / 948 us
//   the same of 8191 x 8191                         1.59 ms,  37 %  shifting into place
// (the middle of several boxes, which differ by up to 3 %)
// An SM takes in 64 bytes a cycle at the most, which is what a whole tile needs at the
// MMAs' full rate: tiles of fewer rows wait for their copies.
#include <type_traits>

#include "block_common.cuh"
#include "grouped_gemm.h"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int kPieceWarps = 8;  // that bring unaligned operands into place
// Epilogue warps: with few steps along the contraction the rows' products wait for
// them (5264 features of 64 for 15364 rows: four 124 us, eight 43).
template <GemmDir DIR, bool PIECES>
constexpr int kEpilogue = DIR == kWeight && !PIECES ? 4 : 8;
template <GemmDir DIR, bool PIECES>
constexpr int kThreads = 128 + 32 * (kEpilogue<DIR, PIECES> + (PIECES ? kPieceWarps : 0));
// An MMA cuts off what its fp32 sum cannot hold, of each product too: 768 numbers of
// one sign come out short by 5e-7 in bf16 and 4e-6 in f16 (whose products have more
// bits to lose), 8192 by 4e-5 and 5e-5.  So sums are made of parts, added to one another
// by rounding, and no shorter however long they are.  fp32 gradients: parts of at most
// 12 stages (768 rows), added on their way to memory; 8192 x 8192 of 1024 rows an expert
// took 959 us so, 867 in one part.  Results of 16 bits: parts of 128 stages, a tenth of
// f16's rounding each, joined in TMEM by the epilogue (one sum of 2^20 was short by
// 7e-3; 2048 x 2048 x 65536 over 2 experts: 363 us, in one part 358).
template <GemmDir DIR, typename OUT>
constexpr bool kJoin = DIR != kWeight || sizeof(OUT) == 2;
template <GemmDir DIR, typename OUT>
constexpr int kPart = kJoin<DIR, OUT> ? 128 : 12;
constexpr int BM = 256, BN = 256, BK = 64;  // of a pair's tile; BK: of a stage
// Tiles that may be on their way to the readers: more where tiles are short, fewer
// where the last ones would wait behind long ones.
template <GemmDir DIR>
constexpr int kSlotsOf = DIR == kWeight ? 4 : 2;
template <GemmDir DIR, bool PIECES>
constexpr int kStagesOf = PIECES ? 3 : DIR == kWeight ? 5 : 6;
// PIECES: stages as they lie in memory, ahead of those; bytes of a row (64 or 128
// elements that start anywhere in their first piece of 16 bytes), of the rows that
// are eight apart, and of an operand.
template <GemmDir DIR>
constexpr int kRawOf = DIR == kWeight ? 2 : 3;
template <bool KMAJOR>
constexpr uint32_t kRawRow = KMAJOR ? 144 : 272;
template <bool KMAJOR>
constexpr uint32_t kRawRows = KMAJOR ? 16 : 8;
template <bool KMAJOR>
constexpr uint32_t kRawEighth = kRawRows<KMAJOR> * kRawRow<KMAJOR>;
constexpr uint32_t kRawOperand = 8 * kRawEighth<true>;
constexpr int kBand = 8;                                // tiles of a band that share their operands in L2
constexpr uint32_t kOperand = 128 * BK * 2;             // a CTA's half of an operand: 16 KB
constexpr uint32_t kBox = 64 * BK * 2;                  // a box of an operand that is not K-major
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxE = 1024;
constexpr uint32_t kOutBytes = 32 * 128;                // kWeight: a warp's 32 rows of 128 bytes, twice
constexpr int kTurn = 33;                               // and in pieces: a row of 32 results and a word between
template <GemmDir DIR, bool PIECES>
constexpr size_t kDynSmem = 1024 + (size_t)kStagesOf<DIR, PIECES> * kStageBytes +
                            (PIECES ? 2 * kRawOf<DIR> * kRawOperand : 0) +
                            (DIR != kWeight ? 0 : PIECES ? 8 * 32 * kTurn * 4 : 8 * kOutBytes);

struct TcParams {
  const int32_t *offsets, *counts;
  int32_t* status;
  int32_t* next;  // tile counter, or NULL: tiles in turn
  void* out;
  const float* addend;
  int64_t sout;
  int64_t cap;
  int64_t routes;  // of all tokens
  int E;
  int features, contraction;  // rows' products
  int N, Kd;                  // kWeight
  int mt;                     // tiles of 256 features (kWeight: of N)
  int kt;                     // kWeight: tiles of 256 of Kd
  bool a_groups, b_groups;    // the operand's map has columns in groups of 64
  const uint16_t *a, *b;      // PIECES: the operands, strides of their rows
  int64_t sa, sb;
};

// Routed rows [beg, end) of expert e below the capacity; empty where the handle
// holds no segment, and no more than the shape has routes (there are maps for no
// more), whatever the handle says.
MOE_DEVICE void gemm_segment(const TcParams& p, int e, int64_t& beg, int64_t& end) {
  const int64_t off = p.offsets[e], cnt = min64(p.counts[e], p.routes);
  beg = min64(max64(off, 0), p.cap);
  end = off < 0 || cnt <= 0 ? beg : max64(min64(off + cnt, p.cap), beg);
}

// A tile as the pair's readers get it.
struct alignas(16) Tile {
  int e, m, n;   // expert, -1 behind the last tile; tile of features; kWeight: tile of Kd
  int row, end;  // rows [row, end) of the tile, or of the expert (kWeight)
  int cols;      // columns of the MMA
  int blocks;    // stages along the contraction
  int pad;
};

// Maps of the operands.  The second's have boxes of 16, 32, .. 128 rows, so that a
// tile's half of a stage is one copy whatever its rows (as copies of 16 rows, 8192 x
// 8192 x 8192 over experts of about 1024 rows took 1031 us where whole tiles took
// 717); kWeight and the first operand: one.  PIECES: the rows r of either with r % 8
// equal to the index.
struct Maps {
  CUtensorMap a[8], b[8], out;
};

// Tiles of an expert in bands of kBand along one side, the other side outermost in
// a band: tiles that run at once share few operands.
MOE_DEVICE void banded(int local, int along, int across, int& a, int& c) {
  const int band = local / (kBand * across), in = local - band * kBand * across;
  const int width = min(kBand, along - band * kBand);
  c = in / width;
  a = band * kBand + in - c * width;
}

// Tiles of rows of an expert with `rows` rows, and rows of each.
MOE_DEVICE int row_tiles(int64_t rows) { return (int)((rows + BN - 1) / BN); }
MOE_DEVICE int tile_rows(int64_t rows, int tiles) { return (int)((rows + tiles - 1) / tiles + 31) & ~31; }

// The order of the tiles.  Experts of up to BN rows cost their matrix's bytes, the
// others products.  The rows' products deal the tiles of both kinds out evenly among
// each other, so that HBM and the tensor cores work together (FC1 of 8192 tokens, one
// kind behind the other 3550 us, so 3481; by expert 3499 when that was 3315); the
// weights' gradient takes the long tiles first (FC2's 1192 us, mixed 1220).
struct Order {
  int tiles[2];            // of either kind: 0 products, 1 bytes
  int experts[2];
  uint64_t share;          // of the second kind, in 2^-32
  int before[2][kMaxE];    // tiles of the kind's experts before
  uint16_t expert[2][kMaxE];
};

// Filled by one warp, whose lanes take a run of experts each: one scan, whatever
// their number.  per: tiles of an expert (kForward, kData: of each of its tiles of
// rows).
template <bool WEIGHT>
MOE_DEVICE void make_order(Order& o, const TcParams& p, int per) {
  const int lane = threadIdx.x & 31, run = (p.E + 31) / 32, e0 = lane * run, e1 = min(e0 + run, p.E);
  auto rows_of = [&](int e) {
    int64_t beg = 0, end = 0;
    if (e < e1) gemm_segment(p, e, beg, end);
    return (int)(end - beg);
  };
  int tiles[2] = {0, 0}, experts[2] = {0, 0};
  auto add = [&](int rows, int (&t)[2], int (&x)[2]) {
    const int mine = WEIGHT ? per : row_tiles(rows) * per;
    t[0] += rows > BN ? mine : 0;
    t[1] += rows > BN ? 0 : mine;
    x[0] += mine && rows > BN;
    x[1] += mine && rows <= BN;
  };
  constexpr int kAhead = 8;
  for (int e = e0; e < e0 + run; e += kAhead) {
    int rows[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; j++) rows[j] = rows_of(e + j);
#pragma unroll
    for (int j = 0; j < kAhead; j++)
      if (e + j < e1) add(rows[j], tiles, experts);
  }
  int t_sum[2] = {tiles[0], tiles[1]}, x_sum[2] = {experts[0], experts[1]};  // up to this lane
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int a = __shfl_up_sync(0xffffffffu, t_sum[k], d), b = __shfl_up_sync(0xffffffffu, x_sum[k], d);
      if (lane >= d) t_sum[k] += a, x_sum[k] += b;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < 2; k++) o.tiles[k] = t_sum[k], o.experts[k] = x_sum[k];
    // rounded up: after all tiles the second kind has had all of its
    const uint64_t total = (uint64_t)t_sum[0] + t_sum[1];
    o.share = total ? (((uint64_t)t_sum[1] << 32) + total - 1) / total : 0;
  }
  int t[2] = {t_sum[0] - tiles[0], t_sum[1] - tiles[1]}, x[2] = {x_sum[0] - experts[0], x_sum[1] - experts[1]};
  for (int e = e0; e < e1; e++) {
    const int rows = rows_of(e), kind = rows <= BN;
    if (WEIGHT || rows > 0) {
      o.expert[kind][kind ? x[1] : x[0]] = (uint16_t)e;
      o.before[kind][kind ? x[1] : x[0]] = kind ? t[1] : t[0];
    }
    add(rows, t, x);
  }
  __syncwarp();
}

template <GemmDir DIR>
MOE_DEVICE Tile tile_of(int64_t t, const Order& o, const TcParams& p) {
  Tile i = {};
  const int64_t total = (int64_t)o.tiles[0] + o.tiles[1];
  if (t >= total) {
    i.e = -1;
    return i;
  }
  // bytes' tiles before t, and before t + 1
  auto bytes = [&](int64_t n) {
    return DIR == kWeight ? max64(n - o.tiles[0], 0) : (int64_t)((uint64_t)n * o.share >> 32);
  };
  const int64_t s = bytes(t);
  const int kind = bytes(t + 1) > s ? 1 : 0;
  const int at = (int)(kind ? s : t - s);
  const int x = expert_of_row(o.before[kind], o.experts[kind], at), local = at - o.before[kind][x];
  int64_t beg, end;
  i.e = o.expert[kind][x];
  gemm_segment(p, i.e, beg, end);
  if (DIR == kWeight) {
    banded(local, p.mt, p.kt, i.m, i.n);
    i.row = (int)beg;
    i.end = (int)end;
    i.cols = BN;
    i.blocks = (int)((end - beg + BK - 1) / BK);
  } else {
    const int tiles = row_tiles(end - beg);
    banded(local, tiles, p.mt, i.n, i.m);
    i.cols = tile_rows(end - beg, tiles);
    i.row = (int)(beg + (int64_t)i.n * i.cols);
    i.end = (int)min64((int64_t)i.row + i.cols, end);
    i.blocks = (p.contraction + BK - 1) / BK;
  }
  return i;
}

template <typename T>
MOE_DEVICE uint32_t pack2(float a, float b);
template <>
MOE_DEVICE uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
MOE_DEVICE uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 columns of TMEM added to 32 others, by a warp whose lanes they are.
MOE_DEVICE void add_columns(uint32_t to, uint32_t from) {
  float a[32], b[32];
  uint32_t sum[32];
  tmem_ld32(to, a);
  tmem_ld32(from, b);
#pragma unroll
  for (int j = 0; j < 32; j++) sum[j] = __float_as_uint(a[j] + b[j]);
  tmem_st32(to, sum);
}

MOE_DEVICE void settle(uint64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) __nanosleep(1000);
}

// PIECES: operands whose rows TMA does not take one after another (odd widths, rows
// that start anywhere).  Rows that are eight apart lie a multiple of 16 bytes apart
// whatever the stride, so that eight copies a stage bring an operand's rows to shared
// memory as they lie; from there each eight elements are shifted into the place that
// the MMA reads.  (Loaded by threads, a stage ahead, 8191 x 8191 x 8192 took 2.9 ms,
// most of it in the loads' issue.)  Beyond the end of the contraction are zeros; rows
// and columns beyond the operand's give results that are not stored, whatever is there.

// The eight elements of two pieces of 16 bytes from word WORDS and `half` bits (0 or 16) on.
template <int WORDS>
MOE_DEVICE uint4 shifted(int4 lo, int4 hi, uint32_t half) {
  const int w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = __funnelshift_r(w[WORDS + i], w[WORDS + i + 1], half);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Zeros from the n-th element on.
MOE_DEVICE uint4 first_of(uint4 v, int n) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) w[i] = 2 * i >= n ? 0u : 2 * i + 1 >= n ? w[i] & 0xffffu : w[i];
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA's half of an operand in place: 128 rows of 64 elements in shared memory, of
// which a thread has eight elements of every 32nd.  KMAJOR: they are rows of the
// operand; otherwise two runs of 64 columns along 64 rows.  From row to row of a
// thread and from stage to stage lie multiples of eight rows and of 64 elements, so
// that a thread's elements keep their place in their pieces.  A warp's rows are eight
// apart too, so that one branch a stage finds the words of all its pieces, and reads of
// an operand's pieces all go out before the first is written (8191 x 8191 x 8192, then:
// 1.61 ms; four rows next to each other in a warp, each thread selecting its words,
// 1.70; reading and writing in turn besides, 1.96).
template <bool KMAJOR>
struct Half {
  uint32_t raw;   // where this thread's first piece is in a stage
  uint32_t from;  // byte of the piece, the same in a warp
  int k;          // of the contraction left: elements from this thread's first on, or rows

  // Of a thread: its warp's, and eight apart.
  static MOE_DEVICE int first_row(int t) { return (t >> 5) + (t & 24); }

  // KMAJOR: rows from `row` on along k elements; otherwise columns
  // from `col` on, along k rows from `row` on.
  MOE_DEVICE void begin_tile(const uint16_t* base, int64_t stride, int64_t row, int col, int contraction, int t) {
    const int q = t & 7, j = first_row(t), eighth = (int)((row + j) & 7);
    from = __shfl_sync(0xffffffffu, (uint32_t)(reinterpret_cast<uintptr_t>(base + (row + j) * stride) & 15), 0);
    raw = eighth * kRawEighth<KMAJOR> + (uint32_t)(((row + j) >> 3) - ((row - eighth + 7) >> 3)) * kRawRow<KMAJOR> + q * 16;
    k = contraction - (KMAJOR ? q * 8 : j);
  }

  // (all 128 rows whatever the tile's: a branch for fewer costs whole tiles 8 %)
  template <int WORDS>
  MOE_DEVICE void shift_by(uint8_t* to, const uint8_t* at, bool whole) {
    int4 lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint8_t* piece = at + (KMAJOR ? 4 * i * kRawRow<true> : 4 * (i & 1) * kRawRow<false> + 128 * (i >> 1));
      lo[i] = ld_shared_v4(piece), hi[i] = ld_shared_v4(piece + 16);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint4 v = shifted<WORDS>(lo[i], hi[i], (from & 2) * 8);
      if (!whole) v = first_of(v, KMAJOR ? k : k > 32 * (i & 1) ? 8 : 0);
      st_shared_v4(to + 32 * i * 128, v);
    }
  }

  MOE_DEVICE void shift(uint8_t* to, const uint8_t* stage, int t) {
    const int q = t & 7, j = first_row(t);
    to += j * 128 + ((q ^ (j & 7)) * 16);
    const uint8_t* at = stage + raw;
    // a warp's elements are all of the contraction
    const bool whole = __all_sync(0xffffffffu, KMAJOR ? k >= 8 : k > 32);
    switch (from >> 2) {
      case 0: shift_by<0>(to, at, whole); break;
      case 1: shift_by<1>(to, at, whole); break;
      case 2: shift_by<2>(to, at, whole); break;
      default: shift_by<3>(to, at, whole);
    }
    k -= BK;
  }
};

// Copies of the rows of a stage, one for each that are eight apart.
template <bool KMAJOR>
MOE_DEVICE void copy_eighths(uint8_t* to, const CUtensorMap* maps, int64_t row, int col, uint64_t* bar) {
#pragma unroll 1
  for (int r = 0; r < 8; r++)
    tma_load_2d(to + r * kRawEighth<KMAJOR>, maps + r, col, (int)((row - r + 7) >> 3), bar);
}

// T: 16-bit type of the operands; OUT: of the result; PIECES: operands of any
// alignment, without the maps.
template <GemmDir DIR, typename T, typename OUT, bool PIECES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<DIR, PIECES>, 1)
    grouped_gemm_kernel(const __grid_constant__ Maps maps, TcParams p) {
  constexpr int kStages = kStagesOf<DIR, PIECES>, kSlots = kSlotsOf<DIR>, kRaw = PIECES ? kRawOf<DIR> : 1;
  constexpr int kEpi = kEpilogue<DIR, PIECES>;
  constexpr bool kW = DIR == kWeight, kAmn = DIR != kForward, kBmn = kW;
  extern __shared__ uint8_t dyn_smem[];
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_placed[kStages], s_tfull[2], s_tempty[2];
  __shared__ __align__(8) uint64_t s_raw[kRaw], s_raw_free[kRaw];  // PIECES, each CTA's own
  __shared__ __align__(8) uint64_t s_have[kSlots], s_free[kSlots], s_drain;
  __shared__ Tile s_tile[kSlots];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_filled;  // s_filled: stages copied by warp 0, ever
  __shared__ Order s_order;  // the leader's

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  volatile int *abort_flag = &s_abort, *filled = &s_filled;

  if (threadIdx.x == 0) {
    s_abort = s_filled = 0;
    for (int s = 0; s < kStages; s++) {
      // on the leader: its producer and both CTAs' bytes; PIECES: every warp that fills it
      // there, and the other CTA's warp 1 for all that do here
      mbar_init(&s_full[s], PIECES ? kPieceWarps + 1 : 1);
      mbar_init(&s_empty[s], 1);             // each CTA's own, by the leader's commit
      mbar_init(&s_placed[s], kPieceWarps);  // PIECES, the other CTA's own
    }
    for (int a = 0; a < 2; a++) {
      mbar_init(&s_tfull[a], 1);
      mbar_init(&s_tempty[a], 2 * kEpi);  // on the leader: the epilogue warps of each CTA
    }
    for (int s = 0; s < kSlots; s++) {
      mbar_init(&s_have[s], 1);
      // on the leader, every reader of both CTAs: its warp 1 (PIECES: both CTAs'), and in
      // each the producers, the epilogue's and the pieces' warps
      mbar_init(&s_free[s], (PIECES ? 2 : 1) + 2 * (2 + kEpi + (PIECES ? kPieceWarps : 0)));
    }
    for (int s = 0; s < kRaw; s++) {
      mbar_init(&s_raw[s], 1);
      mbar_init(&s_raw_free[s], kPieceWarps);
    }
    mbar_init(&s_drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (warp == 1) tmem_alloc_pair(&s_tmem, kTmemCols);
  if (warp == 2 && rank == 0) make_order<kW>(s_order, p, kW ? p.mt * p.kt : p.mt);
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;

  // The i-th tile of this pair; waits for it, reads it and, once, says so.
  auto next_tile = [&](int i, Tile& ti) {
    const int s = i % kSlots;
    if (!mbar_wait_cluster(&s_have[s], (i / kSlots) & 1, abort_flag, p.status, filled)) return false;
    const int4 a = ld_shared_v4(&s_tile[s]), b = ld_shared_v4(reinterpret_cast<const int4*>(&s_tile[s]) + 1);
    ti.e = a.x, ti.m = a.y, ti.n = a.z, ti.row = a.w;
    ti.end = b.x, ti.cols = b.y, ti.blocks = b.z;
    return true;
  };
  // (after the values are there, which the branch asks for; it is always taken)
  auto have_read = [&](int i, const Tile& ti) {
    if ((ti.e | ti.blocks) >= -1) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&s_free[i % kSlots]), 0));
  };
  // one thread's, and a whole warp's
  auto take_tile = [&](int i, Tile& ti) {
    if (!next_tile(i, ti)) return false;
    have_read(i, ti);
    return ti.e >= 0;
  };
  auto take_tile_warp = [&](int i, Tile& ti) {
    if (!__all_sync(0xffffffffu, next_tile(i, ti))) return false;
    if (lane == 0) have_read(i, ti);
    return ti.e >= 0;
  };

  // Waits until the MMAs have read every stage that was filled, `stage` being the next:
  // the commits that say so arrive by themselves, in the other CTA of the pair too, and
  // neither may leave before its last one has (a stage that was never filled counts as
  // read).
  auto all_consumed = [&](int stage, uint32_t phase) {
    for (int s = 0; s < kStages; s++) {
      if (!mbar_wait(&s_empty[stage], phase ^ 1, abort_flag, p.status)) return false;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    return true;
  };

  // Parts of a tile's contraction that are summed on their own.
  auto parts_of = [](int blocks) {
    constexpr int kMost = kPart<DIR, OUT>;
    return blocks <= kMost ? 1 : (blocks + kMost - 1) / kMost;
  };
  // TMEM buffer of a part, `first` being that of the tile's first: the other one in turn,
  // or, where parts are joined there, the first keeps the sum and the others meet the
  // epilogue in the other.  The next tile begins in the one that the last part left free.
  auto buffer_of = [](int first, int part) {
    return kJoin<DIR, OUT> ? first ^ (part > 0 ? 1 : 0) : first ^ (part & 1);
  };

  if (PIECES && (warp == 0 || warp == 3)) {
    // --------------------------------- producers of the operands as they lie
    if (elect_one_lane()) {
      const bool first = warp == 0;  // of the first operand; it announces both's bytes
      constexpr uint32_t kBytes = 8 * (kRawEighth<DIR == kForward> + kRawEighth<!kW>);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; i++) {
        Tile ti;
        if (!take_tile(i, ti)) break;
        const int f0 = (first ? ti.m * BM : ti.n * BN) + (int)rank * 128;
        const int64_t w = (int64_t)ti.e * p.N;
        for (int kb = 0; kb < ti.blocks; kb++) {
          if (!mbar_wait(&s_raw_free[stage], phase ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          uint8_t* to = smem + (size_t)kStages * kStageBytes + (size_t)(2 * stage + (first ? 0 : 1)) * kRawOperand;
          const int k0 = kb * BK;
          if (first) {
            *filled = *filled + 1;
            mbar_arrive_expect_tx(&s_raw[stage], kBytes);
            if (DIR == kForward)
              copy_eighths<true>(to, maps.a, w + f0, k0, &s_raw[stage]);
            else
              copy_eighths<false>(to, maps.a, (kW ? ti.row : w) + k0, f0, &s_raw[stage]);
          } else if (kW) {
            copy_eighths<false>(to, maps.b, ti.row + k0, f0, &s_raw[stage]);
          } else {
            copy_eighths<true>(to, maps.b, ti.row + (int)rank * (ti.cols / 2), k0, &s_raw[stage]);
          }
          if (++stage == kRaw) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok || *abort_flag) settle(2000000);  // 2 ms: far longer than any single copy takes
    }
  } else if (warp == 0 || warp == 3) {
    // ------------------------------------------------------- TMA producers
    if (elect_one_lane()) {
      const bool first = warp == 0;  // of the first operand; it announces both's bytes
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_parity[kStages];
      bool issued[kStages];
      for (int s = 0; s < kStages; s++) issued[s] = false;
      bool ok = true;
      for (int i = 0; ok; i++) {
        Tile ti;
        if (!take_tile(i, ti)) break;
        const int nkb = ti.blocks;
        const int half = ti.cols / 2;  // columns of this CTA
        // first feature of this CTA, or kWeight's second operand: its first column
        const int f0 = (first ? ti.m * BM : ti.n * BN) + (int)rank * 128;
        const int row = ti.row + (int)rank * half;
        const CUtensorMap* map = first ? maps.a : kW ? maps.b : maps.b + half / 16 - 1;
        const uint32_t bytes = kW ? kStageBytes : kOperand + (uint32_t)half * BK * 2;
        const bool groups = first ? p.a_groups : p.b_groups;
        for (int kb = 0; kb < nkb; kb++) {
          if (!mbar_wait(&s_empty[stage], phase ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          uint8_t* to = smem + (size_t)stage * kStageBytes + (first ? 0 : kOperand);
          const uint32_t bar = mapa_shared(smem_u32(&s_full[stage]), 0);
          if (first) *filled = *filled + 1;
          if (first && rank == 0) mbar_arrive_expect_tx(&s_full[stage], 2 * bytes);
          const int k0 = kb * BK;
          if (kW) {
            const int from = ti.row + k0, before = min(ti.end - from - BK, 0);  // rows of zeros in front, negative
            if (groups) {
              tma_load_4d_pair(to, map, 0, before, from, f0 / 64, bar);
            } else {
              tma_load_3d_pair(to, map, f0, before, from, bar);
              tma_load_3d_pair(to + kBox, map, f0 + 64, before, from, bar);
            }
          } else if (!first) {
            tma_load_2d_pair(to, map, k0, row, bar);
          } else if (DIR == kForward) {
            tma_load_3d_pair(to, map, k0, f0, ti.e, bar);
          } else if (groups) {
            tma_load_4d_pair(to, map, 0, k0, f0 / 64, ti.e, bar);
          } else {
            tma_load_3d_pair(to, map, f0, k0, ti.e, bar);
            tma_load_3d_pair(to + kBox, map, f0 + 64, k0, ti.e, bar);
          }
          issued[stage] = true;
          issued_parity[stage] = phase;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      ok = ok && !*abort_flag;
      if (first) ok = ok && all_consumed(stage, phase);
      if (!ok) {
        if (rank == 0) {
          for (int s = 0; s < kStages; s++) {
            if (!issued[s]) continue;
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&s_full[s], issued_parity[s]) && globaltimer_ns() - t0 < kWaitLimitNs) {
            }
          }
        }
        settle(2000000);  // 2 ms: far longer than any single copy takes
      }
    }
  } else if (PIECES && rank == 1 && warp == 1) {
    // ------------------------------ tells the leader of the stages filled here
    // The warps that fill a stage arrive in their own CTA, which orders their writes
    // before this lane's one arrival in the leader, at the cluster's scope, and so before
    // the MMAs that read them (8191 x 8191 x 8192: 1584 us; each warp arriving there by
    // itself 1681; an arrival that orders accesses to global memory too 2154).
    if (elect_one_lane()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; i++) {
        Tile ti;
        if (!take_tile(i, ti)) break;
        for (int kb = 0; kb < ti.blocks; kb++) {
          if (!mbar_wait(&s_placed[stage], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_leader(mapa_shared(smem_u32(&s_full[stage]), 0));
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer (leader)
    // One elected lane waits and issues, the others stay at the end: known to be one,
    // it needs no care for others that might issue another MMA.
    if (rank == 0 && elect_one_lane()) {
      int stage = 0, acc = 0;  // acc: of the tile's first part
      uint32_t phase = 0, acc_phases = 0;
      bool ok = true;
      for (int i = 0; ok; i++) {
        Tile ti;
        if (!take_tile(i, ti)) break;
        const int nkb = ti.blocks, parts = parts_of(nkb), part = (nkb + parts - 1) / parts;
        const uint32_t idesc = idesc_16bit(BM, (uint32_t)ti.cols, std::is_same<T, __nv_bfloat16>::value, kAmn, kBmn);
        for (int kb0 = 0, done = 0; done < parts; kb0 += part, done++) {
          const int now = buffer_of(acc, done);
          if (!mbar_wait_cluster(&s_tempty[now], (acc_phases >> now & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(now * BN);
          for (int kb = kb0; kb < min(kb0 + part, nkb); kb++) {
            if (!mbar_wait_cluster(&s_full[stage], phase, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + (size_t)stage * kStageBytes), sb = sa + kOperand;
            const uint64_t adesc = kAmn ? smem_desc_sw128_mn(sa, kBox) : smem_desc_sw128(sa);
            const uint64_t bdesc = kBmn ? smem_desc_sw128_mn(sb, kBox) : smem_desc_sw128(sb);
            // a step of 16: 32 bytes of K-major rows, or 16 rows of 128 bytes
            constexpr uint64_t kAstep = kAmn ? 128 : 2, kBstep = kBmn ? 128 : 2;
            // the last stage's steps that hold anything: its first ones, or (kWeight,
            // not PIECES) those behind the zeros
            const int left = kW ? (ti.end - ti.row) - kb * BK : p.contraction - kb * BK;
            constexpr bool kZerosFirst = kW && !PIECES;
            const int begin = kZerosFirst && left < BK ? (BK - left) / 16 : 0;
#pragma unroll
            for (int k = 0; k < BK / 16; k++)
              if (kZerosFirst ? k >= begin : k * 16 < left)
                mma_bf16_pair(d_tmem, adesc + kAstep * k, bdesc + kBstep * k, idesc, kb > kb0 || k > begin ? 1u : 0u);
            mma_commit_pair(&s_empty[stage], 0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          mma_commit_pair(&s_tfull[now], 0x3);
          acc_phases ^= 1u << now;
        }
        acc = buffer_of(acc, parts - 1) ^ 1;
      }
      if (!ok || *abort_flag) {
        mma_commit_pair(&s_drain, 0x1);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&s_drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
        settle(2000000);  // the arrivals of the commits before it, in the other CTA too
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------- tiles (leader)
    if (lane == 0 && rank == 0) {
      const int64_t total = (int64_t)s_order.tiles[0] + s_order.tiles[1];
      int64_t t = p.next ? atomicAdd(p.next, 1) : cluster;
      for (int i = 0;; i++) {
        const int s = i % kSlots;
        const int64_t then = p.next ? atomicAdd(p.next, 1) : t + clusters;  // on its way meanwhile
        const Tile ti = tile_of<DIR>(t, s_order, p);
        if (!mbar_wait_cluster(&s_free[s], ((i / kSlots) & 1) ^ 1, abort_flag, p.status, filled)) break;
        for (uint32_t r = 0; r < 2; r++)
          send_32(mapa_shared(smem_u32(&s_tile[s]), r), mapa_shared(smem_u32(&s_have[s]), r),
                  make_int4(ti.e, ti.m, ti.n, ti.row), make_int4(ti.end, ti.cols, ti.blocks, 0));
        if (t >= total) break;
        t = then;
      }
    }
  } else if (PIECES && warp >= 4 + kEpi) {
    // ------------------------------------------ operands brought into place
    const int at = threadIdx.x - 32 * (4 + kEpi);
    int stage = 0, raw = 0;
    uint32_t phase = 0, raw_phase = 0;
    for (int i = 0, ok = 1; ok; i++) {
      Tile ti;
      if (!take_tile_warp(i, ti)) break;
      const int half = ti.cols / 2, f0 = ti.m * BM + (int)rank * 128, c0 = ti.n * BN + (int)rank * 128;
      Half<DIR == kForward> a;
      Half<!kW> b;
      if (kW) {
        a.begin_tile(p.a, p.sa, ti.row, f0, ti.end - ti.row, at);
        b.begin_tile(p.b, p.sb, ti.row, c0, ti.end - ti.row, at);
      } else {
        const int64_t w = (int64_t)ti.e * p.N;
        if (DIR == kForward)
          a.begin_tile(p.a, p.sa, w + f0, 0, p.contraction, at);
        else
          a.begin_tile(p.a, p.sa, w, f0, p.contraction, at);
        b.begin_tile(p.b, p.sb, ti.row + (int)rank * half, 0, p.contraction, at);
      }
      for (int kb = 0; kb < ti.blocks; kb++) {
        const bool both = mbar_wait(&s_raw[raw], raw_phase, abort_flag, p.status) &&
                          mbar_wait(&s_empty[stage], phase ^ 1, abort_flag, p.status);
        if (!__all_sync(0xffffffffu, both)) {
          ok = 0;
          break;
        }
        uint8_t* to = smem + (size_t)stage * kStageBytes;
        const uint8_t* from = smem + (size_t)kStages * kStageBytes + (size_t)(2 * raw) * kRawOperand;
        a.shift(to, from, at);
        b.shift(to + kOperand, from + kRawOperand, at);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_raw_free[raw]);
          mbar_arrive(rank == 0 ? &s_full[stage] : &s_placed[stage]);
        }
        if (++raw == kRaw) {
          raw = 0;
          raw_phase ^= 1;
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (warp == 4 + kEpi && !*abort_flag) all_consumed(stage, phase);
  } else {
    // ---------------------------------------------------------- epilogue
    const int lane_base = 32 * (warp & 3);
    const int turn_of = (warp - 4) >> 2;  // of the warps with the same lanes
    constexpr int kTurns = kEpi / 4;
    uint8_t* s_out = smem + (size_t)kStages * kStageBytes + (PIECES ? 2 * kRaw * kRawOperand : 0) +
                     (size_t)(warp - 4) * (PIECES ? 32 * kTurn * 4 : 2 * kOutBytes);  // kWeight
    int out_at = 0;
    int acc = 0;  // of the tile's first part
    uint32_t acc_phases = 0;
    // the loads from this buffer are done; stores to memory may still be on their way
    auto release = [&](int at) {
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&s_tempty[at]), 0));
    };
    bool ok = true;
    for (int i = 0; ok; i++) {
      Tile ti;
      if (!take_tile_warp(i, ti)) break;
      const int parts = parts_of(ti.blocks);
      const uint32_t tsum = tmem_base + ((uint32_t)lane_base << 16) + (uint32_t)(acc * BN);
      const int f_warp = ti.m * BM + (int)rank * 128 + lane_base;  // first feature of this warp
      for (int done = 0; done < parts; done++) {
        int there = 0;
        const int now = buffer_of(acc, done);
        if (lane == 0) there = mbar_wait(&s_tfull[now], acc_phases >> now & 1, abort_flag, p.status, filled) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, there, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        acc_phases ^= 1u << now;
        uint32_t taddr = tmem_base + ((uint32_t)lane_base << 16) + (uint32_t)(now * BN);
        if (kJoin<DIR, OUT> && parts > 1) {
          if (done) {
            for (int c = 32 * turn_of; c < ti.cols; c += 32 * kTurns) add_columns(tsum + c, taddr + c);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            release(now);
          }
          if (done < parts - 1) continue;
          taddr = tsum;
        }
        if constexpr (kW && PIECES) {
          // 32 columns of 32 rows at a time, turned in shared memory
          float* turn = reinterpret_cast<float*>(s_out);
          const bool none = ti.end == ti.row;
          const int cols = min(p.Kd - ti.n * BN, BN), rows = min(p.N - f_warp, 32);
          const int64_t first = ((int64_t)ti.e * p.N + f_warp) * p.Kd + ti.n * BN;
          for (int c = 32 * turn_of; c < cols && rows > 0; c += 32 * kTurns) {
            float v[32];
            if (none) {
#pragma unroll
              for (int j = 0; j < 32; j++) v[j] = 0.0f;
            } else {
              tmem_ld32(taddr + c, v);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; j++) turn[lane * kTurn + j] = v[j];
            __syncwarp();
            const int64_t at = first + c + lane;
            OUT* to = static_cast<OUT*>(p.out) + at;
            const int here = c + lane < cols ? rows : 0;
            if (sizeof(OUT) == 4 && done) {  // added to the parts before, in memory
#pragma unroll
              for (int r = 0; r < 32; r++, to += p.Kd)
                if (r < here) atomicAdd(reinterpret_cast<float*>(to), turn[r * kTurn + lane]);
            } else if (sizeof(OUT) == 4 && p.addend) {
              const float* add = p.addend + at;
              for (int r0 = 0; r0 < here; r0 += 8) {  // eight summands on their way before the first is stored
                float x[8];
#pragma unroll
                for (int r = 0; r < 8; r++) x[r] = r0 + r < here ? add[(int64_t)(r0 + r) * p.Kd] : 0.0f;
#pragma unroll
                for (int r = 0; r < 8; r++)
                  if (r0 + r < here) to[(int64_t)(r0 + r) * p.Kd] = from_float<OUT>(turn[(r0 + r) * kTurn + lane] + x[r]);
              }
            } else {
#pragma unroll
              for (int r = 0; r < 32; r++, to += p.Kd)
                if (r < here) *to = from_float<OUT>(turn[r * kTurn + lane]);
            }
          }
        } else if constexpr (kW) {
          // 128 bytes of this lane's row of the matrix at a time, through shared memory
          constexpr int kCols = 128 / (int)sizeof(OUT);
          const bool none = ti.end == ti.row;
          const int n = f_warp + lane;
          const float* add = p.addend && !done ? p.addend + ((int64_t)ti.e * p.N + n) * p.Kd + ti.n * BN : nullptr;
          // this part is added to the one before, once that has been written
          if (!kJoin<DIR, OUT> && done && lane == 0) bulk_wait_all();
          const int cols = min(p.Kd - ti.n * BN, BN);
          for (int c = 0; c < cols && f_warp < p.N; c += kCols) {
            uint4 piece[8];
#pragma unroll
            for (int h = 0; h < kCols / 32; h++) {
              float v[32];
              if (none) {
#pragma unroll
                for (int j = 0; j < 32; j++) v[j] = 0.0f;
              } else {
                tmem_ld32(taddr + c + h * 32, v);
              }
              if constexpr (sizeof(OUT) == 4) {
                if (add && n < p.N) {
#pragma unroll
                  for (int j = 0; j < 32; j += 4)
                    if (c + j < cols) {
                      const float4 x = *reinterpret_cast<const float4*>(add + c + j);
                      v[j] += x.x, v[j + 1] += x.y, v[j + 2] += x.z, v[j + 3] += x.w;
                    }
                }
#pragma unroll
                for (int q = 0; q < 8; q++)
                  piece[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                        __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
              } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                  piece[h * 4 + q] =
                      make_uint4(pack2<T>(v[8 * q], v[8 * q + 1]), pack2<T>(v[8 * q + 2], v[8 * q + 3]),
                                 pack2<T>(v[8 * q + 4], v[8 * q + 5]), pack2<T>(v[8 * q + 6], v[8 * q + 7]));
              }
            }
            uint8_t* buf = s_out + out_at * kOutBytes;
            if (lane == 0) bulk_wait_read<1>();  // the copy before the last has left this buffer
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; q++)
              *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) * 16)) = piece[q];
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (!kJoin<DIR, OUT> && done)
                tma_add_3d(&maps.out, buf, ti.n * BN + c, f_warp, ti.e);
              else
                tma_store_3d(&maps.out, buf, ti.n * BN + c, f_warp, ti.e);
              bulk_commit();
            }
            out_at ^= 1;
          }
        } else if constexpr (PIECES) {
          // columns are rows of the result, lanes features
          const int f = f_warp + lane;
          T* out = static_cast<T*>(p.out) + f;
          for (int c = 32 * turn_of; c < ti.cols; c += 32 * kTurns) {
            float v[32];
            tmem_ld32(taddr + c, v);
            T* to = out + (int64_t)(ti.row + c) * p.sout;
            const int left = f < p.features ? ti.end - ti.row - c : 0;
#pragma unroll
            for (int j = 0; j < 32; j++, to += p.sout)
              if (j < left) *to = from_float<T>(v[j]);
          }
        } else {
          // columns are rows of the result, lanes features: neighbouring lanes exchange
          // one of two rows, so that each stores two features of one
          const int f = f_warp + (lane & ~1);
          const bool odd = lane & 1, mine = f < p.features;
          for (int c = 32 * turn_of; c < ti.cols; c += 32 * kTurns) {
            float v[32];
            tmem_ld32(taddr + c, v);
            T* out = static_cast<T*>(p.out) + (int64_t)(ti.row + c + (odd ? 1 : 0)) * p.sout + f;
            const int64_t two = 2 * p.sout;
            const int left = mine ? ti.end - ti.row - c - (odd ? 1 : 0) : 0;  // rows from this lane's first on
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
              const uint32_t w = odd ? pack2<T>(other, v[j + 1]) : pack2<T>(v[j], other);
              if (j < left) *reinterpret_cast<uint32_t*>(out) = w;
              out += two;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        release(kJoin<DIR, OUT> ? acc : now);
      }
      acc = buffer_of(acc, parts - 1) ^ 1;
    }
  }

  if (kW && !PIECES && warp >= 4 && warp < 8 && lane == 0) bulk_wait_all();
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <GemmDir DIR, typename T, typename OUT, bool PIECES>
cudaError_t launch(const Maps& maps, TcParams p, int64_t most_tiles, cudaStream_t st) {
  constexpr size_t smem = kDynSmem<DIR, PIECES>;
  static int at_once[PerDeviceOnce::kMaxDevices];
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run([&] {
    cudaError_t r = cudaFuncSetAttribute(grouped_gemm_kernel<DIR, T, OUT, PIECES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (r != cudaSuccess) return r;
    cudaLaunchAttribute cluster = {};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = 2;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)device_sm_count() / 2 * 2);
    cfg.blockDim = dim3(kThreads<DIR, PIECES>);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(&at_once[dev], grouped_gemm_kernel<DIR, T, OUT, PIECES>, &cfg);
  });
  if (e != cudaSuccess) return e;
  const int64_t clusters = at_once[dev] < 1 ? 1 : at_once[dev] < most_tiles ? at_once[dev] : most_tiles;
  // one or two tiles each: in turn, without the counter, whose clearing takes 4 us
  if (most_tiles <= 2 * clusters) p.next = nullptr;
  if (p.next && (e = cudaMemsetAsync(p.next, 0, sizeof(int32_t), st)) != cudaSuccess) return e;
  grouped_gemm_kernel<DIR, T, OUT, PIECES><<<(unsigned)(2 * clusters), kThreads<DIR, PIECES>, smem, st>>>(maps, p);
  return cudaGetLastError();
}

template <typename T, bool PIECES>
cudaError_t run(GemmDir dir, const GroupedGemm& g, cudaStream_t st) {
  const CUtensorMapDataType type =
      g.dtype == MOE_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  TcParams p = {};
  p.offsets = g.offsets;
  p.counts = g.counts;
  p.status = g.status;
  p.out = g.out;
  p.addend = g.addend;
  p.sout = g.sout;
  p.cap = g.cap;
  p.routes = g.T * g.K;
  p.E = (int)g.E;
  p.N = (int)g.N;
  p.Kd = (int)g.Kd;
  const uint16_t *rows = static_cast<const uint16_t*>(g.a), *b = static_cast<const uint16_t*>(g.b);
  Maps maps = {};
  auto eighths = [&](CUtensorMap (&of)[8], const uint16_t* m, int64_t count, int64_t cols, int64_t stride, bool kmajor) {
    cudaError_t r = cudaSuccess;
    for (int i = 0; i < 8 && r == cudaSuccess; i++)
      r = make_tensor_map_eighth_rows(&of[i], m, type, count, cols, stride, i, kmajor ? kRawRows<true> : kRawRows<false>,
                                      (kmajor ? kRawRow<true> : kRawRow<false>) / 2);
    return r;
  };
  cudaError_t e;
  if (dir == kWeight) {
    p.mt = (int)((g.N + BM - 1) / BM);
    p.kt = (int)((g.Kd + BN - 1) / BN);
    p.next = static_cast<int32_t*>(g.workspace);
    const bool f32 = g.out_dtype == MOE_ELEM_F32;
    const int64_t tiles = g.E * p.mt * p.kt;
    if constexpr (PIECES) {
      p.a = rows, p.sa = g.sa;
      p.b = b, p.sb = g.sb;
      if (g.cap > 0) {  // (without rows no copy is made)
        if ((e = eighths(maps.a, rows, g.cap, g.N, g.sa, false)) != cudaSuccess) return e;
        if ((e = eighths(maps.b, b, g.cap, g.Kd, g.sb, false)) != cudaSuccess) return e;
      }
      return f32 ? launch<kWeight, T, float, true>(maps, p, tiles, st)
                 : launch<kWeight, T, T, true>(maps, p, tiles, st);
    }
    p.a_groups = g.N % 64 == 0;
    p.b_groups = g.Kd % 64 == 0;
    if ((e = make_tensor_map_row_windows(&maps.a[0], g.a, type, g.cap, g.N, g.sa, BK)) != cudaSuccess) return e;
    if ((e = make_tensor_map_row_windows(&maps.b[0], g.b, type, g.cap, g.Kd, g.sb, BK)) != cudaSuccess) return e;
    if ((e = make_tensor_map_matrices(&maps.out, g.out, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type, f32 ? 4 : 2, g.E, g.N,
                                      g.Kd, 32, f32 ? 32 : 64)) != cudaSuccess)
      return e;
    return f32 ? launch<kWeight, T, float, false>(maps, p, tiles, st)
               : launch<kWeight, T, T, false>(maps, p, tiles, st);
  }
  p.features = (int)(dir == kForward ? g.N : g.Kd);
  p.contraction = (int)(dir == kForward ? g.Kd : g.N);
  p.mt = (p.features + BM - 1) / BM;
  const bool fwd = dir == kForward;
  const int64_t routes = p.routes;
  const int64_t tiles = (routes / BN + (routes < g.E ? routes : g.E)) * p.mt;
  // up to 256 routes no expert has a second tile and every tile costs its weights:
  // in turn, without the counter and its clearing
  if (routes > BN) p.next = static_cast<int32_t*>(g.workspace);
  if constexpr (PIECES) {
    p.a = b, p.sa = g.Kd;
    p.b = rows, p.sb = g.sa;
    if ((e = eighths(maps.a, b, g.E * g.N, g.Kd, g.Kd, fwd)) != cudaSuccess) return e;
    if ((e = eighths(maps.b, rows, g.cap, p.contraction, g.sa, true)) != cudaSuccess) return e;
    return fwd ? launch<kForward, T, T, true>(maps, p, tiles, st)
               : launch<kData, T, T, true>(maps, p, tiles, st);
  }
  p.a_groups = !fwd && g.Kd % 64 == 0;
  e = p.a_groups ? make_tensor_map_matrix_groups(&maps.a[0], g.b, type, g.E, g.N, g.Kd, BK)
                 : make_tensor_map_matrices(&maps.a[0], g.b, type, 2, g.E, g.N, g.Kd, fwd ? 128 : BK, 64);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 8 && (i == 0 || i * 32 < routes); i++)  // a tile has no more rows than there are routes
    if ((e = make_tensor_map_rows(&maps.b[i], g.a, type, g.cap, p.contraction, g.sa, 16 * (i + 1), BK)) != cudaSuccess)
      return e;
  return fwd ? launch<kForward, T, T, false>(maps, p, tiles, st)
             : launch<kData, T, T, false>(maps, p, tiles, st);
}

}  // namespace

size_t grouped_gemm_workspace_bytes(const moe_shape& s, const moe_layout& l, int64_t N, int64_t Kd) {
  return 16;  // the tile counter
}

bool grouped_gemm_counts(const moe_shape& s, const moe_layout& l, int64_t features) {
  return (l.capacity / BN + s.E) * ((features + BM - 1) / BM) < (int64_t(1) << 30);
}

cudaError_t launch_grouped_gemm(GemmDir dir, const GroupedGemm& g, cudaStream_t st) {
  const bool copies = g.cap > 0 && g.N % 8 == 0 && g.Kd % 8 == 0 && aligned16(g.a) && aligned16(g.b) &&
                      aligned16(g.out) && aligned16(g.addend) &&
                      (g.cap == 1 || (g.sa % 8 == 0 && (dir == kWeight ? g.sb % 8 == 0 : g.sout % 8 == 0)));
  if (g.dtype == MOE_ELEM_BF16)
    return copies ? run<__nv_bfloat16, false>(dir, g, st) : run<__nv_bfloat16, true>(dir, g, st);
  return copies ? run<__half, false>(dir, g, st) : run<__half, true>(dir, g, st);
}

}  // namespace moe
