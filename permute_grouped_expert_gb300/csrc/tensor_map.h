// tensor_map.h -- host-side construction of 2-D TMA tensor maps through the
// driver entry point (no link-time dependency on libcuda).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// Row-major [rows][cols] matrix of `elem_bytes`-byte elements; boxes of
// box_rows x box_cols with the 128-byte swizzle (box_cols * elem_bytes must be
// <= 128).  Out-of-range box elements read as zero.
inline cudaError_t make_tensor_map_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype,
                                      int elem_bytes, uint64_t rows, uint64_t cols, uint32_t box_rows,
                                      uint32_t box_cols, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * (uint64_t)elem_bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, dtype, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tiled map of 16-bit elements with the 128-byte swizzle; strides in bytes, of all
// dimensions but the innermost.
inline cudaError_t make_tensor_map(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int rank,
                                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                                   CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, dtype, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Bytes between the rows of a row matrix (any multiple of 16 where there is one row).
inline uint64_t row_bytes(uint64_t rows, uint64_t cols, uint64_t stride) {
  return (rows > 1 ? stride : (cols + 7) / 8 * 8) * 2;
}

// Row matrix [rows][cols] of 16-bit elements whose rows lie `stride` elements apart.
inline cudaError_t make_tensor_map_rows(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, uint64_t rows,
                                        uint64_t cols, uint64_t stride, uint32_t box_rows, uint32_t box_cols) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {row_bytes(rows, cols, stride)};
  const cuuint32_t box[2] = {box_cols, box_rows};
  return make_tensor_map(map, base, dtype, 2, dims, strides, box);
}

// The same as windows of box_rows rows, one from each row on: coordinates (column,
// row of the window, first row).  A box that begins at a negative row of its window
// has zeros in front of the rows from the first on, and ends where the window would
// go on: no row behind is read.  Boxes of 64 columns, or, where cols is a multiple of
// 64, columns in groups of 64 (their number is a fourth coordinate) and boxes of two
// groups, one after the other in shared memory.
inline cudaError_t make_tensor_map_row_windows(CUtensorMap* map, const void* base, CUtensorMapDataType dtype,
                                               uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows) {
  const bool groups = cols % 64 == 0;
  const uint64_t apart = row_bytes(rows, cols, stride);
  const cuuint64_t dims[4] = {groups ? 64 : cols, box_rows, rows, cols / 64}, strides[3] = {apart, apart, 128};
  const cuuint32_t box[4] = {64, box_rows, 1, 2};
  return make_tensor_map(map, base, dtype, groups ? 4 : 3, dims, strides, box);
}

// Every eighth row of a row matrix that starts anywhere, from row `first` on: such
// rows lie a multiple of 16 bytes apart.  The map starts at the aligned 16 bytes that
// hold the first element, so that column c of it is column c minus their distance of
// the matrix; boxes without swizzle.  Without such a row it is the first row's, which
// no result depends on then.
inline cudaError_t make_tensor_map_eighth_rows(CUtensorMap* map, const uint16_t* base, CUtensorMapDataType dtype,
                                               uint64_t rows, uint64_t cols, uint64_t stride, uint64_t first,
                                               uint32_t box_rows, uint32_t box_cols) {
  if (first >= rows) first = 0;
  const uintptr_t at = reinterpret_cast<uintptr_t>(base + first * stride), start = at & ~uintptr_t(15);
  const uint64_t count = (rows - first + 7) / 8, width = (at - start) / 2 + cols;
  const cuuint64_t dims[2] = {width, count}, strides[1] = {count > 1 ? stride * 16 : (width + 7) / 8 * 16};
  const cuuint32_t box[2] = {box_cols, box_rows};
  return make_tensor_map(map, reinterpret_cast<const void*>(start), dtype, 2, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Matrices [count][rows][cols] of 16-bit elements, contiguous, columns in groups of
// 64: boxes of two groups of box_rows rows of one matrix.
inline cudaError_t make_tensor_map_matrix_groups(CUtensorMap* map, const void* base, CUtensorMapDataType dtype,
                                                 uint64_t count, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const cuuint64_t dims[4] = {64, rows, cols / 64, count}, strides[3] = {cols * 2, 128, rows * cols * 2};
  const cuuint32_t box[4] = {64, box_rows, 2, 1};
  return make_tensor_map(map, base, dtype, 4, dims, strides, box);
}

// Matrices [count][rows][cols], contiguous; boxes within one matrix.
inline cudaError_t make_tensor_map_matrices(CUtensorMap* map, const void* base, CUtensorMapDataType dtype,
                                            int elem_bytes, uint64_t count, uint64_t rows, uint64_t cols,
                                            uint32_t box_rows, uint32_t box_cols) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {cols, rows, count};
  cuuint64_t strides[2] = {cols * elem_bytes, rows * cols * elem_bytes};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, dtype, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace moe
