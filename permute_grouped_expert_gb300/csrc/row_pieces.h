// row_pieces.h -- which rows of a matrix may be read in whole 16-byte pieces
// (host code).
#pragma once

#include <cstdint>

namespace moe {

// Rows that lie `stride` elements apart are read as the aligned pieces of n
// elements that hold them. The last piece of a row holds up to n - 1 elements
// behind it: the next rows', or, where fewer than n - 1 elements of the matrix
// follow, from behind the matrix. Returns the first such row; from it on a piece
// that is not the row's alone is read element by element.
inline int64_t first_cut_row(int64_t rows, int64_t stride, int n) {
  if (rows <= 1) return 0;
  const int64_t cut = (n - 1 + stride - 1) / stride;
  return rows > cut ? rows - cut : 0;
}

}  // namespace moe
