// dsa_prefix_index.cuh -- where the shared-prefix kernels find their work:
// index arithmetic only, so that it also compiles as plain C++ and is tested
// without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DSA_HD __host__ __device__ __forceinline__
#else
#define DSA_HD inline
#endif

namespace dsa {

// The parts of a query row: the pairs c0..c1 whose ranges meet its row tile
// (none: c1 < c0, an empty prefix). The partial of pair c lies in the pair's
// first 128 rows when the tile is its first, else in its second 128 (`late`:
// only c0 can have begun before the tile). A pair without units has left -inf
// in its first rows.
struct RowParts {
  int32_t c0, c1, late, row;   // late: 0 or 128; row: of the tile's 128
  DSA_HD int32_t count() const { return c1 - c0 + 1; }
  DSA_HD int64_t slot(int32_t i) const { return (int64_t)(c0 + i) * 256 + (i == 0 ? late : 0) + row; }
  // The partial that is loaded for part i, ahead of knowing whether it counts:
  // the last one again past the end, and one of the workspace where there is
  // none at all (that load is left out).
  DSA_HD int64_t loaded(int32_t i) const {
    const int32_t last = count() - 1, j = i < last ? i : last;
    return slot(j > 0 ? j : 0);
  }
};

}  // namespace dsa
