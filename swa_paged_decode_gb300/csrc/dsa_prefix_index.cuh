// dsa_prefix_index.cuh -- where the shared-prefix kernels find their work:
// index arithmetic only, so that it also compiles as plain C++ and is tested
// without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DSA_HD __host__ __device__ __forceinline__
#define DSA_KERNEL __device__ __forceinline__   // (calls back into code of the device only)
#else
#define DSA_HD inline
#define DSA_KERNEL inline
#endif

namespace dsa {

// Units are (row tile, key tile) pairs, row tile major, R x KT of them. Pair c
// owns [begin(c), begin(c + 1)): equal shares of the cost, a unit's 1 and, for
// a row tile that starts within the range, tile_cost = 2 for its Q staging,
// first scores and epilogue (a range that starts within a tile pays these too,
// but so does every range). With 2048 rows x 4096 keys (3.4 units to a pair)
// the attend kernel took 31 us without that and 24 us with it; 3, 4 or 6 gave
// nothing more. With fewer than 2 units to a pair a whole unit more or less
// counts for more, and a tile's start costs nothing (16.3 against 11.8 us at 2
// units for 2 pairs). A pair may own nothing; with no key tiles every one does.
struct Schedule {
  int32_t R, KT, C, tile_cost;
  DSA_HD int64_t total() const { return (int64_t)R * (KT + tile_cost); }
  // a / b for a, b >= 0, in 32 bits where they do
  static DSA_HD int64_t div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
  }
  DSA_HD int64_t begin(int32_t c) const {
    if (KT == 0) return 0;   // (an empty prefix: no units, and no tile to divide by)
    const int64_t x = div(total() * c, C), t = div(x, KT + tile_cost), w = x - t * (KT + tile_cost) - tile_cost;
    return t * KT + (w > 0 ? w : 0);
  }
};

DSA_HD Schedule make_schedule(int32_t R, int32_t KT, int32_t C) {
  return {R, KT, C, (int64_t)R * KT >= 2 * (int64_t)C ? 2 : 0};
}

// A run of units of one row tile that a pair works on.
struct TileRun {
  int32_t qt;         // row tile
  int64_t g0;         // its first row
  int32_t n;          // its rows, 1..128
  int64_t half;       // image half at which the first unit starts
  int32_t units;
  bool head, tail;    // begins, ends with the tile
  int32_t key0;       // chunk: list position of the first unit's first key,
  int32_t shift;      // and of a row g's token less g / H
};
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
