// dsa_chunk_index.cuh -- where the chunk kernels find their work: index
// arithmetic only, so that it also compiles as plain C++ and is tested without
// a GPU.
#pragma once

#include "dsa_prefix_index.cuh"

namespace dsa {

// A sequence of a chunk call: tokens s0 .. s0 + n - 1 of the batch, the last n
// entries of a list of `len`. Token i sits at list position len - n + i and
// attends positions position - window + 1 .. position (window 0: 0 .. position)
// that exist. Keys are worked in halves of 128 list positions, two halves to a
// unit; a row tile's units start at the half of its first key, so a window of
// 129 keys never takes more than a unit for one token.
struct Sequence {
  int32_t s0, n, len, window;
  DSA_HD int32_t first_half(int32_t position) const {
    return window > 0 && position >= window ? (position - window + 1) >> 7 : 0;
  }
  // Halves of the list that the sequence's units read: [gather_begin(),
  // gather_end()). A unit's second half may lie one past the list's last.
  DSA_HD bool any() const { return n > 0 && len > 0; }
  DSA_HD int32_t gather_begin() const { return first_half(len - n); }
  DSA_HD int32_t gather_end() const {
    const int32_t last = (len - 1) >> 7;
    return window > 0 ? last + 2 : (last + 2) & ~1;
  }
  // The n * H query rows in tiles of 128; tile i: its rows, its first half and
  // its units.
  DSA_HD int32_t tiles(int32_t H) const { return (int32_t)(((int64_t)n * H + 127) >> 7); }
  DSA_HD int32_t tile_rows(int32_t H, int32_t i) const {
    const int64_t left = (int64_t)n * H - 128 * (int64_t)i;
    return left < 128 ? (int32_t)left : 128;
  }
  DSA_HD int32_t row_position(int32_t H, int64_t row) const { return len - n + (int32_t)((uint32_t)row / (uint32_t)H); }
  DSA_HD int32_t tile_units(int32_t H, int32_t i, int32_t &half) const {
    const int64_t r0 = 128 * (int64_t)i;
    half = first_half(row_position(H, r0));
    const int32_t hi = row_position(H, r0 + tile_rows(H, i) - 1);
    return hi < 0 ? 0 : ((hi >> 7) + 2 - half) >> 1;
  }
};

// Row tiles and image halves that a call can need at most.
DSA_HD int64_t chunk_row_tiles(int64_t T, int64_t H, int64_t B) { return T * H / 128 + (B < T ? B : T); }
DSA_HD int64_t chunk_seq_halves(int64_t width) { return (width + 127) / 128 + 1; }

}  // namespace dsa
