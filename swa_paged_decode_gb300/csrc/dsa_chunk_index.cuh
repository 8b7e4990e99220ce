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

// What the lay-out leaves of a row tile; without units none of its rows has a key.
struct RowTile {
  int32_t g0, rows, units;     // first row, rows
  int32_t half, key0, shift;   // as in TileRun, of the tile's first unit
};
// Its place: those with units first, in order, so that the pairs' ranges meet no
// other one (a pair that looked for the next tile with units waited for its
// record: 240 us against 235 for a window of 128); `live`: tiles with units,
// live_before: of them before tile t.
DSA_HD int32_t tile_place(int32_t t, int32_t units, int64_t live_before, int64_t live) {
  return (int32_t)(units > 0 ? live_before : live + (t - live_before));
}

// The pairs whose ranges begin in a tile of `units` > 0 units: of C equal shares
// of `total` those that begin within the tile's cost, units + tile_cost from `at`
// on. f(pair, unit) for each of them, in order.
template <class F>
DSA_KERNEL void pairs_in_tile(int64_t at, int32_t units, int64_t tile_cost, int64_t total, int32_t C, F f) {
  const int64_t next = at + units + tile_cost;
  for (int64_t c = (at * C + total - 1) / total; c < C; ++c) {   // the first with at <= total c / C
    const int64_t x = total * c / C, unit = x - at - tile_cost;
    if (x >= next) break;
    f((int32_t)c, unit > 0 ? (int32_t)unit : 0);
  }
}

// A pair's range, from unit w of row tile t to before unit w1 of tile t1, tile
// by tile, all of them with units; load(t, tile) reads a row tile. peek names the
// tile that next returns.
template <class Load>
struct TileWalk {
  Load load;
  int32_t t, w, t1, w1;
  RowTile tile;   // row tile t, loaded ahead
  DSA_KERNEL TileWalk(Load l, int32_t t_, int32_t w_, int32_t t1_, int32_t w1_) : load(l), t(t_), w(w_), t1(t1_), w1(w1_), tile() {
    ahead();
  }
  DSA_KERNEL bool empty() const { return t > t1 || (t == t1 && w >= w1); }
  DSA_KERNEL void ahead() {   // (loaded, not looked at: a role would wait for it)
    if (t < t1 || (t == t1 && w1 > 0)) load(t, tile);
  }
  DSA_KERNEL bool next(TileRun &s) {
    if (empty()) return false;
    const int32_t end = t == t1 ? w1 : tile.units;
    s.qt = t;
    s.g0 = tile.g0;
    s.n = tile.rows;
    s.half = tile.half + 2 * w;
    s.key0 = tile.key0 + 256 * w;
    s.shift = tile.shift;
    s.units = end - w;
    s.head = w == 0;
    s.tail = end == tile.units;
    ++t;
    w = 0;
    ahead();
    return true;
  }
  // rows of the next segment's tile (0: none)
  DSA_KERNEL int32_t peek(const TileRun &, int64_t &g0) const {
    g0 = tile.g0;
    return empty() ? 0 : tile.rows;
  }
};

// Row tiles and image halves that a call can need at most.
DSA_HD int64_t chunk_row_tiles(int64_t T, int64_t H, int64_t B) { return T * H / 128 + (B < T ? B : T); }
DSA_HD int64_t chunk_seq_halves(int64_t width) { return (width + 127) / 128 + 1; }

}  // namespace dsa
