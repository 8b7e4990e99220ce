// A batch laid out as the chunk kernels lay it out, one tile after the other, and
// every pair's range walked as their roles walk it (dsa_chunk_index.cuh).
#include <vector>

#include "dsa_chunk_index.cuh"

using namespace dsa;

// -> 0, or what is wrong: 1 a segment that peek did not name before, 2 a segment
// outside its tile or without units, 3 a unit of a tile that not exactly one pair
// takes, 4 head or tail marks that do not meet the segment's ends, 5 a walk that
// does not end, 6 units for a tile's keyless rows alone, 7 two tiles in one
// place.
extern "C" int walk_batch(int B, const int *n, const int *len, int window, int H, int C) {
  std::vector<RowTile> all;
  int32_t s0 = 0;
  const int32_t seq_halves = 1 << 16;
  for (int b = 0; b < B; ++b) {
    const Sequence s = {s0, n[b], len[b], window};
    for (int32_t i = 0; i < s.tiles(H); ++i) {
      int32_t half;
      const int32_t units = s.tile_units(H, i, half);
      const int32_t last = s.row_position(H, 128 * (int64_t)i + s.tile_rows(H, i) - 1);
      if ((units > 0) != (last >= 0)) return 6;
      all.push_back({s0 * H + 128 * i, s.tile_rows(H, i), units, b * seq_halves + half, half * 128, s.len - s.n - s0});
    }
    s0 += n[b];
  }
  int64_t units = 0, live = 0;
  for (const RowTile &t : all) {
    units += t.units;
    live += t.units > 0;
  }
  const int64_t tile_cost = units >= 2 * (int64_t)C ? 2 : 0, total = units + tile_cost * live;
  const int32_t R = (int32_t)all.size();
  std::vector<RowTile> tiles(R);
  std::vector<int> filled(R, 0);
  std::vector<int32_t> from(C + 1, 0), at_unit(C + 1, 0);
  from[C] = (int32_t)live;
  int64_t at = 0, before = 0;
  for (int32_t t = 0; t < R; ++t) {
    const int32_t to = tile_place(t, all[t].units, before, live);
    if (to < 0 || to >= R || filled[to]++) return 7;
    tiles[to] = all[t];
    if (all[t].units == 0) continue;
    ++before;
    pairs_in_tile(at, all[t].units, tile_cost, total, C, [&](int32_t c, int32_t unit) {
      from[c] = to;
      at_unit[c] = unit;
    });
    at += all[t].units + tile_cost;
  }
  std::vector<std::vector<int>> taken(R);
  for (int32_t t = 0; t < R; ++t) taken[t].assign(tiles[t].units, 0);
  auto load = [&](int32_t t, RowTile &r) { r = tiles.at(t); };
  for (int c = 0; c < C; ++c) {
    TileWalk<decltype(load)> walk(load, from[c], at_unit[c], from[c + 1], at_unit[c + 1]);
    TileRun seg = {};
    int64_t g0 = -1;
    int32_t rows = walk.peek(seg, g0);
    if ((rows > 0) == walk.empty()) return 1;
    for (int32_t steps = 0; walk.next(seg); ++steps) {
      if (steps > R) return 5;
      if (seg.g0 != g0 || seg.n != rows) return 1;
      const RowTile &t = tiles.at(seg.qt);
      const int32_t w = (int32_t)(seg.half - t.half) / 2;
      if (seg.g0 != t.g0 || seg.n != t.rows || seg.shift != t.shift || seg.units < 1 || w < 0 || w + seg.units > t.units ||
          seg.key0 != t.key0 + 256 * w)
        return 2;
      if (seg.head != (w == 0) || seg.tail != (w + seg.units == t.units)) return 4;
      for (int32_t u = w; u < w + seg.units; ++u) taken[seg.qt][u]++;
      rows = walk.peek(seg, g0);
    }
    if (rows != 0) return 1;
  }
  for (const auto &t : taken)
    for (int k : t)
      if (k != 1) return 3;
  return 0;
}
