// The index arithmetic of the shared-prefix kernels as a plain library, for
// tests without a GPU.
#include "dsa_prefix_index.cuh"

extern "C" int64_t part_loaded(int32_t c0, int32_t c1, int32_t late, int32_t row, int32_t i) {
  return dsa::RowParts{c0, c1, late, row}.loaded(i);
}
extern "C" int64_t part_slot(int32_t c0, int32_t c1, int32_t late, int32_t row, int32_t i) {
  return dsa::RowParts{c0, c1, late, row}.slot(i);
}
extern "C" int64_t schedule_begin(int32_t R, int32_t KT, int32_t C, int32_t c) {
  return dsa::make_schedule(R, KT, C).begin(c);
}
