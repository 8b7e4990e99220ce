// The index arithmetic of dsa_chunk_index.cuh behind C functions.
#include "dsa_chunk_index.cuh"

extern "C" {
int seq_any(int n, int len, int window) { return dsa::Sequence{0, n, len, window}.any(); }
int gather_begin(int n, int len, int window) { return dsa::Sequence{0, n, len, window}.gather_begin(); }
int gather_end(int n, int len, int window) { return dsa::Sequence{0, n, len, window}.gather_end(); }
int seq_tiles(int n, int len, int window, int H) { return dsa::Sequence{0, n, len, window}.tiles(H); }
int tile_rows(int n, int len, int window, int H, int i) { return dsa::Sequence{0, n, len, window}.tile_rows(H, i); }
int tile_units(int n, int len, int window, int H, int i, int *half) {
  return dsa::Sequence{0, n, len, window}.tile_units(H, i, *half);
}
long long most_row_tiles(long long T, long long H, long long B) { return dsa::chunk_row_tiles(T, H, B); }
long long most_halves(long long width) { return dsa::chunk_seq_halves(width); }
}
