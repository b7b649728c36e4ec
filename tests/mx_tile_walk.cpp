// The plan of the tiled MXFP4 products (csrc/mxfp4_tile_plan.h), walked on the CPU for
// tests/test_mxfp4_tile_plan.py.
#define __host__
#define __device__
#include "mxfp4_tile_plan.h"

using namespace coli;

extern "C" {

int dense_strip_of(int N, int BF, int ny, int slots) { return dense_strip(N, BF, ny, slots); }

// Every weight row that the tiles of a product load: -1 if a row is outside the matrix (of N, for
// gate/up 2 N rows), -2 if the strips do not cover each column tile once, else the rows loaded past
// a tile's columns again.
int walk_rows(int gate_up, int N, int BN, int strip) {
  const int BF = gate_up ? BN / 2 : BN, nx = (N + BF - 1) / BF, rows = gate_up ? 2 * N : N;
  int next = 0, again = 0;
  for (int i = 0; i < tile_strips(N, BF, strip); i++) {
    int first, cols;
    strip_tiles(N, BF, strip, i, first, cols);
    if (first != next || cols < 1 || cols > strip) return -2;
    next += cols;
    for (int c = 0; c < cols; c++)
      for (int r = 0; r < BN; r++) {
        const int row = (first + c) * BF + tile_weight_row(gate_up, r, N, first * BF);
        if (row < 0 || row >= rows) return -1;
        // what the epilogue takes column r for
        const int want = (first + c) * BF + (gate_up ? (r >> 4) * 8 + (r & 7) : r);
        if (want < N && row != want + (gate_up && (r >> 3 & 1) ? N : 0)) return -3;
        again += want >= N;
      }
  }
  return next == nx ? again : -2;
}
}
