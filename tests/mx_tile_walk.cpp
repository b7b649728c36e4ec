// The plan of the tiled MXFP4 products (csrc/mxfp4_tile_plan.h), walked on the CPU for
// tests/test_mxfp4_tile_plan.py.
#define __host__
#define __device__
#include "mxfp4_tile_plan.h"

using namespace coli;

// The buffers and scale windows of a workgroup's `cols` column tiles of nst stages. Barriers cut the
// work into intervals; wavefronts differ by less than one. Interval 0 loads stages 0 .. NBUF - 2
// and the codes' first part of stage NBUF - 1; interval n + 1 multiplies stage n: it reads its
// codes and (at its start) its scales, loads the rest of stage n + NBUF - 1, its scales among it,
// and before that, behind the barrier that ended stage n - 1, the first codes of the same stage.
// 0 if no stage's data is overwritten in the interval that reads it or before, and the products'
// place finds what the loads' place wrote; else the failing rule.
template <typename S>
static int walk_stages(int nst, int cols) {
  const int total = nst * cols;
  TilePlace<S> in[512];
  if (total >= 512) return -1;
  for (int m = 0; m + 1 < total; m++) {
    in[m + 1] = in[m];
    if (in[m + 1].advance(nst) != (in[m + 1].stage == 0)) return 1;
  }
  TilePlace<S> out;  // the products' place
  for (int n = 0; n < total; n++) {
    if (out.slot != in[n].slot || out.win != in[n].win || out.stage != in[n].stage) return 2;
    const int w = n - (in[n].stage & 1);  // the stage whose loads brought its window
    if (in[w].win != in[n].win) return 3;
    for (int m = 0; m < total; m++) {
      const int scales_in = m < S::NBUF - 1 ? 0 : m - S::NBUF + 2, codes_in = m < S::NBUF ? 0 : m - S::NBUF + 2;
      if (m > n && in[m].slot == in[n].slot && codes_in <= n + 1) return 4;
      if (!S::WIDE || (in[m].stage & 1) || in[m].win != in[n].win) continue;
      if (m > w && scales_in <= n + 1) return 5;  // refilled while, or before, stage n's scales are read
    }
    out.advance(nst);
  }
  return 0;
}

extern "C" {

int walk_dense(int nst, int cols) { return walk_stages<TileDense>(nst, cols); }
int walk_dense_small(int nst, int cols) { return walk_stages<TileDenseSmall>(nst, cols); }
int walk_experts(int nst, int cols) { return walk_stages<TileExperts>(nst, cols); }
int walk_experts_short(int nst, int cols) { return walk_stages<TileExpertsShort>(nst, cols); }
int strip_experts(int nb) { return expert_strip<TileExperts>(nb); }
int strip_experts_short(int nb) { return expert_strip<TileExpertsShort>(nb); }

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
