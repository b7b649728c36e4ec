// mxfp4_tile_plan.h — which columns, weight rows and buffers a workgroup of the tiled MXFP4
// products (mxfp4_tile.hip) works on. Plain arithmetic without HIP's headers, so that the tests
// walk it on the CPU.
#pragma once

namespace coli {

constexpr int MX_CUS = 256;
constexpr int EXP_STRIP = 2;  // column tiles of a workgroup over a route

__host__ __device__ inline int tile_min(int a, int b) { return a < b ? a : b; }

// A workgroup runs a strip of column tiles one after another, its weight rows worked out for the
// first: strips of `strip` whole tiles of BF columns. A last tile of fewer columns is a strip of
// its own, since only the first tile's rows are held within the matrix.
__host__ __device__ inline int tile_strips(int N, int BF, int strip) {
  return (N / BF + strip - 1) / strip + (N % BF != 0);
}
// Strip i: tiles first .. first + cols - 1
__host__ __device__ inline void strip_tiles(int N, int BF, int strip, int i, int &first, int &cols) {
  const int whole = N / BF;
  first = tile_min(i * strip, whole);
  cols = first < whole ? tile_min(strip, whole - first) : 1;
}

// Weight row of column r of a strip's first tile, relative to that tile's first column col0. Gate/up:
// by eights, gate rows, then the up rows of the same features.
__host__ __device__ inline int tile_weight_row(bool gate_up, int r, int N, int col0) {
  if (gate_up) return (r >> 3 & 1) * N + tile_min((r >> 4) * 8 + (r & 7), N - 1 - col0);
  return tile_min(r, N - 1 - col0);
}

// Column tiles of a dense workgroup: `slots` workgroups run at a time, and a strip's start and
// end cost about a third of a tile.
inline int dense_strip(int N, int BF, int ny, int slots) {
  int best = 1;
  double cost = 1e300;
  for (int s = 1; s <= 8 && s <= (N + BF - 1) / BF; s++) {
    const long long groups = (long long)tile_strips(N, BF, s) * ny;
    const double c = (double)((groups + slots - 1) / slots) * (s + 0.33);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

}  // namespace coli
