// mxfp4_tile_plan.h — which columns, weight rows and buffers a workgroup of the tiled MXFP4
// products (mxfp4_tile.hip) works on. Plain arithmetic without HIP's headers, so that the tests
// walk it on the CPU.
#pragma once

namespace coli {

constexpr int MX_CUS = 256;

// BM x BN tile, WM x WN wavefronts, NBUF K stages of 8 blocks (256 inputs) in LDS, OCC workgroups per CU
template <int BM_, int BN_, int WM_, int WN_, int NBUF_, int OCC_, bool WIDE_ = true>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NBUF = NBUF_, OCC = OCC_;
  static constexpr int KB = 8, KS = 4;                          // blocks of a stage, its K steps of 64 inputs
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;    // 32 x 32 tiles of a wavefront
  static constexpr int ROWS = BM + BN;
  static constexpr int LA = BM / 32, LB = BN / 32;              // 16-byte loads of a wavefront per stage (8 rows each)
  // Scales. WIDE: a window of 16 bytes of a row serves two stages (rows of 16 blocks or more);
  // it is loaded with the first (with the second its loads are empty) and NSB windows are held.
  // Else: the two dwords of a stage with the stage.
  static constexpr bool WIDE = WIDE_;
  static constexpr int NSB = 1 + NBUF / 2;
  static constexpr int RA = BM / 4, RB = BN / 4;                // scale rows of a wavefront
  static constexpr int LS = WIDE ? 2 : 4;
  static constexpr int STAGE = ROWS * (KB * 16 + (WIDE ? 0 : 8));  // LDS bytes: codes, then two planes of dwords
  static constexpr int WINDOWS = NBUF * STAGE;                     // offset of the windows
  static constexpr int IDS = WINDOWS + (WIDE ? NSB * ROWS * 16 : 0);  // offset of the row ids
  static constexpr int BYTES = IDS + BM * 4;
  static_assert(LB % 2 == 0 && RA <= 64 && RB <= 64);
};

typedef TileShape<256, 256, 2, 2, 2, 1> TileDense;
typedef TileShape<128, 128, 1, 4, 2, 2> TileDenseSmall;
typedef TileShape<128, 256, 1, 4, 3, 1> TileExperts;
typedef TileShape<128, 256, 1, 4, 3, 1, false> TileExpertsShort;  // fewer than 16 blocks in a row

// A place in the stages of a workgroup's column tiles, of nst stages each, one after another: the
// loads' and, NBUF - 1 stages behind, the products'.
template <typename S>
struct TilePlace {
  int stage = 0, slot = 0, win = 0;  // stage of the column tile, its buffer and (WIDE) scale window
  __host__ __device__ bool advance(int nst) {  // true: on to the next column tile
    slot = slot == S::NBUF - 1 ? 0 : slot + 1;
    stage++;
    const bool wrap = stage == nst;
    if ((stage & 1) == 0 || wrap) win = win == S::NSB - 1 ? 0 : win + 1;
    if (wrap) stage = 0;
    return wrap;
  }
};

// Column tiles of a workgroup over a route, rows of nb blocks: two, but one where an odd number of
// stages with scale windows ends in a window of one stage. Three windows are live at the way to a
// next column tile then, two are held (a third passes the LDS), and the first of the next tile would
// be filled while other wavefronts still read the window it replaces. Strips of 1 and 2: gate/up of
// 2048 tokens over 256 experts of 6144 x 2048 822 and 825 us, down 613 and 598.
template <typename S>
inline int expert_strip(int nb) {
  const int nst = (nb + S::KB - 1) / S::KB;
  return S::WIDE && (nst & 1) ? 1 : 2;
}

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
