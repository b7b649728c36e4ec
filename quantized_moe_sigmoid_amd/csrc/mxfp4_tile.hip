// mxfp4_tile.hip — MXFP4 x MXFP4 products of many rows: LDS-tiled GEMMs on the scaled
// 32x32x64 matrix instruction of gfx950, dense and grouped over a route (batch-union:
// colibri-strix README, "What's implemented").
#include "mxfp4_impl.h"

namespace coli {

// 16 (4) bytes from each lane's global address to consecutive LDS bytes at the wave-uniform
// address lds, for the lanes of the mask hi : lo. Written as asm because the compiler would wait for every
// such load before the next LDS read; the kernel counts them itself. No register is loaded. A
// load whose mask is empty moves nothing and is counted like the others.
__device__ __forceinline__ void dma16(const uint8_t *base, uint32_t off, uint32_t lds, int lo, int hi) {
  asm volatile(
      "s_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1" ::"s"(
          lds),
      "v"(off), "s"(base), "s"(lo), "s"(hi)
      : "memory");
}
__device__ __forceinline__ void dma4(const uint8_t *base, uint32_t off, uint32_t lds, int lo, int hi) {
  asm volatile(
      "s_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2\n\ts_mov_b64 exec, -1" ::"s"(
          lds),
      "v"(off), "s"(base), "s"(lo), "s"(hi)
      : "memory");
}
__device__ __forceinline__ void dma16(uint64_t addr, uint32_t lds, int lo, int hi) {  // an address of each lane's own
  asm volatile("s_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %3\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, -1" ::"s"(
                   lds),
               "v"(addr), "s"(lo), "s"(hi)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the last N loads of this wavefront have arrived
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int BM_, int BN_, int WM_, int WN_, int KB_, int NBUF_, int OCC_, bool WIDE_ = true>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;  // tile; wavefronts along its rows and columns
  static constexpr int KB = KB_, KS = KB / 2;                   // blocks of a K stage, its K steps of 64 inputs
  static constexpr int NBUF = NBUF_, OCC = OCC_;                // stages in LDS; workgroups per CU
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;    // 32 x 32 tiles of a wavefront
  static constexpr int ROWS = BM + BN;
  static constexpr int RPL = 64 / KB;                           // rows of a 16-byte load (64 lanes)
  static constexpr int LA = BM / 4 / RPL, LB = BN / 4 / RPL;    // 16-byte loads of a wavefront per stage
  // Scales. WIDE: a window of 16 bytes of a row serves QN = 16 / KB stages (rows of 16 blocks or
  // more); it is loaded in QN parts, one with each stage, and NSB windows are held. Else: the
  // dwords of a stage with the stage.
  static constexpr bool WIDE = WIDE_;
  static constexpr int QN = 16 / KB, RQ = ROWS / (4 * QN);      // parts of a window, rows of a wavefront in one
  static constexpr int NSB = 2 + (NBUF - 2 + QN - 1) / QN;      // the window after next starts before this one ends
  static constexpr int LR = (ROWS + 255) / 256, LS = WIDE ? 1 : LR * (KB / 4);
  static constexpr int LOADS = LA + LB + LS;
  static constexpr int STAGE = ROWS * KB * 16 + (WIDE ? 0 : LS * 1024);  // LDS bytes: codes, then planes of dwords
  static constexpr int WINDOWS = NBUF * STAGE;                           // offset of the windows
  static constexpr int BYTES = WINDOWS + (WIDE ? NSB * ROWS * 16 : 0);
};

template <int SA, int SB>
__device__ __forceinline__ v16f mx_mfma32(uint4 a, uint32_t ua, uint4 b, uint32_t ub, v16f c) {
  const v8i32 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i32 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SA, (int)ua, SB, (int)ub);
}

// Slot of 16-byte chunk c of an LDS row of KB chunks is c ^ swizzle: the rows that one LDS
// access reads at the same chunk fall on different banks.
template <int KB>
__device__ __forceinline__ int tile_swizzle(int row) {
  return KB == 4 ? ((row >> 1) & 3) ^ ((row >> 3) & 1) : row & 7;
}

// Workgroup id -> tile (x of nx, y of ny) of a dense product. Consecutive ids go to different
// XCDs (id % 8); each XCD gets a run of tiles in strips of TILE_STRIP columns, so that the
// tiles it works on at a time share rows and columns in its L2.
constexpr int TILE_STRIP = 4;
__device__ __forceinline__ void tile_of(int id, int nx, int ny, int &x, int &y) {
  const int n = nx * ny, xcd = id & 7, q = n >> 3, r = n & 7;
  const int t = xcd * q + min(xcd, r) + (id >> 3);
  const int strip = t / (TILE_STRIP * ny), in = t - strip * TILE_STRIP * ny;
  const int w = min(TILE_STRIP, nx - strip * TILE_STRIP);
  y = in / w;
  x = strip * TILE_STRIP + in - y * w;
}

template <MxMode MODE, typename T, typename S>
__global__ __launch_bounds__(256, S::OCC) void mx_tile_kernel(MxArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int BM = S::BM, BN = S::BN, MI = S::MI, NI = S::NI, NBUF = S::NBUF, KB = S::KB, KS = S::KS;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / S::WN, wn = wv % S::WN;
  const int nb = a.K / 32, nbp = mx_padded(a.K) / 32, nst = (nb + KB - 1) / KB;
  constexpr int BF = MODE == MX_GATEUP ? BN / 2 : BN;  // output columns of a tile
  int bx = blockIdx.x, by = blockIdx.y;
  if constexpr (MODE == MX_LINEAR) tile_of(blockIdx.x, (a.N + BF - 1) / BF, (a.M + BM - 1) / BM, bx, by);
  const int n0 = bx * BF;

  // the rows of activations: first .. first + n - 1 of perm, or of the tokens
  int e = 0, first = 0, n = 0;
  bool routed = false;
  if constexpr (MODE == MX_LINEAR) {
    first = by * BM;
    n = min(BM, a.M - first);
  } else {
    if (by >= *a.ntiles) return;
    const int4 c = a.tiles[by];
    e = c.x;
    first = c.y;
    n = c.z;
    routed = c.w != 0;
  }
  const int64_t P = (int64_t)a.M * a.k;
  auto act_row = [&](int i) -> int64_t {  // row of activations of tile row i
    const int ci = first + min(i, n - 1);
    if constexpr (MODE == MX_LINEAR) return ci;
    const int64_t pair = routed ? a.perm[ci] : P + ci;
    return MODE == MX_DOWN ? pair : (routed ? pair / a.k : ci);
  };
  auto w_row = [&](int r) -> int {  // weight row of tile column r
    if constexpr (MODE == MX_GATEUP) {
      constexpr int WT = BN / S::WN;
      const int rr = r % WT, m = rr / (WT / 2);
      return m * a.N + min(n0 + (r / WT) * (WT / 2) + rr % (WT / 2), a.N - 1);
    }
    return min(n0 + r, a.N - 1);
  };
  const uint8_t *wc = a.wc + (int64_t)e * a.wc_stride, *ws = a.ws + (int64_t)e * a.ws_stride;
  // tile-relative bases keep the lanes' offsets within 32 bits
  const int wr0 = MODE == MX_GATEUP ? 0 : n0, ar0 = MODE == MX_LINEAR ? first : 0;
  const uint8_t *ac = a.ac + (int64_t)ar0 * nbp * 16, *as = a.as + (int64_t)ar0 * nbp;
  wc += (int64_t)wr0 * nb * 16;
  ws += (int64_t)wr0 * a.ws_pitch;

  // loads of this wavefront: RPL rows of KB chunks each; lane l: row l / KB, slot l % KB
  constexpr int RPL = S::RPL;
  const int lr = lane / KB, chunk = (lane % KB) ^ tile_swizzle<KB>(lr);
  uint32_t oa[S::LA], ob[S::LB], os[S::LR];
  uint64_t pw[S::QN];  // scale rows of this lane
#pragma unroll
  for (int i = 0; i < S::LA; i++) oa[i] = (uint32_t)(act_row((wv * S::LA + i) * RPL + lr) - ar0) * (uint32_t)(nbp * 16) + chunk * 16;
#pragma unroll
  for (int i = 0; i < S::LB; i++) ob[i] = (uint32_t)(w_row((wv * S::LB + i) * RPL + lr) - wr0) * (uint32_t)(nb * 16);
  if constexpr (S::WIDE) {
#pragma unroll
    for (int q = 0; q < S::QN; q++) {
      const int r = (q * 4 + wv) * S::RQ + min(lane, S::RQ - 1);
      const uint8_t *p = r < BM ? as + (act_row(r) - ar0) * nbp : ws + (int64_t)(w_row(r - BM) - wr0) * a.ws_pitch;
      pw[q] = reinterpret_cast<uint64_t>(p);
    }
  } else
#pragma unroll
  for (int i = 0; i < S::LR; i++) {
    const int r = i * 256 + wv * 64 + lane;  // BM is a multiple of 64: a wavefront's rows are of one side
    os[i] = r < BM ? (uint32_t)(act_row(r) - ar0) * (uint32_t)nbp
                   : (uint32_t)(w_row(min(r, S::ROWS - 1) - BM) - wr0) * (uint32_t)a.ws_pitch;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int wlast = a.ws_pitch - 16;  // the last window ends with the row
  auto window = [&](int u, int q, int on) {  // part q of scale window u
    uint64_t p = pw[0];
#pragma unroll
    for (int i = 1; i < S::QN; i++) {
      const uint64_t m = -(uint64_t)(q == i);  // (a select here becomes an array in memory)
      p = (p & ~m) | (pw[i] & m);
    }
    const uint32_t dst = lds0 + S::WINDOWS + (u % S::NSB) * (S::ROWS * 16) + (q * 4 + wv) * (S::RQ * 16);
    constexpr uint64_t lanes = ~0ull >> (64 - S::RQ);
    dma16(p + min(16 * u, wlast), dst, on & (int)lanes, on & (int)(lanes >> 32));
  };
  // load q of stage s (an empty one past the last), into the buffer that stage s - NBUF had
  auto issue = [&](int s, int q) {
    const int on = __builtin_amdgcn_readfirstlane(s < nst ? -1 : 0);
    const uint32_t buf = lds0 + (s % NBUF) * S::STAGE;
    if (q < S::LA) {
      dma16(ac + s * (KB * 16), oa[q], buf + (wv * S::LA + q) * 1024, on, on);
    } else if (q < S::LA + S::LB) {
      const int i = q - S::LA;
      // weight blocks past K repeat the last one: they meet activations of zero
      dma16(wc, ob[i] + min(s * KB + chunk, nb - 1) * 16, buf + BM * (KB * 16) + (wv * S::LB + i) * 1024, on, on);
    } else if constexpr (S::WIDE) {
      window((s + S::QN - 1) / S::QN, (s + S::QN - 1) % S::QN, on);  // stage 0 completes window 0
    } else {
      const int i = (q - S::LA - S::LB) % S::LR, d = (q - S::LA - S::LB) / S::LR, r0 = i * 256 + wv * 64;
      // a dword past the row's scales is replaced by its last: nb is a multiple of 4 or the rows are padded
      const int b = r0 < BM ? s * KB + 4 * d : min(s * KB + 4 * d, a.ws_pitch - 4);
      dma4((r0 < BM ? as : ws) + b, os[i], buf + S::ROWS * (KB * 16) + d * (S::LR * 1024) + r0 * 4, on, on);
    }
  };

  v16f acc[MI][NI] = {};
  const int li = lane & 31, hh = lane >> 5;
  const int ra = wm * (BM / S::WM) + li, rb = wn * (BN / S::WN) + li;
  uint4 fa[2][MI], fb[2][NI];
  uint32_t sa[KB / 4][MI], sb[KB / 4][NI], sa_next[KB / 4][MI], sb_next[KB / 4][NI];
  auto read = [&](int s, int t) {  // fragments of K step t of stage s
    const uint8_t *buf = lds + (s % NBUF) * S::STAGE;
    const int c = ((2 * t + hh) ^ tile_swizzle<KB>(li)) * 16;
#pragma unroll
    for (int i = 0; i < MI; i++) fa[t & 1][i] = *reinterpret_cast<const uint4 *>(buf + (ra + i * 32) * (KB * 16) + c);
#pragma unroll
    for (int j = 0; j < NI; j++)
      fb[t & 1][j] = *reinterpret_cast<const uint4 *>(buf + (BM + rb + j * 32) * (KB * 16) + c);
  };
  auto read_scales = [&](int s) {  // a dword: four blocks of a row
#pragma unroll
    for (int d = 0; d < KB / 4; d++) {
      const uint8_t *p;
      constexpr int step = S::WIDE ? 16 : 4;  // bytes between rows
      if constexpr (S::WIDE) {
        const int u = s / S::QN, at = s * KB + 4 * d - min(16 * u, wlast);  // past the row's end: its last dword
        p = lds + S::WINDOWS + (u % S::NSB) * (S::ROWS * 16) + min(at, 12);
      } else {
        p = lds + (s % NBUF) * S::STAGE + S::ROWS * (KB * 16) + d * (S::LR * 1024);
      }
#pragma unroll
      for (int i = 0; i < MI; i++) sa_next[d][i] = *reinterpret_cast<const uint32_t *>(p + (ra + i * 32) * step);
#pragma unroll
      for (int j = 0; j < NI; j++) sb_next[d][j] = *reinterpret_cast<const uint32_t *>(p + (BM + rb + j * 32) * step);
    }
  };
  auto take_scales = [&]() {  // bytes 0 and 2: this lane's blocks of two K steps
#pragma unroll
    for (int d = 0; d < KB / 4; d++) {
#pragma unroll
      for (int i = 0; i < MI; i++) sa[d][i] = sa_next[d][i] >> (8 * hh);
#pragma unroll
      for (int j = 0; j < NI; j++) sb[d][j] = sb_next[d][j] >> (8 * hh);
    }
  };
  auto mul = [&](int t, int i, int j) {
    acc[i][j] = t & 1 ? mx_mfma32<2, 2>(fa[1][i], sa[t / 2][i], fb[1][j], sb[t / 2][j], acc[i][j])
                      : mx_mfma32<0, 0>(fa[0][i], sa[t / 2][i], fb[0][j], sb[t / 2][j], acc[i][j]);
  };

  // Stages s + 1 .. s + NBUF - 1 are on their way while stage s is multiplied. A stage's last K
  // step is in registers before its buffer is given up, and is multiplied while the loads of
  // stage s + NBUF and the first fragments of stage s + 1 are under way. The body has no branch:
  // the compiler would move products across it, behind the wait.
  if constexpr (S::WIDE)
#pragma unroll
    for (int q = 0; q < S::QN - 1; q++) window(0, q, -1);
#pragma unroll
  for (int s = 0; s < NBUF; s++)
#pragma unroll
    for (int q = 0; q < S::LOADS; q++) issue(s, q);
  static_assert((NBUF - 1) * S::LOADS <= 63, "vmcnt");
  wait_loads<(NBUF - 1) * S::LOADS>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read_scales(0);
  read(0, 0);
  take_scales();
  for (int s = 0; s < nst; s++) {
#pragma unroll
    for (int t = 0; t < KS - 1; t++) {
      read(s, t + 1);
#pragma unroll
      for (int q = 0; q < MI * NI; q++) mul(t, q / NI, q % NI);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_loads<(NBUF - 2) * S::LOADS>();  // stage s + 1 has arrived; stage s is in registers
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // products and loads take turns: a burst of loads would leave the matrix cores without work
    constexpr int TURNS = MI * NI > 3 ? MI * NI : 3, PER = (S::LOADS + TURNS - 3) / (TURNS - 2);
#pragma unroll
    for (int q = 0; q < TURNS; q++) {
      __builtin_amdgcn_sched_barrier(0);
      if (q < MI * NI) mul(KS - 1, q / NI, q % NI);
      if (q == 0) read_scales(s + 1);  // past the last stage: not used
      if (q == 1) read(s + 1, 0);
#pragma unroll
      for (int p = (q - 2) * PER; p < (q - 1) * PER; p++)
        if (p >= 0 && p < S::LOADS) issue(s + NBUF, p);
    }
    take_scales();
  }

  // results: lane column li of a tile, rows 8 (r / 4) + 4 hh + r % 4
#pragma unroll
  for (int i = 0; i < MI; i++)
#pragma unroll
    for (int r = 0; r < 16; r++) {
      const int row = wm * (BM / S::WM) + i * 32 + 8 * (r / 4) + 4 * hh + (r & 3);
      if (row >= n) continue;
      const int ci = first + row;
      const int64_t orow = MODE == MX_LINEAR ? ci : (routed ? (int64_t)a.perm[ci] : P + ci);
      if constexpr (MODE == MX_GATEUP) {
#pragma unroll
        for (int j = 0; j < NI / 2; j++) {
          const int col = n0 + wn * (BN / S::WN / 2) + j * 32 + li;
          if (col < a.N) static_cast<T *>(a.out)[orow * a.N + col] = (T)(silu(acc[i][j][r]) * acc[i][j + NI / 2][r]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NI; j++) {
          const int col = n0 + wn * (BN / S::WN) + j * 32 + li;
          if (col < a.N) static_cast<T *>(a.out)[orow * a.N + col] = (T)acc[i][j][r];
        }
      }
    }
}

// Tiles of a route: {expert, first (of perm, or token), rows, routed}, the shared expert's first.
__global__ __launch_bounds__(1024) void mx_plan_kernel(MxArgs a, int bm, int cap) {
  __shared__ int wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int na = max(0, min(*a.nact, a.E));
  const int shared = a.has_shared ? (a.M + bm - 1) / bm : 0;
  int e = 0, first = 0, n = 0;
  if (tid < na) {
    e = a.active[tid];
    first = a.off[e];
    n = a.off[e + 1] - first;
  }
  const int mine = (n + bm - 1) / bm;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 63) wsum[wv] = incl;
  __syncthreads();
  int base = shared, total = shared;
  for (int i = 0; i < 16; i++) {
    if (i < wv) base += wsum[i];
    total += wsum[i];
  }
  for (int c = tid; c < shared && c < cap; c += 1024) a.tiles[c] = make_int4(a.E, c * bm, min(bm, a.M - c * bm), 0);
  int g = base + incl - mine;
  for (int c = 0; c < mine; c++, g++)
    if (g < cap) a.tiles[g] = make_int4(e, first + c * bm, min(bm, n - c * bm), 1);
  if (tid == 0) *a.ntiles = min(total, cap);
}

template <MxMode MODE, typename T, typename S>
static hipError_t launch_tile(const MxArgs &a, int ny, hipStream_t s) {
  static_assert(S::BYTES <= 160 * 1024, "LDS");
  constexpr int BF = MODE == MX_GATEUP ? S::BN / 2 : S::BN;
  auto kernel = mx_tile_kernel<MODE, T, S>;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
  if (attr != hipSuccess) return attr;
  const unsigned nx = (unsigned)((a.N + BF - 1) / BF);
  const dim3 g = MODE == MX_LINEAR ? dim3(nx * (unsigned)ny) : dim3(nx, (unsigned)ny);
  hipLaunchKernelGGL(kernel, g, dim3(256), S::BYTES, s, a);
  return hipGetLastError();
}

#ifndef TD
#define TD 256, 256, 2, 2, 4, 4, 1
#endif
#ifndef TE
#define TE 128, 256, 1, 4, 4, 4, 1
#endif
typedef TileShape<TD> TileDense;
typedef TileShape<TE> TileExperts;
typedef TileShape<TE, false> TileExpertsShort;  // fewer than 16 blocks in a row

int64_t mx_tile_cap(int32_t T, int32_t k, int32_t E, int32_t has_shared) {
  const int64_t P = (int64_t)T * k, bm = TileExperts::BM;
  return P / bm + (P < E ? P : E) + (has_shared ? (T + bm - 1) / bm : 0);
}

template <typename T>
static hipError_t launch_tile_t(MxMode mode, const MxArgs &a, hipStream_t s) {
  if (mode == MX_LINEAR) return launch_tile<MX_LINEAR, T, TileDense>(a, (a.M + TileDense::BM - 1) / TileDense::BM, s);
  const int cap = (int)mx_tile_cap(a.M, a.k, a.E, a.has_shared);
  hipLaunchKernelGGL(mx_plan_kernel, dim3(1), dim3(1024), 0, s, a, TileExperts::BM, cap);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  const bool wide = a.K >= 512;
  if (mode == MX_GATEUP)
    return wide ? launch_tile<MX_GATEUP, T, TileExperts>(a, cap, s) : launch_tile<MX_GATEUP, T, TileExpertsShort>(a, cap, s);
  return wide ? launch_tile<MX_DOWN, float, TileExperts>(a, cap, s) : launch_tile<MX_DOWN, float, TileExpertsShort>(a, cap, s);
}

hipError_t launch_mx_tile(MxMode mode, int dtype, const MxArgs &a, hipStream_t s) {
  if (dtype == COLI_F32) return launch_tile_t<float>(mode, a, s);
  if (dtype == COLI_BF16) return launch_tile_t<bf16_t>(mode, a, s);
  return launch_tile_t<f16_t>(mode, a, s);
}

}  // namespace coli
