// mxfp4_tile.hip — MXFP4 x MXFP4 products of many rows: LDS-tiled GEMMs on the scaled
// 32x32x64 matrix instruction of gfx950, dense and grouped over a route (batch-union:
// colibri-strix README, "What's implemented").
#include "mxfp4_impl.h"

namespace coli {

// 64 lanes x 16 (4) bytes from each lane's global address to consecutive LDS bytes at the
// wave-uniform address lds. Written as asm because the compiler would wait for every such
// load before the next LDS read; the kernel counts them itself. No register is loaded.
__device__ __forceinline__ void dma16(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void dma4(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the last N loads of this wavefront have arrived
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Waits until at most `ahead` stages (0 .. NBUF - 1, the same in every lane) are still on their way.
template <typename S>
__device__ __forceinline__ void wait_stages(int ahead) {
  static_assert(S::NBUF <= 4 && 3 * S::LOADS <= 63, "vmcnt");
  if (ahead >= 3) wait_loads<3 * S::LOADS>();
  else if (ahead == 2) wait_loads<2 * S::LOADS>();
  else if (ahead == 1) wait_loads<S::LOADS>();
  else wait_loads<0>();
}

template <int SA, int SB>
__device__ __forceinline__ v16f mx_mfma32(uint4 a, uint32_t ua, uint4 b, uint32_t ub, v16f c) {
  const v8i32 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i32 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SA, (int)ua, SB, (int)ub);
}

template <int BM_, int BN_, int WM_, int WN_, int NBUF_>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NBUF = NBUF_;
  static constexpr int KB = 4;                                 // blocks of a K stage: 128 inputs
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;   // 32 x 32 tiles of a wavefront
  static constexpr int ROWS = BM + BN;
  static constexpr int LA = BM / 64, LB = BN / 64;             // 16-byte loads of a wavefront per stage
  static constexpr int LS = (ROWS + 255) / 256;                // 4-byte loads
  static constexpr int LOADS = LA + LB + LS;
  static constexpr int STAGE = ROWS * KB * 16 + LS * 1024;     // LDS bytes: codes, then a scale dword per row
  static constexpr int BYTES = NBUF * STAGE;
};

// Slot of 16-byte chunk c of an LDS row: permuted so that the rows that one LDS access reads
// at the same chunk fall on different banks.
__device__ __forceinline__ int tile_swizzle(int row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); }

template <MxMode MODE, typename T, typename S>
__global__ __launch_bounds__(256, 1) void mx_tile_kernel(MxArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int BM = S::BM, BN = S::BN, MI = S::MI, NI = S::NI, NBUF = S::NBUF;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / S::WN, wn = wv % S::WN;
  const int nb = a.K / 32, nbp = mx_padded(a.K) / 32, nst = (nb + 3) / 4;
  constexpr int BF = MODE == MX_GATEUP ? BN / 2 : BN;  // output columns of a tile
  const int n0 = blockIdx.x * BF;

  // the rows of activations: first .. first + n - 1 of perm, or of the tokens
  int e = 0, first = 0, n = 0;
  bool routed = false;
  if constexpr (MODE == MX_LINEAR) {
    first = blockIdx.y * BM;
    n = min(BM, a.M - first);
  } else {
    if ((int)blockIdx.y >= *a.ntiles) return;
    const int4 c = a.tiles[blockIdx.y];
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

  // loads of this wavefront: 16 rows of 64 bytes each; lane l: row l / 4, slot l % 4
  const int lr = lane >> 2, chunk = (lane & 3) ^ tile_swizzle(lr);
  uint32_t oa[S::LA], ob[S::LB], os[S::LS];
#pragma unroll
  for (int i = 0; i < S::LA; i++) oa[i] = (uint32_t)(act_row((wv * S::LA + i) * 16 + lr) - ar0) * (uint32_t)(nbp * 16) + chunk * 16;
#pragma unroll
  for (int i = 0; i < S::LB; i++) ob[i] = (uint32_t)(w_row((wv * S::LB + i) * 16 + lr) - wr0) * (uint32_t)(nb * 16);
#pragma unroll
  for (int i = 0; i < S::LS; i++) {
    const int r = i * 256 + wv * 64 + lane;  // BM is a multiple of 64: a wavefront's rows are of one side
    os[i] = r < BM ? (uint32_t)(act_row(r) - ar0) * (uint32_t)nbp
                   : (uint32_t)(w_row(min(r, S::ROWS - 1) - BM) - wr0) * (uint32_t)a.ws_pitch;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  // load q of stage s, into the buffer that stage s - NBUF had
  auto issue = [&](int s, int q) {
    const uint32_t buf = lds0 + (s % NBUF) * S::STAGE;
    if (q < S::LA) {
      dma16(ac + s * 64, oa[q], buf + (wv * S::LA + q) * 1024);
    } else if (q < S::LA + S::LB) {
      const int i = q - S::LA;
      // weight blocks past K repeat the last one: they meet activations of zero
      dma16(wc, ob[i] + min(s * 4 + chunk, nb - 1) * 16, buf + BM * 64 + (wv * S::LB + i) * 1024);
    } else {
      const int i = q - S::LA - S::LB, r0 = i * 256 + wv * 64;
      dma4((r0 < BM ? as : ws) + s * 4, os[i], buf + S::ROWS * 64 + r0 * 4);
    }
  };

  v16f acc[MI][NI] = {};
  const int li = lane & 31, hh = lane >> 5;
  const int ra = wm * (BM / S::WM) + li, rb = wn * (BN / S::WN) + li;
  uint4 fa[2][MI], fb[2][NI];
  uint32_t sa[MI], sb[NI], sa_next[MI], sb_next[NI];
  auto read = [&](int s, int t) {  // fragments of K step t (64 inputs) of stage s
    const uint8_t *buf = lds + (s % NBUF) * S::STAGE;
    const int c = ((2 * t + hh) ^ tile_swizzle(li)) * 16;
#pragma unroll
    for (int i = 0; i < MI; i++) fa[t][i] = *reinterpret_cast<const uint4 *>(buf + (ra + i * 32) * 64 + c);
#pragma unroll
    for (int j = 0; j < NI; j++) fb[t][j] = *reinterpret_cast<const uint4 *>(buf + (BM + rb + j * 32) * 64 + c);
  };
  auto read_scales = [&](int s) {  // a dword: the four blocks of the stage
    const uint32_t *p = reinterpret_cast<const uint32_t *>(lds + (s % NBUF) * S::STAGE + S::ROWS * 64);
#pragma unroll
    for (int i = 0; i < MI; i++) sa_next[i] = p[ra + i * 32];
#pragma unroll
    for (int j = 0; j < NI; j++) sb_next[j] = p[BM + rb + j * 32];
  };
  auto take_scales = [&]() {  // bytes 0 and 2: this lane's blocks of K steps 0 and 1
#pragma unroll
    for (int i = 0; i < MI; i++) sa[i] = sa_next[i] >> (8 * hh);
#pragma unroll
    for (int j = 0; j < NI; j++) sb[j] = sb_next[j] >> (8 * hh);
  };

  // Stages s + 1 .. s + NBUF - 1 are on their way while stage s is multiplied. A stage's second
  // K step is in registers before its buffer is given up, and is multiplied while the loads of
  // stage s + NBUF and the first fragments of stage s + 1 are under way. Steps of one body per
  // number of stages ahead (AHEAD, -1: the last stage): a branch inside would let the compiler
  // move the first K step's products behind the wait.
  auto step = [&]<int AHEAD, bool ISSUE>(int s) {
    read(s, 1);
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
      for (int j = 0; j < NI; j++) acc[i][j] = mx_mfma32<0, 0>(fa[0][i], sa[i], fb[0][j], sb[j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (AHEAD >= 0) {
      wait_loads<AHEAD * S::LOADS>();  // stage s + 1 has arrived; stage s is in registers
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    // products and loads take turns: a burst of loads would leave the matrix cores without work
#pragma unroll
    for (int q = 0; q < (MI * NI > S::LOADS + 2 ? MI * NI : S::LOADS + 2); q++) {
      __builtin_amdgcn_sched_barrier(0);
      const int i = q / NI, j = q % NI;
      if (q < MI * NI) acc[i][j] = mx_mfma32<2, 2>(fa[1][i], sa[i], fb[1][j], sb[j], acc[i][j]);
      if constexpr (AHEAD >= 0) {
        if (q == 0) read_scales(s + 1);
        if (q == 1) read(s + 1, 0);
        if (ISSUE && q >= 2 && q < S::LOADS + 2) issue(s + NBUF, q - 2);
      }
    }
    if constexpr (AHEAD >= 0) take_scales();
  };
  static_assert(NBUF == 4, "the tail below");
#pragma unroll
  for (int s = 0; s < NBUF; s++)
    if (s < nst) {
#pragma unroll
      for (int q = 0; q < S::LOADS; q++) issue(s, q);
    }
  wait_stages<S>(min(nst, NBUF) - 1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read_scales(0);
  read(0, 0);
  take_scales();
  int s = 0;
  for (; s + NBUF < nst; s++) step.template operator()<2, true>(s);
  if (nst - s > 3) step.template operator()<2, false>(s++);
  if (nst - s > 2) step.template operator()<1, false>(s++);
  if (nst - s > 1) step.template operator()<0, false>(s++);
  step.template operator()<-1, false>(s);

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
  hipLaunchKernelGGL(kernel, dim3((unsigned)((a.N + BF - 1) / BF), (unsigned)ny), dim3(256), S::BYTES, s, a);
  return hipGetLastError();
}

typedef TileShape<256, 256, 2, 2, 4> TileDense;
typedef TileShape<128, 256, 1, 4, 4> TileExperts;

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
  if (mode == MX_GATEUP) return launch_tile<MX_GATEUP, T, TileExperts>(a, cap, s);
  return launch_tile<MX_DOWN, float, TileExperts>(a, cap, s);
}

hipError_t launch_mx_tile(MxMode mode, int dtype, const MxArgs &a, hipStream_t s) {
  if (dtype == COLI_F32) return launch_tile_t<float>(mode, a, s);
  if (dtype == COLI_BF16) return launch_tile_t<bf16_t>(mode, a, s);
  return launch_tile_t<f16_t>(mode, a, s);
}

}  // namespace coli
