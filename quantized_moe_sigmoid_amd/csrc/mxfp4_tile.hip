// mxfp4_tile.hip — MXFP4 x MXFP4 products of many rows: LDS-tiled GEMMs on the scaled
// 32x32x64 matrix instruction of gfx950, dense and grouped over a route (batch-union:
// colibri-strix README, "What's implemented").
//
// y = sum over blocks of 2^(ua - 127) 2^(uw - 127) sum a_i w_i: the instruction takes both
// operands' codes and their E8M0 bytes, so a block costs no work of the vector units.
//
// Dense, M = 4096, N = 12288, K = 6144 bf16: 178 to 185 us (3.3 to 3.5 PFLOP/s). The instruction
// on random codes in registers alone reaches 6.1 to 6.4 PFLOP/s here (9.2 on zeros: the card's
// power, not the issue rate, is the limit), which is 100 us; without its products the kernel
// takes 145, without scales too 132: the tile's way through L2 and LDS and the matrix cores each
// take most of the time, and overlap in part. 256 x 256 tiles need 32 bytes a clock and CU at the
// full rate, close to what whole 128-byte lines reach (36; 64-byte pieces 22), hence stages of
// 256 inputs, one row of a stage to a line. A wavefront's 128 x 128 part fills the accumulators.
//
// Over a route, 2048 tokens, 256 experts of 6144 x 2048, Zipf-like: gate/up 815 us, down 480 (and
// 96 for the combine). Bound by the weights' way from HBM: 3.4 GB, of which the kernel fetches
// 3.9 (a line of scale bytes comes back for every two stages). Measured when the whole took 825:
// without products 804, without scales 749; 8 wavefronts to the tile 851 (with two stages in LDS
// instead of three 960), two workgroups of 128 x 128 tiles to a CU 857; column strips of 1, 2, 3
// and 4 tiles 822, 825, 855 and 869 us for gate/up, 613, 598, 599 and 599 for down.
#include <type_traits>

#include "mxfp4_impl.h"
#include "mxfp4_tile_plan.h"

namespace coli {

// Loads of 64 lanes straight into LDS: 16 (4) bytes from each lane's address base + off to
// consecutive LDS bytes at the wave-uniform address lds; the pair: two, 4096 LDS bytes apart
// (the instruction's offset moves both addresses, so o0 is 4096 high). Lanes outside hi : lo
// load nothing, and a load without lanes is counted like the others. Written as asm because
// the compiler would wait for every such load before the next LDS read; the kernel counts them
// itself. No register is loaded; M0 and the active lanes are put back.
__device__ __forceinline__ uint64_t lanes_of(int lo, int hi) {  // in scalar registers
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(hi) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane(lo);
}
__device__ __forceinline__ void dma16_pair(const uint8_t *base, uint32_t o0, uint32_t o1, uint32_t lds, int lo, int hi) {
  uint64_t active;
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %1, m0\n\ts_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\t"
      "global_load_lds_dwordx4 %4, %6 offset:-4096\n\tglobal_load_lds_dwordx4 %5, %6\n\t"
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %0"
      : "=&s"(active), "=&s"(m0)
      : "s"(lds + 4096), "s"(lanes_of(lo, hi)), "v"(o0), "v"(o1), "s"(base)
      : "memory", "scc");
}
__device__ __forceinline__ void dma16(const uint8_t *base, uint32_t off, uint32_t lds, int lo, int hi) {
  uint64_t active;
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %1, m0\n\ts_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\tglobal_load_lds_dwordx4 %4, %5\n\t"
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %0"
      : "=&s"(active), "=&s"(m0)
      : "s"(lds), "s"(lanes_of(lo, hi)), "v"(off), "s"(base)
      : "memory", "scc");
}
__device__ __forceinline__ void dma4(const uint8_t *base, uint32_t off, uint32_t lds, int lo, int hi) {
  uint64_t active;
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %1, m0\n\ts_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\tglobal_load_lds_dword %4, %5\n\t"
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %0"
      : "=&s"(active), "=&s"(m0)
      : "s"(lds), "s"(lanes_of(lo, hi)), "v"(off), "s"(base)
      : "memory", "scc");
}

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the last N loads of this wavefront have arrived
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef uint32_t v2u32 __attribute__((ext_vector_type(2)));
typedef uint32_t v4u32 __attribute__((ext_vector_type(4)));

template <int S>
__device__ __forceinline__ v16f mx_mfma32(uint4 a, uint32_t ua, uint4 b, uint32_t ub, v16f c) {  // byte S of the scales
  const v8i32 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i32 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)ua, S, (int)ub);
}

// Slot of chunk (block) c of an LDS row of eight is c ^ swizzle: the rows that one LDS access
// reads at the same chunk fall on different banks.
__device__ __forceinline__ int tile_swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

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

template <typename W>
__device__ __forceinline__ void store_out(W w, __amdgpu_buffer_rsrc_t out, uint32_t off) {
  if constexpr (sizeof(W) == 16)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32, w), out, off, 0, 0);
  else if constexpr (sizeof(W) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, w), out, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, w), out, off, 0, 0);
}

// RAGGED: N is no multiple of the columns of a 16-byte piece
template <MxMode MODE, typename T, typename S, bool RAGGED>
__global__ __launch_bounds__(256, S::OCC) void mx_tile_kernel(MxArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int BM = S::BM, BN = S::BN, MI = S::MI, NI = S::NI, NBUF = S::NBUF, KB = S::KB, KS = S::KS;
  constexpr int BF = MODE == MX_GATEUP ? BN / 2 : BN;  // output columns of a tile
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / S::WN, wn = wv % S::WN;
  const int nb = a.K / 32, nbp = mx_padded(a.K) / 32, nst = (nb + KB - 1) / KB;
  const int ns = tile_strips(a.N, BF, a.strip);

  // the rows of activations: first .. first + n - 1 of perm, or of the tokens; and the column
  // tiles bx .. bx + cols - 1, one after another
  int bx, by, cols, e = 0, first = 0, n = 0;
  bool routed = false;
  if constexpr (MODE == MX_LINEAR) {
    int sx;
    tile_of(blockIdx.x, ns, (a.M + BM - 1) / BM, sx, by);
    strip_tiles(a.N, BF, a.strip, sx, bx, cols);
    first = by * BM;
    n = min(BM, a.M - first);
  } else {
    // Each XCD (id % 8) gets a run of (group of an expert's row tiles, column strip, row tile),
    // the row tile fastest: the workgroups that read the same weights run next to each other on
    // one XCD and share them in its L2; the strips of a group share its activations there.
    const int nt = *a.ntiles, xcd = blockIdx.x & 7, total = nt * ns;
    const int q = total >> 3, r = total & 7, local = blockIdx.x >> 3;
    if (local >= q + (xcd < r)) return;
    const int t = xcd * q + min(xcd, r) + local;
    by = t / ns;
    int4 c = a.tiles[by];
    const int grp = c.w >> 16, b0 = by - ((c.w >> 8) & 0xFF), in = t - b0 * ns;
    strip_tiles(a.N, BF, a.strip, in / grp, bx, cols);
    by = min(b0 + in % grp, nt - 1);
    c = a.tiles[by];
    e = c.x;
    first = c.y;
    n = c.z;
    routed = (c.w & 1) != 0;
  }
  const int64_t P = (int64_t)a.M * a.k;
  // tile row i -> row of the output, of the activations
  int *ids = reinterpret_cast<int *>(lds + S::IDS);
  if constexpr (MODE != MX_LINEAR) {
    for (int i = threadIdx.x; i < BM; i += 256) {
      const int ci = first + min(i, n - 1);
      ids[i] = routed ? a.perm[ci] : (int)(P + ci);
    }
    __syncthreads();
  }
  auto out_row = [&](int i) -> int { return MODE == MX_LINEAR ? i : ids[i]; };  // relative to the buffer below
  // the output from its first row on (of a dense product: the tile's); offsets fit in 32 bits
  const int64_t rows = MODE == MX_LINEAR ? n : P + (a.has_shared ? a.M : 0);
  const auto out = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<T *>(a.out) + (MODE == MX_LINEAR ? (int64_t)first * a.N : 0), 0, (int)(uint32_t)(rows * a.N * sizeof(T)),
      0x00027000);
  auto act_row = [&](int i) -> int {  // relative to the base below
    if constexpr (MODE == MX_LINEAR) return min(i, n - 1);
    return MODE == MX_DOWN ? ids[i] : (routed ? ids[i] / a.k : ids[i] - (int)P);
  };
  auto w_row = [&](int r) -> int {  // weight row of column r of the first tile, relative to the base below
    return tile_weight_row(MODE == MX_GATEUP, r, a.N, bx * BF);
  };
  // tile-relative bases keep the lanes' offsets within 32 bits
  const uint8_t *ac = a.ac, *as = a.as;
  if constexpr (MODE == MX_LINEAR) ac += (int64_t)first * nbp * 16, as += (int64_t)first * nbp;
  const uint8_t *wc = a.wc + (int64_t)e * a.wc_stride + (int64_t)bx * BF * nb * 16;
  const uint8_t *ws = a.ws + (int64_t)e * a.ws_stride + (int64_t)bx * BF * a.ws_pitch;

  // code load i of this wavefront: rows (4 i + wv) 8 .. + 7; lane l: row l / 8, slot l % 8
  const int lr = lane >> 3, chunk = (lane & 7) ^ tile_swizzle(8 * wv + lr);
  uint32_t oa[S::LA], ob[S::LB];
#pragma unroll
  for (int i = 0; i < S::LA; i++)
    oa[i] = (uint32_t)act_row((4 * i + wv) * 8 + lr) * (uint32_t)(nbp * 16) + chunk * 16 + (i & 1 ? 0 : 4096);
#pragma unroll
  for (int i = 0; i < S::LB; i++)
    ob[i] = (uint32_t)w_row((4 * i + wv) * 8 + lr) * (uint32_t)(nb * 16) + chunk * 16 + (i & 1 ? 0 : 4096);
  // weight blocks past K repeat the row's last one: they meet activations of zero
  const uint32_t past_k = max((nst - 1) * KB + chunk - (nb - 1), 0) * 16;
  const int srow = min(lane, S::RA - 1), wrow = min(lane, S::RB - 1);
  const uint32_t osa = (uint32_t)act_row(wv * S::RA + srow) * (uint32_t)nbp;
  const uint32_t osb = (uint32_t)w_row(wv * S::RB + wrow) * (uint32_t)a.ws_pitch;
  constexpr uint64_t LANES_A = ~0ull >> (64 - S::RA), LANES_B = ~0ull >> (64 - S::RB);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int wlast = a.ws_pitch - 16;  // the last window ends with the row

  auto run = [&]<int MX>() {  // with MX 32-row tiles to a wavefront
    // The loads run ahead of the products, over the stages of all column tiles, of the one whose
    // weights start at pb.
    TilePlace<S> ahead;
    int left = cols * nst;
    const uint8_t *pb = wc, *psb = ws;
    int on = -1;            // 0 once every stage is under way: the loads are empty
    uint32_t past = 0;      // past_k at a row's last stage
    auto issue_start = [&]() {
      on = __builtin_amdgcn_readfirstlane(-left >> 31);
      past = ahead.stage == nst - 1 ? past_k : 0u;
    };
    constexpr int NA = S::WM == 1 ? MX : S::LA, QA = (NA + 1) / 2, QB = S::LB / 2;  // the codes' loads go in pairs; an odd one alone
    auto issue = [&](int q) {  // load or pair q of the stage
      const int si = ahead.stage;
      const uint32_t buf = lds0 + ahead.slot * S::STAGE;
      if (q < QA) {
        const uint32_t dst = buf + (8 * q + wv) * 1024;
        if (2 * q + 1 < NA)
          dma16_pair(ac + si * (KB * 16), oa[2 * q], oa[2 * q + 1], dst, on, on);
        else
          dma16(ac + si * (KB * 16) - 4096, oa[2 * q], dst, on, on);
      } else if (q < QA + QB) {
        const int i = q - QA;
        dma16_pair(pb + si * (KB * 16), ob[2 * i] - past, ob[2 * i + 1] - past,
                   buf + BM * (KB * 16) + (8 * i + wv) * 1024, on, on);
      } else if constexpr (S::WIDE) {
        const uint32_t dst = lds0 + S::WINDOWS + ahead.win * (S::ROWS * 16);
        const int at = min(si * KB, wlast);
        const int fresh = on & ((si & 1) - 1);  // the first of the window's two stages
        if (q == QA + QB)
          dma16(as + at, osa, dst + wv * (S::RA * 16), fresh & (int)LANES_A, fresh & (int)(LANES_A >> 32));
        else
          dma16(psb + at, osb, dst + (BM + wv * S::RB) * 16, fresh & (int)LANES_B, fresh & (int)(LANES_B >> 32));
      } else {
        const int i = q - QA - QB, d = i & 1;
        const uint32_t dst = buf + S::ROWS * (KB * 16) + d * (S::ROWS * 4);
        // a dword past the row's scales is replaced by its last
        if (i < 2)
          dma4(as + si * KB + 4 * d, osa, dst + wv * (S::RA * 4), on & (int)LANES_A, on & (int)(LANES_A >> 32));
        else
          dma4(psb + min(si * KB + 4 * d, a.ws_pitch - 4), osb, dst + (BM + wv * S::RB) * 4, on & (int)LANES_B, on & (int)(LANES_B >> 32));
      }
    };
    constexpr int ISSUES = QA + QB + S::LS, LOADS = NA + S::LB + S::LS;
    static_assert((NBUF - 1) * LOADS <= 63, "vmcnt");
    // The first EARLY issues of a stage go out in the K step after the barrier, the others in the
    // next one. With three buffers there is time: a quarter early 811 us for gate/up of 2048
    // tokens, half 816, all 825; with two (dense) half: the same as all, a quarter 2 % slower.
    constexpr int EARLY = NBUF > 2 ? ISSUES / 4 : ISSUES / 2;
    static_assert(EARLY <= QA + QB, "scale windows are filled one barrier later than codes");
    constexpr int EARLY_LOADS = EARLY <= QA ? (EARLY * 2 < NA ? EARLY * 2 : NA)
                              : EARLY <= QA + QB ? NA + (EARLY - QA) * 2 : NA + S::LB + (EARLY - QA - QB);
    auto issue_end = [&]() {
      left--;
      if (ahead.advance(nst)) {
        pb += (int64_t)BF * nb * 16;
        psb += (int64_t)BF * a.ws_pitch;
      }
    };

    v16f acc[MX][NI];
    const int li = lane & 31, hh = lane >> 5;
    // K step t takes block t of a stage in lanes 0-31 and block 4 + t in lanes 32-63, so that a
    // lane's scales are the four bytes of one dword
    uint32_t ra[KS], rb[KS];
#pragma unroll
    for (int t = 0; t < KS; t++) {
      const int c = ((t + 4 * hh) ^ tile_swizzle(li)) * 16;
      ra[t] = (wm * (BM / S::WM) + li) * (KB * 16) + c;
      rb[t] = (BM + wn * (BN / S::WN) + li) * (KB * 16) + c;
    }
    uint4 fa[2][MX], fb[2][NI];
    uint32_t sa[2][MX], sb[2][NI];
    auto read = [&](int slot, int t, int p) {  // fragment p (rows', then columns') of K step t of a stage
      const uint8_t *buf = lds + slot * S::STAGE;
      if (p < MX)
        fa[t & 1][p] = *reinterpret_cast<const uint4 *>(buf + ra[t] + p * (32 * KB * 16));
      else
        fb[t & 1][p - MX] = *reinterpret_cast<const uint4 *>(buf + rb[t] + (p - MX) * (32 * KB * 16));
    };
    auto read_scales = [&](int slot, int win, int s) {
      const uint8_t *p;
      constexpr int step = S::WIDE ? 16 : 4;  // bytes between rows
      if constexpr (S::WIDE)  // the lane's dword of the window; past the row's end: the last one
        p = lds + S::WINDOWS + win * (S::ROWS * 16) + min(s * KB - min(s / 2 * 16, wlast) + 4 * hh, 12);
      else
        p = lds + slot * S::STAGE + S::ROWS * (KB * 16) + hh * (S::ROWS * 4);
      p += (wm * (BM / S::WM) + li) * step;
#pragma unroll
      for (int i = 0; i < MX; i++) sa[1][i] = *reinterpret_cast<const uint32_t *>(p + i * 32 * step);
      p += (BM + wn * (BN / S::WN) - wm * (BM / S::WM)) * step;
#pragma unroll
      for (int j = 0; j < NI; j++) sb[1][j] = *reinterpret_cast<const uint32_t *>(p + j * 32 * step);
    };
    auto take_scales = [&]() {
#pragma unroll
      for (int i = 0; i < MX; i++) sa[0][i] = sa[1][i];
#pragma unroll
      for (int j = 0; j < NI; j++) sb[0][j] = sb[1][j];
    };
    auto mul = [&](int t, int i, int j) {
      const uint4 x = fa[t & 1][i], y = fb[t & 1][j];
      const uint32_t u = sa[0][i], v = sb[0][j];
      acc[i][j] = t == 0 ? mx_mfma32<0>(y, v, x, u, acc[i][j]) : t == 1 ? mx_mfma32<1>(y, v, x, u, acc[i][j])
                : t == 2 ? mx_mfma32<2>(y, v, x, u, acc[i][j]) : mx_mfma32<3>(y, v, x, u, acc[i][j]);
    };

    // While a stage is multiplied the NBUF - 1 after it are on their way. Its last K step is in
    // registers before its buffer is given up, and is multiplied while the first loads of stage
    // + NBUF and the first fragments of the next stage are under way. The products' part of the body
    // has no branch: the compiler would move products across it, behind the wait.
#pragma unroll
    for (int s = 0; s < NBUF; s++) {
      issue_start();
#pragma unroll
      for (int q = 0; q < (s < NBUF - 1 ? ISSUES : EARLY); q++) issue(q);
      if (s < NBUF - 1) issue_end();
    }
    wait_loads<(NBUF - 2) * LOADS + EARLY_LOADS>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    TilePlace<S> at;  // the stage that is multiplied
    read_scales(0, 0, 0);
#pragma unroll
    for (int p = 0; p < MX + NI; p++) read(0, 0, p);
    take_scales();
    for (int col = 0; col < cols; col++) {
#pragma unroll
      for (int i = 0; i < MX; i++)
#pragma unroll
        for (int j = 0; j < NI; j++) acc[i][j] = v16f{};
      for (int s = 0; s < nst; s++) {
        // products, fragment reads and loads take turns, in this order: the next step's fragments
        // are read early in a step, and a burst of loads would leave the matrix cores without work
        constexpr int MUL = MX * NI, RT = (MUL + 1) / 2, RP = (MX + NI + RT - 1) / RT;
#pragma unroll
        for (int t = 0; t < KS - 1; t++)
#pragma unroll
          for (int q = 0; q < MUL; q++) {
            mul(t, q / NI, q % NI);
#pragma unroll
            for (int p = q * RP; p < (q + 1) * RP && p < MX + NI; p++) read(at.slot, t + 1, p);
            if (t == 0) {
              constexpr int PER0 = (ISSUES - EARLY + MUL - 1) / MUL;
#pragma unroll
              for (int p = EARLY + q * PER0; p < EARLY + (q + 1) * PER0 && p < ISSUES; p++) issue(p);
              if (q == MUL - 1) issue_end();
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        at.advance(nst);
        issue_start();
        wait_loads<(NBUF - 2) * LOADS>();  // the next stage has arrived; this one is in registers
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        constexpr int PER = (EARLY + MUL - 1) / MUL;
#pragma unroll
        for (int q = 0; q < MUL; q++) {
          __builtin_amdgcn_sched_barrier(0);
          mul(KS - 1, q / NI, q % NI);
          if (q == 0) read_scales(at.slot, at.win, at.stage);  // past the last stage: not used
#pragma unroll
          for (int p = q * PER; p < (q + 1) * PER && p < EARLY; p++) issue(p);
#pragma unroll
          for (int p = q * RP; p < (q + 1) * RP && p < MX + NI; p++) read(at.slot, 0, p);
        }
        __builtin_amdgcn_sched_barrier(0);
        take_scales();
      }
      // Results: lane column li (a row of activations) of a 32 x 32 tile, rows (weight rows)
      // 8 (r / 4) + 4 hh + r % 4, so that a lane holds runs of four output columns. Two bytes to a
      // value: the halves of the wavefront trade runs and each lane stores eight columns.
      // The stores have no branch (it would bring all results out of the accumulators at once,
      // as it does for a ragged N, whose last piece's columns go one by one): lanes without a row,
      // and pieces past the last column, give an offset past the buffer's end, where a store is
      // dropped.
      constexpr int GROUPS = MODE == MX_GATEUP ? 2 : 4, WF = BF / S::WN, JF = MODE == MX_GATEUP ? 16 : 32;
      typedef T piece_t __attribute__((ext_vector_type(16 / sizeof(T))));
      constexpr int PC = 16 / sizeof(T);                          // columns of a piece
      const int left = a.N - (bx + col) * BF - wn * WF;           // columns from the wavefront's first on
      const bool edge = left < WF;
      int lo = li, ho = hh;
      asm volatile("" : "+v"(lo), "+v"(ho));  // or the stores' offsets would all be kept over the column tiles
#pragma unroll
      for (int i = 0; i < MX; i++) {
        const int row = wm * (BM / S::WM) + i * 32 + lo;
        const bool there = row < n;
        const uint32_t off = ((uint32_t)out_row(row) * (uint32_t)a.N + (bx + col) * BF + wn * WF) * sizeof(T);
#pragma unroll
        for (int j = 0; j < NI; j++) {
          auto value = [&](int g, int r) -> T {
            if constexpr (MODE == MX_GATEUP)
              return (T)(silu_fast(acc[i][j][8 * g + r]) * acc[i][j][8 * g + 4 + r]);
            else
              return (T)acc[i][j][4 * g + r];
          };
          auto put = [&](piece_t w, int c) {
            const uint32_t at = off + c * sizeof(T);
            store_out(w, out, there && c + PC <= left ? at : ~0u);
            if (RAGGED && __builtin_expect(edge, 0)) {
#pragma unroll
              for (int r = 0; r < PC; r++)
                store_out(w[r], out, there && c + PC > left && c + r < left ? at + r * (int)sizeof(T) : ~0u);
            }
          };
#pragma unroll
          for (int g = 0; g < GROUPS; g += sizeof(T) == 4 ? 1 : 2) {
            if constexpr (sizeof(T) == 4) {
              piece_t w;
#pragma unroll
              for (int r = 0; r < 4; r++) w[r] = value(g, r);
              put(w, j * JF + 8 * g + 4 * ho);
            } else {
              typedef T half_t __attribute__((ext_vector_type(4)));
              half_t x, y;
#pragma unroll
              for (int r = 0; r < 4; r++) x[r] = value(g, r), y[r] = value(g + 1, r);
              const v2u32 xu = __builtin_bit_cast(v2u32, x), yu = __builtin_bit_cast(v2u32, y);
              // the lower lanes get their partner's run of g, the upper ones theirs of g + 1
              const auto p = __builtin_amdgcn_permlane32_swap(xu[0], yu[0], false, false);
              const auto q = __builtin_amdgcn_permlane32_swap(xu[1], yu[1], false, false);
              put(__builtin_bit_cast(piece_t, v4u32{p[0], q[0], p[1], q[1]}), j * JF + 8 * (g + ho));
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }
  };
  // routed rows and short batches seldom fill a tile: the products of the 32-row tiles that hold
  // none are left out
  if constexpr (S::WM > 1) {
    run.template operator()<MI>();
  } else {
    static_assert(MI == 4);
    if (n <= 32)
      run.template operator()<1>();
    else if (n <= 64)
      run.template operator()<2>();
    else
      run.template operator()<4>();
  }
}

// Row tiles of an expert that go through a column strip together, so that its weights come from
// the fabric once (4.23 -> 3.95 GB for gate/up of 2048 tokens); 2 and 8: 833 and 825 us
constexpr int EXP_GROUP = 8;

// Tile c of an expert's `all`: its w entry, routed | place in its group << 8 | size of the group << 16
__device__ __forceinline__ int tile_place(int c, int all, int routed) {
  const int i = c % EXP_GROUP;
  return routed | i << 8 | min(EXP_GROUP, all - (c - i)) << 16;
}

// Tiles of a route: {expert, first (of perm, or token), rows, place}, the shared expert's first.
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
  for (int c = tid; c < shared && c < cap; c += 1024)
    a.tiles[c] = make_int4(a.E, c * bm, min(bm, a.M - c * bm), tile_place(c, shared, 0));
  int g = base + incl - mine;
  for (int c = 0; c < mine; c++, g++)
    if (g < cap) a.tiles[g] = make_int4(e, first + c * bm, min(bm, n - c * bm), tile_place(c, mine, 1));
  if (tid == 0) *a.ntiles = min(total, cap);
}

template <MxMode MODE, typename T, typename S, bool RAGGED = false>
static hipError_t launch_tile(MxArgs a, int ny, hipStream_t s) {
  static_assert(S::BYTES <= 160 * 1024, "LDS");
  constexpr int BF = MODE == MX_GATEUP ? S::BN / 2 : S::BN;
  auto kernel = mx_tile_kernel<MODE, T, S, RAGGED>;
  static PerDevice allowed;
  if (const hipError_t st = allow_lds(allowed, kernel, S::BYTES); st != hipSuccess) return st;
  a.strip = MODE == MX_LINEAR ? dense_strip(a.N, BF, ny, MX_CUS * S::OCC) : expert_strip<S>(a.K / 32);
  const unsigned groups = (unsigned)tile_strips(a.N, BF, a.strip) * (unsigned)ny;
  hipLaunchKernelGGL(kernel, dim3(MODE == MX_LINEAR ? groups : (groups + 7) / 8 * 8), dim3(256), S::BYTES, s, a);
  return hipGetLastError();
}

// Fewer big tiles than this leave too many CUs without work. K = 6144, N = 12288: 26 us against 49
// with 48 big tiles (M = 256), 61 against 57 with 192; K = 2048, N = 4096: 20 against 27 with 128.
constexpr int DENSE_BIG_TILES = 192;

int64_t mx_tile_cap(int32_t T, int32_t k, int32_t E, int32_t has_shared) {
  const int64_t P = (int64_t)T * k, bm = TileExperts::BM;
  return P / bm + (P < E ? P : E) + (has_shared ? (T + bm - 1) / bm : 0);
}

template <typename T>
static hipError_t launch_tile_t(MxMode mode, const MxArgs &a, hipStream_t s) {
  if (mode == MX_LINEAR) {
    auto go = [&]<typename S>() {
      const int ny = (a.M + S::BM - 1) / S::BM;
      return a.N % (16 / sizeof(T)) == 0 ? launch_tile<MX_LINEAR, T, S>(a, ny, s)
                                         : launch_tile<MX_LINEAR, T, S, true>(a, ny, s);
    };
    const int64_t tiles = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
    return tiles >= DENSE_BIG_TILES ? go.template operator()<TileDense>() : go.template operator()<TileDenseSmall>();
  }
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
