// int8_tile.hip — int8 products of many rows with token and channel scales: LDS-tiled GEMMs on the
// 32x32x32 int8 matrix instruction of gfx950, dense and grouped over a route (batch-union:
// colibri-strix README, "What's implemented").
//
// The sums stay in the instruction's int32 accumulators over all of K, so the inner loop has no work
// for the vector units; scales, bias and SiLU*up come in at the end.
//
// Dense, 4093 x 12288 x 6144 bf16: 273 to 298 us by the card, with the quantisation's 19 to 23 (2.1 to 2.3
// POP/s). The instruction on random codes in registers alone reaches 2.9 to 3.5 POP/s here (4.9 on zeros: the
// card's power is the limit), 177 to 213 us. Of 281 us in all 234 are left without loads and 211 without products: they
// overlap but for 47, with one wavefront to a SIMD, whose 128 x 128 part fills the accumulators (and spills 14
// registers outside the loop over the stages). A row of a stage is one 128-byte line.
//
// Over a route, 2048 tokens, 256 experts of 6144 x 2048 and a shared one, Zipf-like: gate/up 1268 to 1380 us by the
// card, down 739 to 773 (and 77 to 83 for the combine, 20 for the quantisation of h). Bound by the loads' way:
// of 1277 us for gate/up 1259 are left without products and 699 without loads, of 845 for the whole down 848 and 549.
// Gate/up fetches 6.9 GB (6.5 needed), down 3.3 (3.2); a kernel that only moves gate/up's bytes to LDS takes 910
// to 1030, so that the rest is the tiles' starts and ends, one workgroup to a CU. Column strips of 1, 2 and 4 tiles
// 1344, 1381 and 1459 us; weights that one row tile alone reads past the caches 1344 -> 1300 (all weights: 1344, row
// tiles that share them meet in the L2); results past the caches 1307 -> 1283.
#include "int8_impl.h"
#include "mxfp4_tile_plan.h"
#include "tile_impl.h"

namespace coli {

// BM x BN tile, WM x WN wavefronts, NBUF K stages of 8 chunks (128 inputs) in LDS, OCC workgroups per CU.
// STRIPS: a workgroup takes column tiles one after another, the next one's loads under way while a tile is
// written out; else the stages' LDS serves for writing it out.
template <int BM_, int BN_, int WM_, int WN_, int NBUF_, int OCC_, bool STRIPS_>
struct I8Shape {
  static constexpr bool STRIPS = STRIPS_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NBUF = NBUF_, OCC = OCC_;
  static constexpr int KB = 8, KS = 4;                        // chunks of a stage, its K steps of 32 inputs
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;  // 32 x 32 tiles of a wavefront
  static constexpr int LA = BM / 32, LB = BN / 32;            // 16-byte loads of a wavefront per stage (8 rows each)
  static constexpr int STAGE = (BM + BN) * KB * 16;           // LDS bytes
  static constexpr int IDS = NBUF * STAGE;                    // offset of the row ids
  static constexpr int SCALES = IDS + BM * 4;                 // offset of two sets of channel scales and biases
  // 32 rows of 128 bytes and a pad for each wavefront, through which results go to whole lines
  static constexpr int OUT_ROW = 144, OUT_WAVE = 32 * OUT_ROW;
  static constexpr int OUT = STRIPS ? SCALES + 2 * 2 * BN * 4 : 0;
  static constexpr int BYTES = SCALES + 2 * 2 * BN * 4 + (STRIPS ? 4 * OUT_WAVE : 0);
  static_assert(LB % 2 == 0 && 4 * OUT_WAVE <= IDS);
};
typedef I8Shape<256, 256, 2, 2, 2, 1, true> I8Dense;
typedef I8Shape<128, 128, 1, 4, 2, 2, false> I8DenseSmall;
typedef I8Shape<128, 64, 2, 2, 3, 2, false> I8DenseNarrow;
typedef I8Shape<64, 64, 2, 2, 4, 2, false> I8DenseTiny;
typedef I8Shape<128, 256, 1, 4, 3, 1, false> I8Experts;

typedef int v16i __attribute__((ext_vector_type(16)));

__device__ __forceinline__ v16i i8_mfma32(uint4 a, uint4 b, v16i c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(v4i32, a), __builtin_bit_cast(v4i32, b), c, 0, 0, 0);
}

// RAGGED: N is no multiple of the columns of a 16-byte piece
template <I8Mode MODE, typename T, typename S, bool RAGGED>
__global__ __launch_bounds__(256, S::OCC) void i8_tile_kernel(I8Args a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int BM = S::BM, BN = S::BN, MI = S::MI, NI = S::NI, NBUF = S::NBUF, KB = S::KB, KS = S::KS;
  constexpr int BF = MODE == I8_GATEUP ? BN / 2 : BN;  // output columns of a tile
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv / S::WN, wn = wv % S::WN;
  const int K = a.K, nc = K / 16, pitch = i8_padded(K), nst = (nc + KB - 1) / KB;
  const int ns = tile_strips(a.N, BF, a.strip);

  // the rows of activations: first .. first + n - 1 of perm, or of the tokens; and the column
  // tiles bx .. bx + cols - 1, one after another
  int bx, by, cols, e = 0, first = 0, n = 0;
  bool routed = false, once = false;
  if constexpr (MODE == I8_LINEAR) {
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
    once = grp == 1;
  }
  const int64_t P = (int64_t)a.M * a.k;
  // tile row i -> row of the output, of the activations
  int *ids = reinterpret_cast<int *>(lds + S::IDS);
  if constexpr (MODE != I8_LINEAR) {
    for (int i = threadIdx.x; i < BM; i += 256) {
      const int ci = first + min(i, n - 1);
      ids[i] = routed ? a.perm[ci] : (int)(P + ci);
    }
    __syncthreads();
  }
  auto out_row = [&](int i) -> int { return MODE == I8_LINEAR ? i : ids[i]; };  // relative to the buffer below
  // the output from its first row on (of a dense product: the tile's); offsets fit in 32 bits
  const int64_t rows = MODE == I8_LINEAR ? n : P + (a.has_shared ? a.M : 0);
  const auto out = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<T *>(a.out) + (MODE == I8_LINEAR ? (int64_t)first * a.N : 0), 0, (int)(uint32_t)(rows * a.N * sizeof(T)),
      0x00027000);
  auto act_row = [&](int i) -> int {  // relative to the base below
    if constexpr (MODE == I8_LINEAR) return min(i, n - 1);
    return MODE == I8_DOWN ? ids[i] : (routed ? ids[i] / a.k : ids[i] - (int)P);
  };
  // tile-relative bases keep the lanes' offsets within 32 bits
  const uint8_t *aq = reinterpret_cast<const uint8_t *>(a.aq);
  const float *as = a.as;
  if constexpr (MODE == I8_LINEAR) aq += (int64_t)first * pitch, as += first;
  aq = uniform(aq);
  const uint8_t *wq = reinterpret_cast<const uint8_t *>(a.wq) + (int64_t)e * a.wq_stride + (int64_t)bx * BF * K;
  const float *ws = a.ws + (int64_t)e * a.ws_stride;

  // load i of this wavefront: rows (4 i + wv) 8 .. + 7; lane l: row l / 8, slot l % 8
  const int lr = lane >> 3, chunk = (lane & 7) ^ tile_swizzle(8 * wv + lr);
  uint32_t oa[S::LA], ob[S::LB];
#pragma unroll
  for (int i = 0; i < S::LA; i++)
    oa[i] = (uint32_t)act_row((4 * i + wv) * 8 + lr) * (uint32_t)pitch + chunk * 16 + (i & 1 ? 0 : 4096);
#pragma unroll
  for (int i = 0; i < S::LB; i++)
    ob[i] = (uint32_t)tile_weight_row(MODE == I8_GATEUP, (4 * i + wv) * 8 + lr, a.N, bx * BF) * (uint32_t)K + chunk * 16 + (i & 1 ? 0 : 4096);
  // weight chunks past K repeat the row's last one: they meet activations of zero
  const uint32_t past_k = max((nst - 1) * KB + chunk - (nc - 1), 0) * 16;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int li = lane & 31, hh = lane >> 5;

  // with MX 32-row tiles to a wavefront; ONCE: no other workgroup reads these weights
  auto run = [&]<int MX, bool ONCE>() {
    float row_scale[MX];
#pragma unroll
    for (int i = 0; i < MX; i++) row_scale[i] = as[act_row(wm * (BM / S::WM) + i * 32 + li)];
    // channel scales (gate/up: the gate's, then the up's) and biases of column tile `col`
    auto take_scales = [&](int col) {
      float *sc = reinterpret_cast<float *>(lds + S::SCALES) + (col & 1) * 2 * BN;
      for (int i = threadIdx.x; i < BN; i += 256) {
        const int c = min((bx + col) * BF + i % BF, a.N - 1);
        sc[i] = ws[(i / BF) * a.N + c];
        if constexpr (MODE == I8_LINEAR) sc[BN + i] = a.bias ? a.bias[c] : 0.0f;
      }
    };
    take_scales(0);
    // The loads run ahead of the products, over the stages of all column tiles, of the one whose
    // weights start at pb.
    int ahead = 0, ahead_slot = 0;  // stage, buffer
    int left = cols * nst;
    const uint8_t *pb = uniform(wq);
    int on = -1;        // 0 once every stage is under way: the loads are empty
    uint32_t past = 0;  // past_k at a row's last stage
    auto issue_start = [&]() {
      on = __builtin_amdgcn_readfirstlane(-left >> 31);
      past = ahead == nst - 1 ? past_k : 0u;
    };
    constexpr int NA = S::WM == 1 ? MX : S::LA, QA = (NA + 1) / 2, QB = S::LB / 2;  // loads go in pairs; an odd one alone
    auto issue = [&](int q) {  // load or pair q of the stage
      const uint32_t buf = lds0 + ahead_slot * S::STAGE;
      if (q < QA) {
        const uint32_t dst = buf + (8 * q + wv) * 1024;
        if (2 * q + 1 < NA)
          dma16_pair(aq + ahead * (KB * 16), oa[2 * q], oa[2 * q + 1], dst, on, on);
        else
          dma16(aq + ahead * (KB * 16) - 4096, oa[2 * q], dst, on, on);
      } else {
        const int i = q - QA;
        if constexpr (ONCE)
          dma16_pair_once(pb + ahead * (KB * 16), ob[2 * i] - past, ob[2 * i + 1] - past, buf + BM * (KB * 16) + (8 * i + wv) * 1024, on, on);
        else
          dma16_pair(pb + ahead * (KB * 16), ob[2 * i] - past, ob[2 * i + 1] - past, buf + BM * (KB * 16) + (8 * i + wv) * 1024, on, on);
      }
    };
    constexpr int ISSUES = QA + QB, LOADS = NA + S::LB;
    static_assert((NBUF - 1) * LOADS <= 63, "vmcnt");
    // The first EARLY issues of a stage go out in the K step after the barrier, the others in the
    // next one.
    constexpr int EARLY = NBUF > 2 ? ISSUES / 4 : ISSUES / 2;
    constexpr int EARLY_LOADS = EARLY <= QA ? (EARLY * 2 < NA ? EARLY * 2 : NA) : NA + (EARLY - QA) * 2;
    auto issue_end = [&]() {
      left--;
      ahead_slot = ahead_slot == NBUF - 1 ? 0 : ahead_slot + 1;
      if (++ahead == nst) {
        ahead = 0;
        pb += (int64_t)BF * K;
      }
    };

    v16i acc[MX][NI];
    // K step t takes chunk t of a stage in lanes 0-31 and chunk 4 + t in lanes 32-63
    uint32_t ra[KS], rb[KS];
#pragma unroll
    for (int t = 0; t < KS; t++) {
      const int c = ((t + 4 * hh) ^ tile_swizzle(li)) * 16;
      ra[t] = (wm * (BM / S::WM) + li) * (KB * 16) + c;
      rb[t] = (BM + wn * (BN / S::WN) + li) * (KB * 16) + c;
    }
    uint4 fa[2][MX], fb[2][NI];
    auto read = [&](int slot, int t, int p) {  // fragment p (rows', then columns') of K step t of a stage
      const uint8_t *buf = lds + slot * S::STAGE;
      if (p < MX)
        fa[t & 1][p] = *reinterpret_cast<const uint4 *>(buf + ra[t] + p * (32 * KB * 16));
      else
        fb[t & 1][p - MX] = *reinterpret_cast<const uint4 *>(buf + rb[t] + (p - MX) * (32 * KB * 16));
    };
    auto mul = [&](int t, int i, int j) { acc[i][j] = i8_mfma32(fb[t & 1][j], fa[t & 1][i], acc[i][j]); };

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
    int slot = 0;  // buffer of the stage that is multiplied
#pragma unroll
    for (int p = 0; p < MX + NI; p++) read(0, 0, p);
    for (int col = 0; col < cols; col++) {
      if (col) take_scales(col);  // the set that no wavefront reads: a barrier follows before each set's next turn
#pragma unroll
      for (int i = 0; i < MX; i++)
#pragma unroll
        for (int j = 0; j < NI; j++) acc[i][j] = v16i{};
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
            for (int p = q * RP; p < (q + 1) * RP && p < MX + NI; p++) read(slot, t + 1, p);
            if (t == 0) {
              constexpr int PER0 = (ISSUES - EARLY + MUL - 1) / MUL;
#pragma unroll
              for (int p = EARLY + q * PER0; p < EARLY + (q + 1) * PER0 && p < ISSUES; p++) issue(p);
              if (q == MUL - 1) issue_end();
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        slot = slot == NBUF - 1 ? 0 : slot + 1;
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
#pragma unroll
          for (int p = q * PER; p < (q + 1) * PER && p < EARLY; p++) issue(p);
#pragma unroll
          for (int p = q * RP; p < (q + 1) * RP && p < MX + NI; p++) read(slot, 0, p);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // Results: lane column li (a row of activations) of a 32 x 32 tile, rows (weight rows)
      // 8 (r / 4) + 4 hh + r % 4, so that a lane holds runs of four output columns of a row. They go
      // through LDS, up to 128 bytes of 32 rows at a time, so that a store covers whole lines: written
      // from the accumulators, a run each, 32 rows' stores of 32 bytes go out at a time (down of 2048 tokens
      // 872 us and 854 so, 752 without stores; 4093 x 12288 x 6144 299, 290 and 272, all before the loads and stores past
      // the caches).
      // The stores have no branch (it would bring all results out of the accumulators at once,
      // as it does for a ragged N, whose last piece's columns go one by one): lanes without a row,
      // and pieces past the last column, give an offset past the buffer's end, where a store is
      // dropped.
      constexpr int GROUPS = MODE == I8_GATEUP ? 2 : 4, WF = BF / S::WN, JF = MODE == I8_GATEUP ? 16 : 32;
      constexpr int BC = WF * (int)sizeof(T) < 128 ? WF : 128 / (int)sizeof(T);  // columns of a block
      constexpr int JB = BC / JF;                                                // its tiles
      constexpr int LPR = BC * (int)sizeof(T) / 16, RPI = 64 / LPR;              // lanes of a row, rows of a store
      static_assert(JB >= 1 && BC % JF == 0 && WF % BC == 0);
      typedef T piece_t __attribute__((ext_vector_type(16 / sizeof(T))));
      typedef T run_t __attribute__((ext_vector_type(4)));
      constexpr int PC = 16 / sizeof(T);                 // columns of a piece
      const int after = a.N - (bx + col) * BF - wn * WF;  // columns from the wavefront's first on
      const bool edge = after < WF;
      int lo = li, ho = hh, pl = lane % LPR, pr = lane / LPR;
      asm volatile("" : "+v"(lo), "+v"(ho), "+v"(pl), "+v"(pr));  // or the stores' offsets would all be kept over the column tiles
      const float *sc = reinterpret_cast<const float *>(lds + S::SCALES) + (col & 1) * 2 * BN + wn * WF + 4 * ho;
      uint8_t *block = lds + S::OUT + wv * S::OUT_WAVE;
#pragma unroll
      for (int i = 0; i < MX; i++) {
        uint32_t off[32 / RPI];  // of this lane's pieces of a block: the row's start, or past the end
#pragma unroll
        for (int k = 0; k < 32 / RPI; k++) {
          const int row = wm * (BM / S::WM) + i * 32 + k * RPI + pr;
          off[k] = row < n ? ((uint32_t)out_row(row) * (uint32_t)a.N + (bx + col) * BF + wn * WF) * sizeof(T) : ~0u;
        }
#pragma unroll
        for (int j0 = 0; j0 < NI; j0 += JB) {
#pragma unroll
          for (int jj = 0; jj < JB; jj++) {
            const int j = j0 + jj;
#pragma unroll
            for (int g = 0; g < GROUPS; g++) {
              const v4f cs = *reinterpret_cast<const v4f *>(sc + j * JF + 8 * g);
              v4f cb = {};
              if constexpr (MODE != I8_DOWN) cb = *reinterpret_cast<const v4f *>(sc + BF + j * JF + 8 * g);
              run_t w;
#pragma unroll
              for (int r = 0; r < 4; r++) {
                if constexpr (MODE == I8_GATEUP)
                  w[r] = (T)i8_product(i8_silu(i8_value(acc[i][j][8 * g + r], row_scale[i], cs[r])),
                                       i8_value(acc[i][j][8 * g + 4 + r], row_scale[i], cb[r]));
                else if constexpr (MODE == I8_LINEAR)
                  w[r] = (T)i8_biased(acc[i][j][4 * g + r], row_scale[i], cs[r], cb[r]);
                else
                  w[r] = (T)i8_value(acc[i][j][4 * g + r], row_scale[i], cs[r]);
              }
              *reinterpret_cast<run_t *>(block + lo * S::OUT_ROW + (jj * JF + 8 * g + 4 * ho) * (int)sizeof(T)) = w;
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          // a wavefront's LDS accesses are done in order
          __builtin_amdgcn_wave_barrier();
          asm volatile("" ::: "memory");
#pragma unroll
          for (int k = 0; k < 32 / RPI; k++) {
            const piece_t w = *reinterpret_cast<const piece_t *>(block + (k * RPI + pr) * S::OUT_ROW + pl * 16);
            const int c = j0 * JF + pl * PC;
            const bool there = off[k] != ~0u;
            const uint32_t to = off[k] + c * (int)sizeof(T);
            store_out<2>(w, out, there && c + PC <= after ? to : ~0u);
            if (RAGGED && __builtin_expect(edge, 0)) {
#pragma unroll
              for (int r = 0; r < PC; r++)
                store_out(w[r], out, there && c + PC > after && c + r < after ? to + r * (int)sizeof(T) : ~0u);
            }
          }
          __builtin_amdgcn_wave_barrier();
          asm volatile("" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  // routed rows and short batches seldom fill a tile: the products of the 32-row tiles that hold
  // none are left out
  if constexpr (S::WM > 1) {
    run.template operator()<MI, false>();
  } else {
    static_assert(MI == 4);
    auto rows = [&]<bool ONCE>() {
      if (n <= 32)
        run.template operator()<1, ONCE>();
      else if (n <= 64)
        run.template operator()<2, ONCE>();
      else
        run.template operator()<4, ONCE>();
    };
    if (MODE != I8_LINEAR && once)
      rows.template operator()<MODE != I8_LINEAR>();
    else
      rows.template operator()<false>();
  }
}

template <I8Mode MODE, typename T, typename S, bool RAGGED = false>
static hipError_t launch_tile(I8Args a, int ny, hipStream_t s) {
  static_assert(S::BYTES <= 160 * 1024 / S::OCC, "LDS");
  constexpr int BF = MODE == I8_GATEUP ? S::BN / 2 : S::BN;
  auto kernel = i8_tile_kernel<MODE, T, S, RAGGED>;
  static PerDevice allowed;
  if (const hipError_t st = allow_lds(allowed, kernel, S::BYTES); st != hipSuccess) return st;
  a.strip = S::STRIPS ? dense_strip(a.N, BF, ny, MX_CUS * S::OCC) : 1;
  const unsigned groups = (unsigned)tile_strips(a.N, BF, a.strip) * (unsigned)ny;
  hipLaunchKernelGGL(kernel, dim3(MODE == I8_LINEAR ? groups : (groups + 7) / 8 * 8), dim3(256), S::BYTES, s, a);
  return hipGetLastError();
}

// Tiles of a dense product, by how many there are of the next smaller kind: as large as fill the card.
// us with 64 x 64, 128 x 64, 128 x 128 tiles: 64 x 12288 x 6144 (192 tiles of 64 x 64) 22, 25, 37;
// 1000 x 1024 x 4096 (256) 18, 21, 29; 128 x 12288 x 6144 (384) 28, 26, 41; 1000 x 2048 x 6144 (512) 32,
// 30, 42; 256 x 12288 x 6144 (768) 51, 46, 47-51; 1000 x 4096 x 4096 (1024) 39, 31, 32; 500 x 12288 x 6144
// (1536) 71-76, 58, 51-58; 2000 x 4096 x 4096 (2048) 72, 55, 48.
constexpr int64_t DENSE_TINY_TILES = 256, DENSE_NARROW_TILES = 1024, DENSE_BIG_TILES = 192;

int64_t i8_tile_cap(int32_t T, int32_t k, int32_t E, int32_t has_shared) {
  const int64_t P = (int64_t)T * k, bm = I8Experts::BM;
  return P / bm + (P < E ? P : E) + (has_shared ? (T + bm - 1) / bm : 0);
}

template <typename T>
static hipError_t launch_tile_t(I8Mode mode, const I8Args &a, hipStream_t s) {
  if (mode == I8_LINEAR) {
    auto go = [&]<typename S>() {
      const int ny = (a.M + S::BM - 1) / S::BM;
      return a.N % (16 / sizeof(T)) == 0 ? launch_tile<I8_LINEAR, T, S>(a, ny, s)
                                         : launch_tile<I8_LINEAR, T, S, true>(a, ny, s);
    };
    const int64_t big = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
    const int64_t tiny = (int64_t)((a.M + 63) / 64) * ((a.N + 63) / 64);
    if (big >= DENSE_BIG_TILES) return go.template operator()<I8Dense>();
    if (tiny <= DENSE_TINY_TILES) return go.template operator()<I8DenseTiny>();
    return tiny <= DENSE_NARROW_TILES ? go.template operator()<I8DenseNarrow>() : go.template operator()<I8DenseSmall>();
  }
  const int cap = (int)i8_tile_cap(a.M, a.k, a.E, a.has_shared);
  hipLaunchKernelGGL(route_tiles_kernel<I8Args>, dim3(1), dim3(1024), 0, s, a, I8Experts::BM, cap);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  return mode == I8_GATEUP ? launch_tile<I8_GATEUP, T, I8Experts>(a, cap, s) : launch_tile<I8_DOWN, float, I8Experts>(a, cap, s);
}

hipError_t launch_i8_tile(I8Mode mode, int dtype, const I8Args &a, hipStream_t s) {
  if (dtype == COLI_F32) return launch_tile_t<float>(mode, a, s);
  if (dtype == COLI_BF16) return launch_tile_t<bf16_t>(mode, a, s);
  return launch_tile_t<f16_t>(mode, a, s);
}

}  // namespace coli
