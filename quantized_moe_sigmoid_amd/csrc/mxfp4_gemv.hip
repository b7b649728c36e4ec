// mxfp4_gemv.hip — MXFP4 x MXFP4 products of few rows, bound by the weights' way from HBM: dense
// rows, the experts' gate/up rows with SiLU*up and their down rows over a route (batch-union:
// colibri-strix README, "What's implemented"), on the scaled 16x16x128 matrix instruction.
//
// mx_gemv_kernel: a workgroup (4 wavefronts) owns 16 weight rows (of each matrix) and chunks of
// 16 NT rows of activations. The wavefronts take the K groups (16 blocks, 512 inputs: 256
// contiguous bytes of a row) in turn, two groups of weights under way at a time straight into
// the operand registers; their sums meet in LDS, added in wavefront order. One row of
// activations (x in ACT_X) is quantised by every workgroup itself while its first weights are
// under way, which saves a launch. One token, bf16: dense 12288 x 6144 8.3 to 9 us (40 MB, 6.4 us
// at the 6.3 TB/s of a plain streaming read, and a launch), gate/up of 9 experts of 6144 x 2048
// 23 to 24.5 us (120 MB, 5 TB/s); gate/up of 16 tokens over 256 experts 243 us (5.7 TB/s).
//
// mx_down_kernel: the down product of few tokens (16 to a workgroup) with its weighted combine. A
// workgroup (8 wavefronts) owns 8 to 32 output rows of its tokens and goes through all experts
// they hold, a token to a column of the matrix instruction; experts and K groups are dealt to the
// wavefronts, one unit of each under way: with two the loads came in bursts (16 tokens over 256
// experts of 6144 x 2048 118 us, over 64 of 4096 x 4096 100), with one 112 and 92. The pairs' rows
// stay in LDS, no second kernel sums them. The 112 us have the quantisation of h in them: 0.69 GB,
// 6.2 TB/s, the rate of a plain read. One token 15 us, 48 tokens 338.
#include <cmath>

#include "mxfp4_impl.h"

namespace coli {

// 16 blocks of a weight row, as a lane of the matrix instruction takes them: in step s the
// block 4 s + l / 16; u[s] holds its scale in byte 0
struct Group {
  uint4 c[4];
  uint32_t u[4];
};

// How a row's scales come in: SC_FULL: nb is a multiple of 16 and the scales are 16-byte aligned;
// SC_ANY: 16 bytes at any address, nb >= 16 (a group that the row ends in takes the row's last 16,
// shifted at the product); SC_BYTES: byte by byte, for shorter rows. 16 tokens of 64 experts,
// K = 1920: gate/up 94 us with byte loads, 47 with these.
enum ScaleLoad { SC_FULL, SC_ANY, SC_BYTES };
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

template <ScaleLoad SL>
__device__ __forceinline__ void load_group(const uint8_t *codes, const uint8_t *scales, int nb, int g, int lq, Group &o) {
  if constexpr (SL == SC_FULL) {
    const uint4 u = *reinterpret_cast<const uint4 *>(scales + g * 16);
    o.u[0] = u.x, o.u[1] = u.y, o.u[2] = u.z, o.u[3] = u.w;  // shifted at the product
  } else if constexpr (SL == SC_ANY) {
    const u32x4_any u = *reinterpret_cast<const u32x4_any *>(scales + min(g * 16, nb - 16));
    o.u[0] = u[0], o.u[1] = u[1], o.u[2] = u[2], o.u[3] = u[3];
  }
#pragma unroll
  for (int s = 0; s < 4; s++) {
    const int b = g * 16 + 4 * s + lq;
    const int bb = SL == SC_FULL ? b : min(b, nb - 1);  // past the row: the last block; it meets activations of zero
    o.c[s] = *reinterpret_cast<const uint4 *>(codes + bb * 16);
    if constexpr (SL == SC_BYTES) o.u[s] = scales[bb];
  }
}

// SC_ANY, before the products: the group that the row ends in, of which the last 16 scales came
template <ScaleLoad SL>
__device__ __forceinline__ void end_group(Group &o, int nb, int g) {
  if constexpr (SL == SC_ANY) {
    const int past = g * 16 + 16 - nb;  // bytes that came too early; what moves in behind is a scale of the row or 0
    if (past > 0) {
      for (int i = past >> 2; i > 0; i--) o.u[0] = o.u[1], o.u[1] = o.u[2], o.u[2] = o.u[3];
      const uint32_t r = past & 3;
      o.u[0] = __builtin_amdgcn_alignbyte(o.u[1], o.u[0], r);
      o.u[1] = __builtin_amdgcn_alignbyte(o.u[2], o.u[1], r);
      o.u[2] = __builtin_amdgcn_alignbyte(o.u[3], o.u[2], r);
      o.u[3] >>= 8 * r;
    }
  }
}

template <ScaleLoad SL>
__device__ __forceinline__ uint32_t group_scale(const Group &g, int s, int lq) {
  return SL == SC_BYTES ? g.u[s] : g.u[s] >> (8 * lq);
}

// One row x of nb blocks -> codes and scales in LDS (blocks nb .. nbp: zeros), by 256 threads.
// The values of a thread's first two half-blocks come in v (load_x), loaded ahead.
constexpr int XH = 2;
template <typename T>
__device__ __forceinline__ void load_x(const T *x, int nb, int tid, float (&v)[XH][2][8]) {
#pragma unroll
  for (int i = 0; i < XH; i++) {
    const int h = min(tid + 256 * i, 2 * nb - 1), blk = h >> 1, q = h & 1;
    load8(x + blk * 32 + 8 * q, v[i][0]);
    load8(x + blk * 32 + 16 + 8 * q, v[i][1]);
  }
}

__device__ __forceinline__ void put_half(uint8_t *lc, uint8_t *ls, int h, const float (&a)[8], const float (&b)[8]) {
  uint32_t u;
  const uint2 w = mx_quant_half(a, b, u);
  *reinterpret_cast<uint2 *>(lc + h * 8) = w;
  if (!(h & 1)) ls[h >> 1] = (uint8_t)u;
}

template <typename T>
__device__ __forceinline__ void quantise_x(const T *x, int nb, int nbp, int tid, const float (&v)[XH][2][8], uint8_t *lc,
                                           uint8_t *ls) {
#pragma unroll
  for (int i = 0; i < XH; i++) {
    const int h = tid + 256 * i;
    if (h < 2 * nb) put_half(lc, ls, h, v[i][0], v[i][1]);  // both lanes of a block or neither
  }
  for (int h = tid + 256 * XH; h < 2 * nb; h += 256) {
    float a[8], b[8];
    load8(x + (h >> 1) * 32 + 8 * (h & 1), a);
    load8(x + (h >> 1) * 32 + 16 + 8 * (h & 1), b);
    put_half(lc, ls, h, a, b);
  }
  for (int h = 2 * nb + tid; h < 2 * nbp; h += 256) {
    *reinterpret_cast<uint2 *>(lc + h * 8) = make_uint2(0, 0);
    if (!(h & 1)) ls[h >> 1] = 127;
  }
}

enum MxAct { ACT_WS, ACT_X };  // activations: quantised in the workspace; one row of x

// Do eight gate rows and the eight up rows of the same features share a tile of the matrix
// instruction? It takes half the registers of 16 rows of each: one token 26 -> 24.7 us, and rows
// that are no multiple of 16 blocks, whose loads need more registers, 94 -> 52 us (16 tokens,
// K = 1920). Else activations are read twice as often: 16 tokens 243 -> 265 us.
template <MxMode MODE, MxAct ACT, ScaleLoad SL>
constexpr bool gate_up_halves() {
  return MODE == MX_GATEUP && (ACT == ACT_X || SL != SC_FULL);
}

template <MxMode MODE, typename T, int NT, MxAct ACT, ScaleLoad SL>
__global__ __launch_bounds__(256, 2) void mx_gemv_kernel(MxArgs a) {
  constexpr bool HALVES = gate_up_halves<MODE, ACT, SL>();
  constexpr int NMAT = MODE == MX_GATEUP && !HALVES ? 2 : 1;
  constexpr int D = NT == 4 ? 1 : 2;  // groups under way: what the registers hold
  static_assert(ACT == ACT_WS || (NT == 1 && MODE != MX_DOWN));
  extern __shared__ __align__(16) uint8_t lds[];  // ACT_X: the quantised row
  __shared__ float red[4][NMAT][NT][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * (HALVES ? 8 : 16);
  const int nb = a.K / 32, nbp = mx_padded(a.K) / 32;
  const int ngw = (nbp / 16 - wv + 3) / 4;  // groups of this wavefront: wv, wv + 4, ..
  // the rows of activations: first .. first + n - 1 of perm (routed) or of the tokens
  int e = 0, first = 0, n = a.M;
  bool routed = false;
  if constexpr (MODE == MX_LINEAR) {
    first = blockIdx.y * (16 * NT);
    n = min(16 * NT, a.M - first);
  } else {
    const int u = (int)blockIdx.y - a.has_shared;
    if (u < 0) {
      e = a.E;
    } else {
      if (const int na = *a.nact; u >= na && (na >= 0 || u >= hit_experts(a.nact, a.off, a.E))) return;
      e = a.active[u];
      first = a.off[e];
      n = a.off[e + 1] - first;
      routed = true;
    }
  }
  const int64_t P = (int64_t)a.M * a.k;
  float xv[XH][2][8];
  const T *x = static_cast<const T *>(a.x);
  if constexpr (ACT == ACT_X) {
    load_x(x, nb, tid, xv);
  }
  const uint8_t *wc[NMAT], *ws[NMAT];
#pragma unroll
  for (int m = 0; m < NMAT; m++) {
    const int64_t row = HALVES ? (int64_t)(li >> 3) * a.N + min(n0 + (li & 7), a.N - 1) : (int64_t)m * a.N + min(n0 + li, a.N - 1);
    wc[m] = a.wc + (int64_t)e * a.wc_stride + row * nb * 16;
    ws[m] = a.ws + (int64_t)e * a.ws_stride + row * nb;
  }
  Group w[D][NMAT], act[D][NT];
  for (int c = 0; c < n; c += 16 * NT) {
    const uint8_t *ac[NT], *as[NT];
    if constexpr (ACT == ACT_WS) {
#pragma unroll
      for (int q = 0; q < NT; q++) {
        const int ci = first + min(c + 16 * q + li, n - 1);
        int64_t arow = ci;
        if constexpr (MODE != MX_LINEAR) {
          const int64_t pair = routed ? a.perm[ci] : P + ci;
          arow = MODE == MX_DOWN ? pair : (routed ? pair / a.k : ci);
        }
        ac[q] = a.ac + arow * nbp * 16;
        as[q] = a.as + arow * nbp;
      }
    }
    // group i of this wavefront: weights and (in the workspace) activations together, since
    // loads arrive in order
    auto load_act = [&](int d, int i) {
#pragma unroll
      for (int q = 0; q < NT; q++) load_group<SC_FULL>(ac[q], as[q], nbp, wv + 4 * i, lq, act[d][q]);
    };
    auto load = [&](int d, int i) {
#pragma unroll
      for (int m = 0; m < NMAT; m++) load_group<SL>(wc[m], ws[m], nb, wv + 4 * i, lq, w[d][m]);
      if constexpr (ACT == ACT_WS) load_act(d, i);
    };
#pragma unroll
    for (int d = 0; d < D; d++)
      if (d < ngw) load(d, d);
    if constexpr (ACT == ACT_X) {
      quantise_x(x, nb, nbp, tid, xv, lds, lds + nbp * 16);
      __syncthreads();
      ac[0] = lds;
      as[0] = lds + nbp * 16;
    }
    v4f acc[NT][NMAT] = {};
    for (int i0 = 0; i0 < ngw; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; d++) {
        if (i0 + d < ngw) {
          if constexpr (ACT == ACT_X) load_act(d, i0 + d);
#pragma unroll
          for (int m = 0; m < NMAT; m++) end_group<SL>(w[d][m], nb, wv + 4 * (i0 + d));
#pragma unroll
          for (int s = 0; s < 4; s++)
#pragma unroll
            for (int q = 0; q < NT; q++)
#pragma unroll
              for (int m = 0; m < NMAT; m++)
                acc[q][m] = mx_mfma16(act[d][q].c[s], group_scale<SC_FULL>(act[d][q], s, lq), w[d][m].c[s],
                                      group_scale<SL>(w[d][m], s, lq), acc[q][m]);
          if (i0 + d + D < ngw) load(d, i0 + d + D);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < NT; q++)
#pragma unroll
      for (int m = 0; m < NMAT; m++)
#pragma unroll
        for (int r = 0; r < 4; r++) red[wv][m][q][4 * lq + r][li] = acc[q][m][r];
    __syncthreads();
    const int tr = tid >> 4, tc = tid & 15;
#pragma unroll
    for (int q = 0; q < NT; q++) {
      auto sum = [&](int m, int col) {
        return ((red[0][m][q][tr][col] + red[1][m][q][tr][col]) + red[2][m][q][tr][col]) + red[3][m][q][tr][col];
      };
      const int row = c + 16 * q + tr;
      if (row < n && n0 + tc < a.N && (!HALVES || tc < 8)) {
        const int ci = first + row;
        const int64_t orow = MODE == MX_LINEAR ? ci : (routed ? (int64_t)a.perm[ci] : P + ci);
        const int64_t o = orow * a.N + n0 + tc;
        if constexpr (MODE == MX_GATEUP)
          static_cast<T *>(a.out)[o] = (T)(silu(sum(0, tc)) * (HALVES ? sum(0, tc + 8) : sum(NMAT - 1, tc)));
        else if constexpr (MODE == MX_DOWN)
          static_cast<float *>(a.out)[o] = sum(0, tc);
        else
          static_cast<T *>(a.out)[o] = (T)sum(0, tc);
      }
    }
    if (c + 16 * NT < n) __syncthreads();
  }
}

// ------------------------------------------------------------------ down with its combine
constexpr int DN_TOK = 16, DN_K = 16, DN_WAVES = 8;

// Dynamic LDS of mx_down_kernel, bytes: slots first, then these; all but the quantised rows of ACT_X
struct DownLds {
  size_t list, y, x;
};
__host__ __device__ inline DownLds down_lds(const MxArgs &a, int step, int lp, int tokens) {
  DownLds L;
  L.list = (size_t)a.E * DN_TOK * 2;
  L.y = L.list + ((size_t)tokens * a.k + 1 + 3) / 4 * 16;
  L.x = L.y + ((size_t)tokens * (a.k + a.has_shared) << lp) * step * sizeof(float);
  return L;
}
__host__ __device__ inline DownLds down_lds(const MxArgs &a, int step, int lp) {
  return down_lds(a, step, lp, a.M < DN_TOK ? a.M : DN_TOK);
}

// RT 16-row tiles of the matrix instruction for the `step` output rows of a workgroup: rows past
// them, like rows past N, read past their buffer's end, which gives zeros without an access.
// 1 << lp wavefronts share an expert's K groups; what each sums for a (token, slot) has its own
// place in LDS, and at the end the parts, then the weighted slots, then the shared expert's row
// are added in order: a token's row does not depend on the tokens beside it.
template <typename T, MxAct ACT, ScaleLoad SL, int RT>
__global__ __launch_bounds__(64 * DN_WAVES) void mx_down_kernel(MxArgs a, int step, int lp, const int32_t *__restrict__ idx,
                                                               const float *__restrict__ w, T *__restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ float weight[DN_TOK * DN_K];
  __shared__ uint32_t there[DN_TOK];  // slots of a token that hold an expert, a bit each
  __shared__ int n_entries, repeats;    // repeats: some token holds an expert in two slots
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * step, nrows = min(step, a.N - n0);
  const int nb = a.K / 32, nbp = mx_padded(a.K) / 32, ng = nbp / 16;
  const int t0 = blockIdx.y * DN_TOK, T_ = min(DN_TOK, a.M - t0);  // this workgroup's tokens
  const int k = a.k, E = a.E, P = a.M * k, ks = k + a.has_shared;
  // slots[e * 16 + t]: the slots of token t that hold expert e, a bit each; list: expert | round << 16 (a
  // token that holds an expert in two slots takes another round of it); y: [token][slot][part][row];
  // ACT_X: the quantised rows
  const DownLds L = down_lds(a, step, lp);
  uint16_t *slots = reinterpret_cast<uint16_t *>(lds);
  int *list = reinterpret_cast<int *>(lds + L.list);
  float *y = reinterpret_cast<float *>(lds + L.y);
  uint8_t *lc = lds + L.x, *ls = lc;
  static_assert(DN_TOK * DN_K <= 64 * DN_WAVES, "a thread for each slot");
  const int my_e = tid < T_ * k ? idx[t0 * k + tid] : -1;
  const float my_w = tid < T_ * k ? w[t0 * k + tid] : 0.0f;
  for (int i = tid; i < E * DN_TOK / 2; i += 64 * DN_WAVES) reinterpret_cast<uint32_t *>(slots)[i] = 0;
  if (tid < DN_TOK) there[tid] = 0;
  if (tid == 0) repeats = 0;
  if constexpr (ACT == ACT_X) {
    ls = lc + (P + a.has_shared) * nbp * 16;
    const T *x = static_cast<const T *>(a.x);
    for (int h = tid; h < (P + a.has_shared) * nbp * 2; h += 64 * DN_WAVES) {
      const int row = h / (2 * nbp), hb = h - row * 2 * nbp, blk = hb >> 1, q = hb & 1;
      float va[8], vb[8];
      uint2 c = make_uint2(0, 0);
      uint32_t u = 127;
      if (blk < nb) {
        load8(x + ((int64_t)row * nb + blk) * 32 + 8 * q, va);
        load8(x + ((int64_t)row * nb + blk) * 32 + 16 + 8 * q, vb);
        c = mx_quant_half(va, vb, u);
      }
      *reinterpret_cast<uint2 *>(lc + h * 8) = c;
      if (q == 0) ls[h >> 1] = (uint8_t)u;
    }
  }
  __syncthreads();
  if (my_e >= 0 && my_e < E) {
    const int t = tid / k, j = tid - t * k;
    const uint32_t at = 16 * (t & 1);
    const uint32_t before = atomicOr(reinterpret_cast<uint32_t *>(slots) + (my_e * DN_TOK + t) / 2, 1u << (j + at));
    if (before >> at & 0xFFFF) repeats = 1;
    atomicOr(&there[t], 1u << j);
    weight[tid] = my_w;
  }
  __syncthreads();
  if (wv == 0) {  // the experts that these tokens hold, in order, and the shared one
    int n = 0;
    const bool twice = __builtin_amdgcn_readfirstlane(repeats) != 0;
    bool more = true;
    for (int round = 0; more; round++) {
      more = false;
      for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = min(e0 + lane, E - 1);
        const uint4 u = reinterpret_cast<const uint4 *>(slots)[2 * e], v = reinterpret_cast<const uint4 *>(slots)[2 * e + 1];
        bool held = e0 + lane < E && (u.x | u.y | u.z | u.w | v.x | v.y | v.z | v.w) != 0;
        if (twice) {
          const uint32_t words[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
          int most = 0;  // slots of one token
#pragma unroll
          for (int i = 0; i < 8; i++) most = max(most, max(__popc(words[i] & 0xFFFF), __popc(words[i] >> 16)));
          held = held && most > round;
          more = more || __ballot(held && most > round + 1) != 0;
        }
        const uint64_t who = __ballot(held);
        if (held) list[n + __popcll(who & ((1ull << lane) - 1))] = e | round << 16;
        n += __popcll(who);
      }
    }
    if (a.has_shared && lane == 0) list[n] = E;
    if (lane == 0) n_entries = n + a.has_shared;
  }
  __syncthreads();
  // this wavefront's entries: first, first + stride, ..; its K groups of each: part, part + parts, ..
  const int parts = 1 << lp, part = wv & (parts - 1), first = wv >> lp, stride = DN_WAVES >> lp;
  const int units = (__builtin_amdgcn_readfirstlane(n_entries) - first + stride - 1) / stride * ((ng - part + parts - 1) >> lp);
  const int rows = P + a.has_shared * a.M;
  v4f acc[RT] = {};
  Group wg[RT], act;
  int slot = -1;  // of this lane's token, that the unit is for, or -1
  // A token's lanes take the row of the slot that holds the expert. A token without one (of 16 that
  // pick 8 of 256 experts, 15 have none) reads past the buffer's end: zeros, and no access to the
  // cache, whose rate this kernel would otherwise meet.
  [[maybe_unused]] const auto acr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(a.ac), 0, rows * nbp * 16, 0x00027000);
  [[maybe_unused]] const auto asr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(a.as), 0, rows * nbp, 0x00027000);
  // weights and activations of the next unit together, since loads arrive in order
  int at = first, g = part;
  auto load = [&]() {
    const int entry = __builtin_amdgcn_readfirstlane(list[at]), e = entry & 0xFFFF;
    const auto wc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(a.wc) + (int64_t)e * a.wc_stride + (int64_t)n0 * nb * 16, 0, nrows * nb * 16, 0x00027000);
    const auto ws = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(a.ws) + (int64_t)e * a.ws_stride + (int64_t)n0 * nb, 0, nrows * nb, 0x00027000);
#pragma unroll
    for (int i = 0; i < RT; i++) {
      const uint32_t row = (uint32_t)(16 * i + li) * (uint32_t)nb;
      if constexpr (SL != SC_BYTES) {
        const uint4 u = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(ws, row + min(g * 16, nb - 16), 0, 0));
        wg[i].u[0] = u.x, wg[i].u[1] = u.y, wg[i].u[2] = u.z, wg[i].u[3] = u.w;
      }
#pragma unroll
      for (int s = 0; s < 4; s++) {
        const int b = min(g * 16 + 4 * s + lq, nb - 1);  // past K: activations of zero
        wg[i].c[s] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(wc, (row + b) * 16, 0, 0));
        if constexpr (SL == SC_BYTES) wg[i].u[s] = __builtin_amdgcn_raw_buffer_load_b8(ws, row + b, 0, 0);
      }
    }
    uint32_t mine = li < T_ ? (e < E ? slots[e * DN_TOK + li] : 1u) : 0u;
    for (int i = entry >> 16; i > 0; i--) mine &= mine - 1;
    const int j = mine ? (e < E ? __builtin_ctz(mine) : k) : -1, p = j < k ? (t0 + li) * k + j : P + t0 + li;
    slot = j;
    if constexpr (ACT == ACT_X) {
      const int row = mine ? p : 0;
      load_group<SC_FULL>(lc + row * nbp * 16, ls + row * nbp, nbp, g, lq, act);
    } else {
      const uint32_t row = (uint32_t)p * (uint32_t)nbp;
      const uint4 u = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(asr, mine ? row + g * 16 : ~0u, 0, 0));
      act.u[0] = u.x, act.u[1] = u.y, act.u[2] = u.z, act.u[3] = u.w;
#pragma unroll
      for (int s = 0; s < 4; s++)
        act.c[s] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(acr, mine ? (row + g * 16 + 4 * s + lq) * 16 : ~0u, 0, 0));
    }
    g += parts;
    if (g >= ng) g = part, at += stride;
  };
  if (units > 0) load();
  int cg = part;  // K group of the unit that is multiplied
  for (int u = 0; u < units; u++) {
#pragma unroll
    for (int i = 0; i < RT; i++) {
      end_group<SL>(wg[i], nb, cg);
#pragma unroll
      for (int s = 0; s < 4; s++)  // rows of the result: weight rows; columns: tokens
        acc[i] = mx_mfma16(wg[i].c[s], group_scale<SL>(wg[i], s, lq), act.c[s], group_scale<SC_FULL>(act, s, lq), acc[i]);
    }
    cg += parts;
    if (cg >= ng) {  // the expert is done
      cg = part;
#pragma unroll
      for (int i = 0; i < RT; i++) {
        if (slot >= 0 && 16 * i + 4 * lq < step)
          *reinterpret_cast<v4f *>(y + (((li * ks + slot) << lp) + part) * step + 16 * i + 4 * lq) = acc[i];
        acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    }
    if (u + 1 < units) load();
  }
  __syncthreads();
  const int t = tid / (16 * RT), r = tid % (16 * RT);
  if (t < T_ && r < nrows) {
    const uint32_t some = there[t];
    float s = 0.f;
    auto add = [&]<int PARTS>() {
      auto row = [&](int j) {
        const float *v = y + (t * ks + j) * PARTS * step + r;
        float sum = v[0];
#pragma unroll
        for (int i = 1; i < PARTS; i++) sum += v[i * step];
        return sum;
      };
#pragma unroll 4
      for (int j = 0; j < k; j++) {
        const float v = row(j);  // of an empty slot: whatever is there
        s = some >> j & 1 ? __builtin_fmaf(weight[t * k + j], v, s) : s;
      }
      if (a.has_shared) s += row(k);
    };
    switch (lp) {
      case 0: add.template operator()<1>(); break;
      case 1: add.template operator()<2>(); break;
      case 2: add.template operator()<4>(); break;
      default: add.template operator()<8>();
    }
    out[(int64_t)(t0 + t) * a.N + n0 + r] = (T)s;
  }
}

// Output rows of a workgroup: so many that the busiest CU has the least to do, a workgroup
// costing about six rows by itself. N = 6144 in 256 workgroups of 24 rows: every CU the same; in
// 384 of 16 a third of the CUs' time was idle.
constexpr int MX_CUS = 256;
static int down_step(int N) {
  int best = 16, cost = 1 << 30;
  for (int step = 8; step <= 32; step += 8) {
    const int groups = (N + step - 1) / step, c = (groups + MX_CUS - 1) / MX_CUS * (step + 6);
    if (c < cost) cost = c, best = step;
  }
  return best;
}

// Wavefronts (1 << lp) to an expert's K groups: so many that one token's experts end soonest, and
// the finer cut of two, which evens out a batch's (16 tokens over 64 experts of 4096 x 1920, 6 to a
// token: 42 us against 46.5 with whole experts; of 4096 x 4096, 8 to a token: 92 against 103), as
// far as the LDS of two workgroups to a CU goes. Nothing of the batch enters: the parts order the sums.
constexpr size_t DN_LDS = 80 * 1024;
static int down_parts(const MxArgs &a, int step) {
  const int ng = mx_padded(a.K) / 512, n = a.k + a.has_shared;
  int best = 0, cost = 1 << 30;
  for (int lp = 0; 1 << lp <= DN_WAVES && 1 << lp <= ng; lp++) {
    if (lp > 0 && down_lds(a, step, lp, DN_TOK).x > DN_LDS) break;
    const int lanes = DN_WAVES >> lp, c = (n + lanes - 1) / lanes * ((ng + (1 << lp) - 1) >> lp);
    if (c <= cost) cost = c, best = lp;
  }
  return best;
}

// The rows of one token in LDS, when mx_down_kernel quantises them itself
static size_t down_rows_lds(const MxArgs &a) {
  return ((size_t)a.M * a.k + (size_t)a.M * a.has_shared) * (mx_padded(a.K) / 32) * 17;
}

// More than 16 tokens go through the weights of their experts once for each 16: worth it while
// that reads less than 1.7 times the distinct experts of an even route. Of 256 experts of
// 6144 x 2048, 8 to a token: 24 tokens 267 -> 180 us, 32 323 -> 228 (1.27 times), 48 398 -> 338
// (1.55 times), 56 429 -> 396 (1.71 times, not taken); 64 (1.85 times) 450 and 445: no gain.
bool mx_down_fused(const MxArgs &a) {
  if (a.k > DN_K) return false;
  if (a.M <= DN_TOK) return true;
  if (a.M > 4 * DN_TOK) return false;
  auto hit = [&](int tokens) { return 1.0 - std::pow(1.0 - (double)a.k / a.E, tokens); };
  return a.M / DN_TOK * hit(DN_TOK) + hit(a.M % DN_TOK) <= 1.7 * hit(a.M);
}
bool mx_down_from_x(const MxArgs &a) { return a.M == 1 && (size_t)a.E * (DN_TOK * 2 + 4) + down_rows_lds(a) <= 46 * 1024; }
// One row quantised by every workgroup
bool mx_gemv_from_x(const MxArgs &a) { return a.M == 1 && mx_padded(a.K) / 32 * 17 <= 48 * 1024; }

static ScaleLoad scale_load(const MxArgs &a) {
  if (a.K < 512) return SC_BYTES;
  return (a.K / 32) % 16 == 0 && (uintptr_t)a.ws % 16 == 0 && a.ws_stride % 16 == 0 ? SC_FULL : SC_ANY;
}

template <MxMode MODE, typename T, int NT, MxAct ACT>
static hipError_t launch_gemv_al(const MxArgs &a, int ny, size_t lds, hipStream_t s) {
  auto go = [&]<ScaleLoad SL>() {
    constexpr int rows = gate_up_halves<MODE, ACT, SL>() ? 8 : 16;  // output columns of a workgroup
    const dim3 g((unsigned)((a.N + rows - 1) / rows), (unsigned)ny), b(256);
    hipLaunchKernelGGL((mx_gemv_kernel<MODE, T, NT, ACT, SL>), g, b, lds, s, a);
  };
  switch (scale_load(a)) {
    case SC_FULL: go.template operator()<SC_FULL>(); break;
    case SC_ANY: go.template operator()<SC_ANY>(); break;
    default: go.template operator()<SC_BYTES>();
  }
  return hipGetLastError();
}

template <MxMode MODE, typename T>
static hipError_t launch_gemv_t(const MxArgs &a, hipStream_t s) {
  const int64_t P = (int64_t)a.M * a.k;
  const size_t xlds = (size_t)(mx_padded(a.K) / 32) * 17;
  if constexpr (MODE == MX_LINEAR) {
    if (a.x) return launch_gemv_al<MODE, T, 1, ACT_X>(a, 1, xlds, s);
    if (a.M <= 16) return launch_gemv_al<MODE, T, 1, ACT_WS>(a, 1, 0, s);
    if (a.M <= 32) return launch_gemv_al<MODE, T, 2, ACT_WS>(a, 1, 0, s);
    return launch_gemv_al<MODE, T, 4, ACT_WS>(a, (a.M + 63) / 64, 0, s);
  } else {
    const int ny = a.has_shared + (int)(P < a.E ? P : a.E);
    if constexpr (MODE == MX_GATEUP)
      if (a.x) return launch_gemv_al<MODE, T, 1, ACT_X>(a, ny, xlds, s);
    return launch_gemv_al<MODE, T, 1, ACT_WS>(a, ny, 0, s);
  }
}

hipError_t launch_mx_gemv(MxMode mode, int dtype, const MxArgs &a, hipStream_t s) {
  if (mode == MX_DOWN) return launch_gemv_t<MX_DOWN, float>(a, s);
  if (mode == MX_LINEAR)
    return dtype == COLI_F32 ? launch_gemv_t<MX_LINEAR, float>(a, s)
         : dtype == COLI_BF16 ? launch_gemv_t<MX_LINEAR, bf16_t>(a, s) : launch_gemv_t<MX_LINEAR, f16_t>(a, s);
  return dtype == COLI_F32 ? launch_gemv_t<MX_GATEUP, float>(a, s)
       : dtype == COLI_BF16 ? launch_gemv_t<MX_GATEUP, bf16_t>(a, s) : launch_gemv_t<MX_GATEUP, f16_t>(a, s);
}

template <typename T>
static hipError_t launch_down_t(const MxArgs &a, const int32_t *idx, const float *w, void *out, hipStream_t s) {
  const int step = down_step(a.N), lp = down_parts(a, step);
  const dim3 g((unsigned)((a.N + step - 1) / step), (unsigned)((a.M + DN_TOK - 1) / DN_TOK)), b(64 * DN_WAVES);
  const size_t lds = down_lds(a, step, lp).x + (a.x ? down_rows_lds(a) : 0);
  auto go = [&]<MxAct ACT, ScaleLoad SL, int RT>() {
    static PerDevice allowed;
    auto kernel = mx_down_kernel<T, ACT, SL, RT>;
    if (const hipError_t st = allow_lds(allowed, kernel, 144 * 1024); st != hipSuccess) return st;
    hipLaunchKernelGGL(kernel, g, b, lds, s, a, step, lp, idx, w, (T *)out);
    return hipGetLastError();
  };
  auto pick = [&]<MxAct ACT, ScaleLoad SL>() {
    return step <= 16 ? go.template operator()<ACT, SL, 1>() : go.template operator()<ACT, SL, 2>();
  };
  auto with_x = [&]<ScaleLoad SL>() {
    return a.x ? pick.template operator()<ACT_X, SL>() : pick.template operator()<ACT_WS, SL>();
  };
  switch (scale_load(a)) {
    case SC_FULL: return with_x.template operator()<SC_FULL>();
    case SC_ANY: return with_x.template operator()<SC_ANY>();
    default: return with_x.template operator()<SC_BYTES>();
  }
}

hipError_t launch_mx_down(const MxArgs &a, const int32_t *idx, const float *w, void *out, int dtype, hipStream_t s) {
  if (dtype == COLI_F32) return launch_down_t<float>(a, idx, w, out, s);
  if (dtype == COLI_BF16) return launch_down_t<bf16_t>(a, idx, w, out, s);
  return launch_down_t<f16_t>(a, idx, w, out, s);
}

// out_t = sum_j w_tj y_tj in slot order, plus the shared expert's row; empty slots skipped. Four columns of a
// token to a thread, the rows of eight slots under way at a time; they are used once and pass the caches by. Down
// products of 2048 tokens with 8 slots and a shared expert, H = 6144: MXFP4 584 us (a slot after another,
// through the caches: 595); int8 828 to 854 by the card, all of these within 5 of each other.
template <typename T>
__global__ __launch_bounds__(256) void mx_combine_kernel(const float *__restrict__ y, const int32_t *__restrict__ idx,
                                                         const float *__restrict__ w, int T_, int k, int E, int H,
                                                         int has_shared, T *__restrict__ out) {
  constexpr int AHEAD = 8;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x, per = (uint32_t)H / 4;  // T k < 2^16: fewer than 2^32
  const uint32_t t = i / per, h = i - t * per;
  if (t >= (uint32_t)T_) return;
  const v4f *py = reinterpret_cast<const v4f *>(y) + h;
  v4f s = {0.f, 0.f, 0.f, 0.f}, last = s;
  if (has_shared) last = __builtin_nontemporal_load(py + ((int64_t)T_ * k + t) * per);
  for (int j0 = 0; j0 < k; j0 += AHEAD) {
    v4f v[AHEAD];
    bool there[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      const int64_t p = (int64_t)t * k + j0 + j;
      const int e = j0 + j < k ? idx[p] : -1;
      there[j] = e >= 0 && e < E;
      if (there[j]) v[j] = __builtin_nontemporal_load(py + p * per);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      if (!there[j]) continue;
      const float wt = w[(int64_t)t * k + j0 + j];
#pragma unroll
      for (int r = 0; r < 4; r++) s[r] = __builtin_fmaf(wt, v[j][r], s[r]);
    }
  }
  if (has_shared) s += last;
  typedef T v4 __attribute__((ext_vector_type(4)));
  v4 o;
#pragma unroll
  for (int r = 0; r < 4; r++) o[r] = (T)s[r];
  *reinterpret_cast<v4 *>(out + (int64_t)i * 4) = o;
}

hipError_t launch_mx_combine(const float *y, const int32_t *idx, const float *w, int T, int k, int E, int H,
                             int has_shared, void *out, int dtype, hipStream_t s) {
  const dim3 g((unsigned)(((int64_t)T * H / 4 + 255) / 256)), b(256);
  if (dtype == COLI_F32)
    hipLaunchKernelGGL(mx_combine_kernel<float>, g, b, 0, s, y, idx, w, T, k, E, H, has_shared, (float *)out);
  else if (dtype == COLI_BF16)
    hipLaunchKernelGGL(mx_combine_kernel<bf16_t>, g, b, 0, s, y, idx, w, T, k, E, H, has_shared, (bf16_t *)out);
  else
    hipLaunchKernelGGL(mx_combine_kernel<f16_t>, g, b, 0, s, y, idx, w, T, k, E, H, has_shared, (f16_t *)out);
  return hipGetLastError();
}

}  // namespace coli
