// int8_gemv.hip — int8 products of few rows with token and channel scales, bound by the weights' way
// from HBM: dense rows, the experts' gate/up rows with SiLU*up and their down rows over a route
// (batch-union: colibri-strix README, "What's implemented"), on the 16x16x64 int8 matrix instruction.
//
// A workgroup (4 wavefronts) owns 16 weight rows (of each matrix) and chunks of 16 NT rows of
// activations. The wavefronts take the K groups (256 contiguous bytes of a row) in turn, weights
// straight into the operand registers; their integer sums meet in LDS. One row of activations (x in
// ACT_X) is quantised by every workgroup itself while its first two groups of weights are under way,
// which saves a launch. bf16: one row of 12288 x 6144 13 us (75 MB, 12 us at the 6.3 TB/s of a plain read);
// gate/up of one token over 9 experts of 6144 x 2048 43 to 49 us by the card (226 MB), of 16 tokens over 256 406 to
// 423 (2.58 GB, 6.1 to 6.3 TB/s). One group under way and four workgroups to a CU where activations come from the
// workspace: gate/up of 16 tokens over 64 experts of 2048 x 1024 60 -> 52 us, of 256 the same.
//
// i8_down_kernel: 16 tokens over 256 experts of 6144 x 2048 232 to 241 us (1.29 GB, 5.4 to 5.6 TB/s with the
// quantisation's launch), one token 23 to 27 (113 MB; a bare read of them in this order takes 18.6).
#include "int8_impl.h"

namespace coli {

// 16 chunks (of 16 inputs) of a row, as a lane of the matrix instruction takes them: in step s the
// chunk 4 s + l / 16
struct I8Group {
  uint4 c[4];
};

__device__ __forceinline__ void i8_load_group(const int8_t *row, int nc, int g, int lq, I8Group &o) {
#pragma unroll
  for (int s = 0; s < 4; s++)  // past the row: its last chunk; it meets activations of zero
    o.c[s] = *reinterpret_cast<const uint4 *>(row + min(g * 16 + 4 * s + lq, nc - 1) * 16);
}

// One row x -> codes in LDS (inputs K .. pitch: zeros) and its scale, by 256 threads. The first XP
// pieces of 8 values of each thread come in v, loaded ahead.
constexpr int XP = 4;
template <typename T>
__device__ __forceinline__ void i8_load_x(const T *x, int n, int tid, float (&v)[XP][8]) {
#pragma unroll
  for (int i = 0; i < XP; i++) load8(x + min(tid + 256 * i, n - 1) * 8, v[i]);
}

template <typename T>
__device__ __forceinline__ float i8_quantise_x(const T *x, int n, int np, int tid, const float (&v)[XP][8], uint32_t *tops,
                                               int8_t *lc) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < XP; i++) top = i8_top8(v[i], top);  // a piece twice does not change it
  for (int u = tid + 256 * XP; u < n; u += 256) {
    float t[8];
    load8(x + u * 8, t);
    top = i8_top8(t, top);
  }
  top = wave_top(top);
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  const I8Row row = i8_row(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll
  for (int i = 0; i < XP; i++) {
    const int u = tid + 256 * i;
    if (u < n) *reinterpret_cast<uint2 *>(lc + u * 8) = i8_codes8(v[i], row);
  }
  for (int u = tid + 256 * XP; u < n; u += 256) {
    float t[8];
    load8(x + u * 8, t);
    *reinterpret_cast<uint2 *>(lc + u * 8) = i8_codes8(t, row);
  }
  for (int u = n + tid; u < np; u += 256) *reinterpret_cast<uint2 *>(lc + u * 8) = make_uint2(0, 0);
  return row.s;
}

enum I8Act { I8_ACT_WS, I8_ACT_X };  // activations: quantised in the workspace; one row of x

// Do eight gate rows and the eight up rows of the same features share a tile of the matrix
// instruction? One token: 52 -> 47 us, the workgroups being twice as many and half as long.
template <I8Mode MODE, I8Act ACT>
constexpr bool i8_gate_up_halves() {
  return MODE == I8_GATEUP && ACT == I8_ACT_X;
}

template <I8Mode MODE, typename T, int NT, I8Act ACT>
__global__ __launch_bounds__(256, ACT == I8_ACT_X || NT == 4 ? 2 : 4) void i8_gemv_kernel(I8Args a) {
  constexpr bool HALVES = i8_gate_up_halves<MODE, ACT>();
  constexpr int NMAT = MODE == I8_GATEUP && !HALVES ? 2 : 1;
  constexpr int D = ACT == I8_ACT_X ? 2 : 1;  // groups under way
  static_assert(ACT == I8_ACT_WS || (NT == 1 && MODE != I8_DOWN));
  extern __shared__ __align__(16) int8_t lds[];  // ACT_X: the quantised row
  __shared__ int red[4][NMAT][NT][16][17];
  __shared__ uint32_t tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * (HALVES ? 8 : 16);
  const int K = a.K, nc = K / 16, pitch = i8_padded(K), ng = pitch / 256;
  const int ngw = (ng - wv + 3) / 4;  // groups of this wavefront: wv, wv + 4, ..
  // the rows of activations: first .. first + n - 1 of perm (routed) or of the tokens
  int e = 0, first = 0, n = a.M;
  bool routed = false;
  if constexpr (MODE == I8_LINEAR) {
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
  float xv[XP][8];
  const T *x = static_cast<const T *>(a.x);
  if constexpr (ACT == I8_ACT_X) i8_load_x(x, K / 8, tid, xv);
  const int8_t *wq[NMAT];
#pragma unroll
  for (int m = 0; m < NMAT; m++)
    wq[m] = a.wq + (int64_t)e * a.wq_stride +
            (HALVES ? (int64_t)(li >> 3) * a.N + min(n0 + (li & 7), a.N - 1) : (int64_t)m * a.N + min(n0 + li, a.N - 1)) * K;
  I8Group w[D][NMAT], act[D][NT];
  float xs = 0.0f;  // ACT_X: the row's scale
  for (int c = 0; c < n; c += 16 * NT) {
    const int8_t *aq[NT];
    if constexpr (ACT == I8_ACT_WS) {
#pragma unroll
      for (int q = 0; q < NT; q++) {
        const int ci = first + min(c + 16 * q + li, n - 1);
        int64_t arow = ci;
        if constexpr (MODE != I8_LINEAR) {
          const int64_t pair = routed ? a.perm[ci] : P + ci;
          arow = MODE == I8_DOWN ? pair : (routed ? pair / a.k : ci);
        }
        aq[q] = a.aq + arow * pitch;
      }
    }
    auto load_act = [&](int d, int i) {
#pragma unroll
      for (int q = 0; q < NT; q++) i8_load_group(aq[q], pitch / 16, min(wv + 4 * i, ng - 1), lq, act[d][q]);
    };
    auto load = [&](int d, int i) {
#pragma unroll
      for (int m = 0; m < NMAT; m++) i8_load_group(wq[m], nc, min(wv + 4 * i, ng - 1), lq, w[d][m]);
      if constexpr (ACT == I8_ACT_WS) load_act(d, i);
    };
    // without a branch, so that the compiler counts the loads and the row's conversion waits for x alone
#pragma unroll
    for (int d = 0; d < D; d++) load(d, d);
    if constexpr (ACT == I8_ACT_X) {
      xs = i8_quantise_x(x, K / 8, pitch / 8, tid, xv, tops, lds);
      __syncthreads();
      aq[0] = lds;
    }
    v4i32 acc[NT][NMAT] = {};
    for (int i0 = 0; i0 < ngw; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; d++) {
        if (i0 + d < ngw) {
          if constexpr (ACT == I8_ACT_X) load_act(d, i0 + d);
#pragma unroll
          for (int s = 0; s < 4; s++)
#pragma unroll
            for (int q = 0; q < NT; q++)
#pragma unroll
              for (int m = 0; m < NMAT; m++) acc[q][m] = i8_mfma16(act[d][q].c[s], w[d][m].c[s], acc[q][m]);
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
    const float *ws = a.ws + (int64_t)e * a.ws_stride + n0 + tc;
#pragma unroll
    for (int q = 0; q < NT; q++) {
      const int row = c + 16 * q + tr;
      if (row < n && n0 + tc < a.N && (!HALVES || tc < 8)) {
        const int ci = first + row;
        int64_t orow = ci, arow = ci;
        if constexpr (MODE != I8_LINEAR) {
          orow = routed ? (int64_t)a.perm[ci] : P + ci;
          arow = MODE == I8_DOWN ? orow : (routed ? orow / a.k : ci);
        }
        const float s = ACT == I8_ACT_X ? xs : a.as[arow];
        auto sum = [&](int m) {  // of the gate's or only matrix, of the up's
          const int i = HALVES ? 0 : m, c = HALVES ? tc + 8 * m : tc;
          return red[0][i][q][tr][c] + red[1][i][q][tr][c] + red[2][i][q][tr][c] + red[3][i][q][tr][c];
        };
        auto value = [&](int m) { return i8_value(sum(m), s, ws[(int64_t)m * a.N]); };
        const int64_t o = orow * a.N + n0 + tc;
        if constexpr (MODE == I8_GATEUP)
          static_cast<T *>(a.out)[o] = (T)i8_product(i8_silu(value(0)), value(1));
        else if constexpr (MODE == I8_DOWN)
          static_cast<float *>(a.out)[o] = value(0);
        else
          static_cast<T *>(a.out)[o] = (T)i8_biased(sum(0), s, ws[0], a.bias ? a.bias[n0 + tc] : 0.0f);
      }
    }
    if (c + 16 * NT < n) __syncthreads();
  }
}

// ------------------------------------------------------------------ down with its combine
constexpr int DN_TOK = 16, DN_K = 16, DN_WAVES = 8;
constexpr int DN_XP = 6;  // pieces of 8 values of h in a thread's registers, one token

// Dynamic LDS of i8_down_kernel, bytes: slots first, then these; with ACT_X (one token, which needs no
// list) the scales first and the quantised rows last
struct I8DownLds {
  size_t list, scales, y, x;
};
__host__ __device__ inline I8DownLds i8_down_lds(const I8Args &a, int step, int lp, int tokens) {
  I8DownLds L;
  const size_t rows = (size_t)tokens * (a.k + a.has_shared);
  L.list = a.x ? 0 : (size_t)a.E * DN_TOK * 2;
  L.scales = a.x ? 0 : L.list + ((size_t)tokens * a.k + 1 + 3) / 4 * 16;
  L.y = L.scales + rows * step * sizeof(float);
  L.x = L.y + (rows << lp) * step * sizeof(int);
  return L;
}

// The down product of up to 16 tokens with its weighted combine. A workgroup (8 wavefronts) owns `step` output
// rows, RT 16-row tiles of the matrix instruction, and goes through all experts that its tokens hold, a token to a
// column; rows past them, like rows past N, read past their buffer's end, which gives zeros without an access. 1 <<
// lp wavefronts share an expert's K groups; what each sums for a (token, slot) has its own place in LDS, and at the
// end the parts, then the weighted slots, then the shared expert's row are added in order: a token's row does not
// depend on the tokens beside it.
template <typename T, I8Act ACT, int RT>
__global__ __launch_bounds__(64 * DN_WAVES) void i8_down_kernel(I8Args a, int step, int lp, const int32_t *__restrict__ idx,
                                                               const float *__restrict__ w, T *__restrict__ out) {
  extern __shared__ __align__(16) int8_t lds[];
  __shared__ float weight[DN_TOK * DN_K], row_scale[DN_TOK * (DN_K + 1)];
  __shared__ uint32_t tops[DN_K + 1];  // ACT_X: the rows' largest magnitudes
  __shared__ uint32_t there[DN_TOK];  // slots of a token that hold an expert, a bit each
  __shared__ int n_entries, repeats;  // repeats: some token holds an expert in two slots
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * step, nrows = min(step, a.N - n0);
  const int K = a.K, nc = K / 16, pitch = i8_padded(K), ng = pitch / 256;
  const int T_ = a.M, k = a.k, E = a.E, P = T_ * k, ks = k + a.has_shared;
  // slots[e * 16 + t]: the slots of token t that hold expert e, a bit each; list: expert | round << 16 (a
  // token that holds an expert in two slots takes another round of it); scales: [token][slot][row] of the
  // weight rows; y: [token][slot][part][row]; ACT_X: the quantised rows
  const I8DownLds L = i8_down_lds(a, step, lp, T_);
  uint16_t *slots = reinterpret_cast<uint16_t *>(lds);
  int *list = reinterpret_cast<int *>(lds + L.list);
  float *scales = reinterpret_cast<float *>(lds + L.scales);
  int *y = reinterpret_cast<int *>(lds + L.y);
  int8_t *lx = lds + L.x;
  static_assert(DN_TOK * DN_K <= 64 * DN_WAVES, "a thread for each slot");
  constexpr bool ONE = ACT == I8_ACT_X;  // one token: an entry is a slot
  // this wavefront's entries: first, first + stride, ..; its K groups of each: part, part + parts, ..
  const int parts = 1 << lp, part = wv & (parts - 1), first = wv >> lp, stride = DN_WAVES >> lp;
  const int ngw = (ng - part + parts - 1) >> lp;
  v4i32 acc[RT] = {};
  I8Group wg[RT], act;
  int at = first, g = part;  // entry and group of the unit whose weights are loaded next
  // one token: the expert of slot `lane`, E for the shared one's, -1 for none and past the slots
  int slot_e = ONE ? idx[min(lane, k - 1)] : -1;
  if constexpr (ONE) slot_e = lane < k ? (slot_e < E ? slot_e : -1) : lane < ks ? E : -1;
  auto expert_of = [&](int entry) -> int {  // E: the shared one; -1: none
    if constexpr (ONE) {
      return __builtin_amdgcn_readlane(slot_e, min(entry, DN_K + 1));
    } else {
      return __builtin_amdgcn_readfirstlane(list[entry]) & 0xFFFF;
    }
  };
  auto load_weights = [&]() {
    const int e = expert_of(at);
    const auto wq = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(a.wq) + (int64_t)max(e, 0) * a.wq_stride + (int64_t)n0 * K,
                                                      0, e < 0 ? 0 : nrows * K, 0x00027000);
#pragma unroll
    for (int i = 0; i < RT; i++) {
      const uint32_t row = (uint32_t)(16 * i + li) * (uint32_t)K;
#pragma unroll
      for (int s = 0; s < 4; s++)  // past K: activations of zero
        wg[i].c[s] = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(wq, row + min(g * 16 + 4 * s + lq, nc - 1) * 16, 0, 0));
    }
    g += parts;
    if (g >= ng) g = part, at += stride;
  };
  // the scale of row r of expert e
  auto load_scale = [&](int e, int r) { return a.ws[(int64_t)max(e, 0) * a.ws_stride + min(n0 + r, a.N - 1)]; };
  // One token: all first loads without a branch, so that the compiler counts them, in the order in which
  // they are waited for: experts, rows of h, scales, weights. (With a branch between, or the scales
  // behind the weights, everything before the products waits for the first weights.)
  const int my_e = idx[min(tid, T_ * k - 1)];
  const float my_w = w[min(tid, T_ * k - 1)];
  int units = 0;
  [[maybe_unused]] float xv[ONE ? DN_XP : 1][8], my_scale[2] = {};
  if constexpr (ONE) {
    static_assert((DN_K + 1) * 32 <= 2 * 64 * DN_WAVES, "two scales to a thread");
    const int n = ks * (K / 8);
#pragma unroll
    for (int q = 0; q < DN_XP; q++) load8(static_cast<const T *>(a.x) + min(tid + 64 * DN_WAVES * q, n - 1) * 8, xv[q]);
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int i = min(tid + 64 * DN_WAVES * q, ks * step - 1), j = i / step;
      my_scale[q] = load_scale(__shfl(slot_e, j), i - j * step);
    }
    units = max(0, (ks - first + stride - 1) / stride) * ngw;
    load_weights();  // of a wavefront without a unit: no access
    if (tid <= DN_K) tops[tid] = 0;
  } else {
    for (int i = tid; i < E * DN_TOK / 2; i += 64 * DN_WAVES) reinterpret_cast<uint32_t *>(slots)[i] = 0;
    if (tid == 0) repeats = 0;
    for (int i = tid; i < T_ * ks * step; i += 64 * DN_WAVES) {
      const int ts = i / step, t = ts / ks, j = ts - t * ks, e = j < k ? idx[t * k + j] : E;
      scales[i] = load_scale(e < E || j == k ? e : -1, i - ts * step);
    }
  }
  if (tid < DN_TOK) there[tid] = 0;
  if constexpr (ACT == I8_ACT_WS)
    for (int i = tid; i < T_ * ks; i += 64 * DN_WAVES) {
      const int t = i / ks, j = i - t * ks;
      row_scale[i] = a.as[j < k ? t * k + j : P + t];
    }
  __syncthreads();
  if (tid < T_ * k && my_e >= 0 && my_e < E) {
    const int t = tid / k, j = tid - t * k;
    if constexpr (!ONE) {
      const uint32_t half = 16 * (t & 1);
      const uint32_t before = atomicOr(reinterpret_cast<uint32_t *>(slots) + (my_e * DN_TOK + t) / 2, 1u << (j + half));
      if (before >> half & 0xFFFF) repeats = 1;
    }
    atomicOr(&there[t], 1u << j);
    weight[tid] = my_w;
  }
  if constexpr (!ONE) __syncthreads();
  if (!ONE && wv == 0) {  // the experts that these tokens hold, in order, and the shared one
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
  if constexpr (!ONE) __syncthreads();
  if constexpr (!ONE) {
    units = (__builtin_amdgcn_readfirstlane(n_entries) - first + stride - 1) / stride * ngw;
    if (units > 0) load_weights();
  }
  const int rows = P + a.has_shared * a.M;
  // A token's lanes take the row of the slot that holds the expert. A token without one (of 16 that
  // pick 8 of 256 experts, 15 have none) reads past the buffer's end: zeros, and no access to the
  // cache, whose rate this kernel would otherwise meet.
  [[maybe_unused]] const auto aqr = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(a.aq), 0, rows * pitch, 0x00027000);
  int slot = -1;  // of this lane's token, that the unit is for, or -1
  int mat = first, cg = part;  // entry and group of the unit that is multiplied
  auto load_act = [&]() {
    if constexpr (ONE) {  // columns without a token are of no use
      slot = mat;
      const int8_t *row = lx + min(mat, ks - 1) * pitch;
#pragma unroll
      for (int s = 0; s < 4; s++) act.c[s] = *reinterpret_cast<const uint4 *>(row + (cg * 16 + 4 * s + lq) * 16);
    } else {
      const int entry = __builtin_amdgcn_readfirstlane(list[mat]), e = entry & 0xFFFF;
      uint32_t mine = li < T_ ? (e < E ? slots[e * DN_TOK + li] : 1u) : 0u;
      for (int i = entry >> 16; i > 0; i--) mine &= mine - 1;
      const int j = mine ? (e < E ? __builtin_ctz(mine) : k) : -1;
      slot = j;
      const uint32_t row = (uint32_t)(j < k ? li * k + j : P + li) * (uint32_t)pitch;
#pragma unroll
      for (int s = 0; s < 4; s++)
        act.c[s] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(aqr, mine ? row + (cg * 16 + 4 * s + lq) * 16 : ~0u, 0, 0));
    }
  };
  if constexpr (ONE) {
    // K / 8 is a multiple of 16: 16 lanes hold pieces of one row
    const int per = K / 8, n = ks * per;
#pragma unroll
    for (int q = 0; q < DN_XP; q++) {
      const int u = tid + 64 * DN_WAVES * q;
      uint32_t top = i8_top8(xv[q], 0);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
      if ((lane & 15) == 0 && u < n) atomicMax(&tops[u / per], top);
    }
    __syncthreads();
    if (tid < ks) row_scale[tid] = i8_scale(tops[tid]);
#pragma unroll
    for (int q = 0; q < 2; q++)
      if (tid + 64 * DN_WAVES * q < ks * step) scales[tid + 64 * DN_WAVES * q] = my_scale[q];
#pragma unroll
    for (int q = 0; q < DN_XP; q++) {
      const int u = tid + 64 * DN_WAVES * q, r = u / per;
      if (u < n) *reinterpret_cast<uint2 *>(lx + r * pitch + (u - r * per) * 8) = i8_codes8(xv[q], i8_row(tops[r]));
    }
    for (int i = tid; i < ks * (pitch / 8 - per); i += 64 * DN_WAVES) {  // up to 16 pieces a row
      const int r = i / (pitch / 8 - per);
      *reinterpret_cast<uint2 *>(lx + r * pitch + K + (i - r * (pitch / 8 - per)) * 8) = make_uint2(0, 0);
    }
    __syncthreads();
  }
  if (ONE || units > 0) load_act();
  for (int u = 0; u < units; u++) {
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int s = 0; s < 4; s++)  // rows of the result: weight rows; columns: tokens
        acc[i] = i8_mfma16(wg[i].c[s], act.c[s], acc[i]);
    cg += parts;
    if (cg >= ng) {  // the entry is done
      cg = part;
      mat += stride;
#pragma unroll
      for (int i = 0; i < RT; i++) {
        if ((ONE ? li == 0 : slot >= 0) && 16 * i + 4 * lq < step)
          *reinterpret_cast<v4i32 *>(y + (((li * ks + slot) << lp) + part) * step + 16 * i + 4 * lq) = acc[i];
        acc[i] = v4i32{0, 0, 0, 0};
      }
    }
    if (u + 1 < units) load_weights(), load_act();
  }
  __syncthreads();
  // the parts of every (token, slot, row), over its scale
  auto sum_parts = [&]<int PARTS>() {
    for (int i = tid; i < T_ * ks * step; i += 64 * DN_WAVES) {
      const int ts = i / step, r = i - ts * step;
      const int *v = y + ts * PARTS * step + r;
      int sum = v[0];
#pragma unroll
      for (int p = 1; p < PARTS; p++) sum += v[p * step];
      scales[i] = i8_value(sum, row_scale[ts], scales[i]);
    }
  };
  switch (lp) {
    case 0: sum_parts.template operator()<1>(); break;
    case 1: sum_parts.template operator()<2>(); break;
    case 2: sum_parts.template operator()<4>(); break;
    default: sum_parts.template operator()<8>();
  }
  __syncthreads();
  const int t = tid / (16 * RT), r = tid % (16 * RT);
  if (t < T_ && r < nrows) {
    const uint32_t some = there[t];
    const float *v = scales + t * ks * step + r;
    float s = 0.f;
#pragma unroll 4
    for (int j = 0; j < k; j++) s = some >> j & 1 ? __builtin_fmaf(weight[t * k + j], v[j * step], s) : s;  // an empty slot's: whatever is there
    if (a.has_shared) s += v[k * step];
    out[(int64_t)t * a.N + n0 + r] = (T)s;
  }
}

// Output rows of a workgroup: so many that the busiest CU has the least to do, a workgroup
// costing about six rows by itself.
constexpr int I8_CUS = 256;
static int down_step(int N) {
  int best = 16, cost = 1 << 30;
  for (int step = 8; step <= 32; step += 8) {
    const int groups = (N + step - 1) / step, c = (groups + I8_CUS - 1) / I8_CUS * (step + 6);
    if (c < cost) cost = c, best = step;
  }
  return best;
}

// Wavefronts (1 << lp) to an expert's K groups: so many that one token's experts end soonest, and
// the finer cut of two, which evens out a batch's, as far as the LDS of two workgroups to a CU goes.
constexpr size_t DN_LDS = 80 * 1024;
static int down_parts(const I8Args &a, int step) {
  const int ng = i8_padded(a.K) / 256, n = a.k + a.has_shared;
  int best = 0, cost = 1 << 30;
  for (int lp = 0; 1 << lp <= DN_WAVES && 1 << lp <= ng; lp++) {
    if (lp > 0 && i8_down_lds(a, step, lp, DN_TOK).x > DN_LDS) break;
    const int lanes = DN_WAVES >> lp, c = (n + lanes - 1) / lanes * ((ng + (1 << lp) - 1) >> lp);
    if (c <= cost) cost = c, best = lp;
  }
  return best;
}

// The rows of one token in LDS, when i8_down_kernel quantises them itself
static size_t down_rows_lds(const I8Args &a) { return (size_t)(a.k + a.has_shared) * i8_padded(a.K); }

// Up to 16 tokens. us, this kernel and the two kernels of pairs' rows and their combine: 256 experts of
// 6144 x 2048 and a shared one, 8 to a token: 1 token 25 and 32, 4 80 and 87, 16 232 and 240, 20 (which
// would take their experts twice) 319 and 292; 64 of 2048 x 1024: 4 tokens 21 and 22, 16 42 and 38.
bool i8_down_fused(const I8Args &a) { return a.k <= DN_K && a.M <= DN_TOK; }
bool i8_down_from_x(const I8Args &a) {
  return a.M == 1 && a.k <= DN_K && (a.k + a.has_shared) * (a.K / 8) <= DN_XP * 64 * DN_WAVES;
}

template <typename T>
static hipError_t launch_down_t(const I8Args &a, const int32_t *idx, const float *w, void *out, hipStream_t s) {
  const int step = down_step(a.N), lp = down_parts(a, step);
  const dim3 g((unsigned)((a.N + step - 1) / step)), b(64 * DN_WAVES);
  const size_t lds = i8_down_lds(a, step, lp, a.M).x + (a.x ? down_rows_lds(a) : 0);
  auto go = [&]<I8Act ACT, int RT>() {
    static PerDevice allowed;
    auto kernel = i8_down_kernel<T, ACT, RT>;
    if (const hipError_t st = allow_lds(allowed, kernel, 144 * 1024); st != hipSuccess) return st;
    hipLaunchKernelGGL(kernel, g, b, lds, s, a, step, lp, idx, w, (T *)out);
    return hipGetLastError();
  };
  if (step <= 16) return a.x ? go.template operator()<I8_ACT_X, 1>() : go.template operator()<I8_ACT_WS, 1>();
  return a.x ? go.template operator()<I8_ACT_X, 2>() : go.template operator()<I8_ACT_WS, 2>();
}

hipError_t launch_i8_down(const I8Args &a, const int32_t *idx, const float *w, void *out, int dtype, hipStream_t s) {
  if (dtype == COLI_F32) return launch_down_t<float>(a, idx, w, out, s);
  if (dtype == COLI_BF16) return launch_down_t<bf16_t>(a, idx, w, out, s);
  return launch_down_t<f16_t>(a, idx, w, out, s);
}

// One row quantised by every workgroup
bool i8_gemv_from_x(const I8Args &a) { return a.M == 1 && i8_padded(a.K) <= 48 * 1024; }

template <I8Mode MODE, typename T>
static hipError_t launch_gemv_t(const I8Args &a, hipStream_t s) {
  const int64_t P = (int64_t)a.M * a.k;
  auto go = [&]<int NT, I8Act ACT>(int64_t ny) {
    constexpr int rows = i8_gate_up_halves<MODE, ACT>() ? 8 : 16;  // output columns of a workgroup
    hipLaunchKernelGGL((i8_gemv_kernel<MODE, T, NT, ACT>), dim3((unsigned)((a.N + rows - 1) / rows), (unsigned)ny), dim3(256),
                       ACT == I8_ACT_X ? i8_padded(a.K) : 0, s, a);
    return hipGetLastError();
  };
  if constexpr (MODE == I8_LINEAR) {
    if (a.x) return go.template operator()<1, I8_ACT_X>(1);
    if (a.M <= 16) return go.template operator()<1, I8_ACT_WS>(1);
    if (a.M <= 32) return go.template operator()<2, I8_ACT_WS>(1);
    return go.template operator()<4, I8_ACT_WS>((a.M + 63) / 64);
  } else {
    const int64_t ny = a.has_shared + (P < a.E ? P : a.E);
    if constexpr (MODE == I8_GATEUP)
      if (a.x) return go.template operator()<1, I8_ACT_X>(ny);
    return go.template operator()<1, I8_ACT_WS>(ny);
  }
}

hipError_t launch_i8_gemv(I8Mode mode, int dtype, const I8Args &a, hipStream_t s) {
  if (mode == I8_DOWN) return launch_gemv_t<I8_DOWN, float>(a, s);
  if (mode == I8_LINEAR)
    return dtype == COLI_F32 ? launch_gemv_t<I8_LINEAR, float>(a, s)
         : dtype == COLI_BF16 ? launch_gemv_t<I8_LINEAR, bf16_t>(a, s) : launch_gemv_t<I8_LINEAR, f16_t>(a, s);
  return dtype == COLI_F32 ? launch_gemv_t<I8_GATEUP, float>(a, s)
       : dtype == COLI_BF16 ? launch_gemv_t<I8_GATEUP, bf16_t>(a, s) : launch_gemv_t<I8_GATEUP, f16_t>(a, s);
}

}  // namespace coli
