// int8_gemv.hip — int8 products of few rows with token and channel scales, bound by the weights' way
// from HBM: dense rows, the experts' gate/up rows with SiLU*up and their down rows over a route
// (batch-union: colibri-strix README, "What's implemented"), on the 16x16x64 int8 matrix instruction.
//
// A workgroup (4 wavefronts) owns 16 weight rows (of each matrix) and chunks of 16 NT rows of
// activations. The wavefronts take the K groups (256 contiguous bytes of a row) in turn, two groups
// of weights under way at a time straight into the operand registers; their integer sums meet in LDS.
// One row of activations (x in ACT_X) is quantised by every workgroup itself while its first weights
// are under way, which saves a launch.
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
  const float s = i8_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3]))), inv = __builtin_amdgcn_rcpf(s);
#pragma unroll
  for (int i = 0; i < XP; i++) {
    const int u = tid + 256 * i;
    if (u < n) *reinterpret_cast<uint2 *>(lc + u * 8) = i8_codes8(v[i], s, inv);
  }
  for (int u = tid + 256 * XP; u < n; u += 256) {
    float t[8];
    load8(x + u * 8, t);
    *reinterpret_cast<uint2 *>(lc + u * 8) = i8_codes8(t, s, inv);
  }
  for (int u = n + tid; u < np; u += 256) *reinterpret_cast<uint2 *>(lc + u * 8) = make_uint2(0, 0);
  return s;
}

enum I8Act { I8_ACT_WS, I8_ACT_X };  // activations: quantised in the workspace; one row of x

template <I8Mode MODE, typename T, int NT, I8Act ACT>
__global__ __launch_bounds__(256, 2) void i8_gemv_kernel(I8Args a) {
  constexpr int NMAT = MODE == I8_GATEUP ? 2 : 1;
  constexpr int D = NT == 4 ? 1 : 2;  // groups under way
  static_assert(ACT == I8_ACT_WS || (NT == 1 && MODE != I8_DOWN));
  extern __shared__ __align__(16) int8_t lds[];  // ACT_X: the quantised row
  __shared__ int red[4][NMAT][NT][16][17];
  __shared__ uint32_t tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16;
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
      const int na = max(0, min(*a.nact, a.E));
      if (u >= na) return;
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
    wq[m] = a.wq + (int64_t)e * a.wq_stride + ((int64_t)m * a.N + min(n0 + li, a.N - 1)) * K;
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
      for (int q = 0; q < NT; q++) i8_load_group(aq[q], pitch / 16, wv + 4 * i, lq, act[d][q]);
    };
    auto load = [&](int d, int i) {
#pragma unroll
      for (int m = 0; m < NMAT; m++) i8_load_group(wq[m], nc, wv + 4 * i, lq, w[d][m]);
      if constexpr (ACT == I8_ACT_WS) load_act(d, i);
    };
#pragma unroll
    for (int d = 0; d < D; d++)
      if (d < ngw) load(d, d);
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
      if (row < n && n0 + tc < a.N) {
        const int ci = first + row;
        int64_t orow = ci, arow = ci;
        if constexpr (MODE != I8_LINEAR) {
          orow = routed ? (int64_t)a.perm[ci] : P + ci;
          arow = MODE == I8_DOWN ? orow : (routed ? orow / a.k : ci);
        }
        const float s = ACT == I8_ACT_X ? xs : a.as[arow];
        auto value = [&](int m) {
          const int sum = red[0][m][q][tr][tc] + red[1][m][q][tr][tc] + red[2][m][q][tr][tc] + red[3][m][q][tr][tc];
          return i8_value(sum, s, ws[(int64_t)m * a.N]);
        };
        const int64_t o = orow * a.N + n0 + tc;
        if constexpr (MODE == I8_GATEUP)
          static_cast<T *>(a.out)[o] = (T)i8_product(i8_silu(value(0)), value(NMAT - 1));
        else if constexpr (MODE == I8_DOWN)
          static_cast<float *>(a.out)[o] = value(0);
        else
          static_cast<T *>(a.out)[o] = (T)(value(0) + (a.bias ? a.bias[n0 + tc] : 0.0f));
      }
    }
    if (c + 16 * NT < n) __syncthreads();
  }
}

// One row quantised by every workgroup
bool i8_gemv_from_x(const I8Args &a) { return a.M == 1 && i8_padded(a.K) <= 48 * 1024; }

template <I8Mode MODE, typename T>
static hipError_t launch_gemv_t(const I8Args &a, hipStream_t s) {
  const int64_t P = (int64_t)a.M * a.k;
  auto go = [&]<int NT, I8Act ACT>(int64_t ny) {
    hipLaunchKernelGGL((i8_gemv_kernel<MODE, T, NT, ACT>), dim3((unsigned)((a.N + 15) / 16), (unsigned)ny), dim3(256),
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
