// mxfp4_product.hip — products whose both operands are MXFP4 on the scaled matrix
// instructions of gfx950: y = x W^T, and over a route the experts' gate/up rows with SiLU*up
// and their down rows (batch-union: colibri-strix README, "What's implemented").
//
// A workgroup (4 wavefronts) owns 16 weight rows (of each matrix) and chunks of 16 rows of
// activations; the wavefronts split K and their sums meet in LDS, added in wavefront order.
#include "mxfp4_impl.h"

namespace coli {

template <MxMode MODE, typename T>
__global__ __launch_bounds__(256) void mx_product_kernel(MxArgs a) {
  constexpr int NMAT = MODE == MX_GATEUP ? 2 : 1;
  __shared__ float red[4][NMAT][16][17];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int nb = a.K / 32, nbp = mx_padded(a.K) / 32;
  // the rows of activations of this workgroup: first .. first + n - 1 of perm (routed), or
  // of the tokens (shared expert, linear)
  int e = 0, first = 0, n = a.M;
  bool routed = false;
  if (MODE == MX_LINEAR) {
    first = blockIdx.y * 16;
    n = min(16, a.M - first);
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
  const uint8_t *wc = a.wc + (int64_t)e * a.wc_stride, *ws = a.ws + (int64_t)e * a.ws_stride;
  const int wrow = min(n0 + li, a.N - 1);
  for (int c = 0; c < n; c += 16) {
    const int ci = first + min(c + li, n - 1);
    const int64_t P = (int64_t)a.M * a.k;
    int64_t arow = ci;
    if (MODE != MX_LINEAR) {
      const int64_t pair = routed ? a.perm[ci] : P + ci;
      arow = MODE == MX_DOWN ? pair : (routed ? pair / a.k : ci);
    }
    v4f acc[NMAT] = {};
    for (int s = wv; s * 4 < nb; s += 4) {
      const int b = s * 4 + lq;
      const uint4 av = *reinterpret_cast<const uint4 *>(a.ac + (arow * nbp + b) * 16);
      const uint32_t ua = a.as[arow * nbp + b];
#pragma unroll
      for (int m = 0; m < NMAT; m++) {
        const int64_t blk = ((int64_t)m * a.N + wrow) * nb + b;
        uint4 wv4 = make_uint4(0, 0, 0, 0);
        uint32_t uw = 127;
        if (b < nb) {
          wv4 = *reinterpret_cast<const uint4 *>(wc + blk * 16);
          uw = ws[blk];
        }
        acc[m] = mx_mfma16(av, ua, wv4, uw, acc[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < NMAT; m++)
#pragma unroll
      for (int r = 0; r < 4; r++) red[wv][m][4 * lq + r][li] = acc[m][r];
    __syncthreads();
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    float v[NMAT];
#pragma unroll
    for (int m = 0; m < NMAT; m++) v[m] = ((red[0][m][tr][tc] + red[1][m][tr][tc]) + red[2][m][tr][tc]) + red[3][m][tr][tc];
    if (c + tr < n && n0 + tc < a.N) {
      const int ci2 = first + c + tr;
      const int64_t orow = MODE == MX_LINEAR ? ci2 : (routed ? (int64_t)a.perm[ci2] : P + ci2);
      const int64_t o = orow * a.N + n0 + tc;
      if constexpr (MODE == MX_GATEUP)
        static_cast<T *>(a.out)[o] = (T)(silu(v[0]) * v[1]);
      else if constexpr (MODE == MX_DOWN)
        static_cast<float *>(a.out)[o] = v[0];
      else
        static_cast<T *>(a.out)[o] = (T)v[0];
    }
    __syncthreads();
  }
}

// out_t = sum_j w_tj y_tj in slot order, plus the shared expert's row; empty slots skipped
template <typename T>
__global__ __launch_bounds__(256) void mx_combine_kernel(const float *__restrict__ y, const int32_t *__restrict__ idx,
                                                         const float *__restrict__ w, int T_, int k, int E, int H,
                                                         int has_shared, T *__restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int64_t t = i / H;
  const int h = (int)(i - t * H);
  if (t >= T_) return;
  v4f s = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; j++) {
    const int64_t p = t * k + j;
    const int e = idx[p];
    if (e < 0 || e >= E) continue;
    s += w[p] * *reinterpret_cast<const v4f *>(y + p * H + h);
  }
  if (has_shared) s += *reinterpret_cast<const v4f *>(y + ((int64_t)T_ * k + t) * H + h);
  typedef T v4 __attribute__((ext_vector_type(4)));
  v4 o;
#pragma unroll
  for (int r = 0; r < 4; r++) o[r] = (T)s[r];
  *reinterpret_cast<v4 *>(out + i) = o;
}

template <MxMode MODE, typename T>
static hipError_t launch_t(const MxArgs &a, hipStream_t s) {
  const int64_t P = (int64_t)a.M * a.k;
  const int64_t ny = MODE == MX_LINEAR ? (a.M + 15) / 16 : a.has_shared + (P < a.E ? P : a.E);
  hipLaunchKernelGGL((mx_product_kernel<MODE, T>), dim3((unsigned)((a.N + 15) / 16), (unsigned)ny), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_mx_product(MxMode mode, int dtype, const MxArgs &a, hipStream_t s) {
  if (mode == MX_DOWN) return launch_t<MX_DOWN, float>(a, s);
  if (mode == MX_LINEAR)
    return dtype == COLI_F32 ? launch_t<MX_LINEAR, float>(a, s)
         : dtype == COLI_BF16 ? launch_t<MX_LINEAR, bf16_t>(a, s) : launch_t<MX_LINEAR, f16_t>(a, s);
  return dtype == COLI_F32 ? launch_t<MX_GATEUP, float>(a, s)
       : dtype == COLI_BF16 ? launch_t<MX_GATEUP, bf16_t>(a, s) : launch_t<MX_GATEUP, f16_t>(a, s);
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
