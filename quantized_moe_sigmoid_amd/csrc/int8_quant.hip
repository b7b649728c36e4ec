// int8_quant.hip — rows of fp32, bf16 or fp16 values to int8 with a scale for each row (int8_impl.h).
//
// Bound by memory: a value is read once and a byte of it written. Rows up to 8192 values stay in
// registers between the search for their largest magnitude and the rounding; longer rows are read twice.
#include "int8_impl.h"

namespace coli {

// WPR wavefronts to a row, REGS pieces of 8 values of it in a lane's registers (0: read twice)
template <typename T, int WPR, int REGS>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const T *__restrict__ x, int64_t rows, int K, int pitch,
                                                          int8_t *__restrict__ codes, float *__restrict__ scales) {
  constexpr int L = 64 * WPR, RPB = 4 / WPR;  // lanes to a row, rows to a workgroup
  __shared__ uint32_t tops[4];
  const int wv = threadIdx.x >> 6, l = threadIdx.x % L;
  const int n = K / 8, np = pitch / 8;
  for (int64_t row = (int64_t)blockIdx.x * RPB + wv / WPR; row < rows; row += (int64_t)gridDim.x * RPB) {
    const T *px = x + row * K;
    int8_t *pc = codes + row * pitch;
    float v[REGS ? REGS : 1][8];
    uint32_t top = 0;
    if constexpr (REGS > 0) {
#pragma unroll
      for (int i = 0; i < REGS; i++) {
        const int u = l + L * i;
        if (u < n) {
          load8(px + u * 8, v[i]);
          top = i8_top8(v[i], top);
        }
      }
    } else {
      for (int u = l; u < n; u += L) {
        load8(px + u * 8, v[0]);
        top = i8_top8(v[0], top);
      }
    }
    top = wave_top(top);
    if constexpr (WPR > 1) {
      __syncthreads();  // the last row's have been read
      if ((threadIdx.x & 63) == 0) tops[wv] = top;
      __syncthreads();
      top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    }
    const I8Row r = i8_row(top);
    if (l == 0) scales[row] = r.s;
    if constexpr (REGS > 0) {
#pragma unroll
      for (int i = 0; i < REGS; i++) {
        const int u = l + L * i;
        if (u < n) *reinterpret_cast<uint2 *>(pc + u * 8) = i8_codes8(v[i], r);
      }
    } else {
      for (int u = l; u < n; u += L) {
        load8(px + u * 8, v[0]);
        *reinterpret_cast<uint2 *>(pc + u * 8) = i8_codes8(v[0], r);
      }
    }
    for (int u = n + l; u < np; u += L) *reinterpret_cast<uint2 *>(pc + u * 8) = make_uint2(0, 0);
  }
}

template <typename T>
static hipError_t launch_q(const T *x, int64_t rows, int K, int pitch, int8_t *codes, float *scales, hipStream_t s) {
  auto go = [&]<int WPR, int REGS>() {
    const int64_t groups = (rows + 4 / WPR - 1) / (4 / WPR);
    hipLaunchKernelGGL((i8_quantize_kernel<T, WPR, REGS>), dim3((unsigned)(groups < (1 << 23) ? groups : 1 << 23)), dim3(256),
                       0, s, x, rows, K, pitch, codes, scales);
    return hipGetLastError();
  };
  if (K <= 512) return go.template operator()<1, 1>();
  if (K <= 1024) return go.template operator()<1, 2>();
  if (K <= 2048) return go.template operator()<4, 1>();
  if (K <= 4096) return go.template operator()<4, 2>();
  if (K <= 8192) return go.template operator()<4, 4>();
  return go.template operator()<4, 0>();
}

hipError_t launch_i8_quantize(const void *x, int dtype, int64_t rows, int K, int pitch, int8_t *codes, float *scales,
                              hipStream_t s) {
  if (dtype == COLI_F32) return launch_q((const float *)x, rows, K, pitch, codes, scales, s);
  if (dtype == COLI_BF16) return launch_q((const bf16_t *)x, rows, K, pitch, codes, scales, s);
  return launch_q((const f16_t *)x, rows, K, pitch, codes, scales, s);
}

}  // namespace coli
