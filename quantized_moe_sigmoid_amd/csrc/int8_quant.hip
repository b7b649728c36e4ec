// int8_quant.hip — rows of fp32, bf16 or fp16 values to int8 with a scale for each row (int8_impl.h).
//
// Bound by memory: a value is read once and a byte of it written. Rows up to 8192 values stay in
// registers between the search for their largest magnitude and the rounding; longer rows are read twice.
// 18432 x 2048 fp32 31 us (6.0 TB/s), 14745 x 2048 bf16 20 (4.6), 4093 x 6144 bf16 19 (4.0). Pieces of 8
// values a lane: 23, 32 and 19.5; a wavefront to a row of 6144: 25.
#include "int8_impl.h"

namespace coli {

// L lanes to a row, REGS pieces of 16 values of it in a lane's registers (0: read twice)
template <typename T, int L, int REGS>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const T *__restrict__ x, int64_t rows, int K, int pitch,
                                                          int8_t *__restrict__ codes, float *__restrict__ scales) {
  constexpr int RPB = 256 / L;  // rows to a workgroup
  __shared__ uint32_t tops[4];
  const int l = threadIdx.x % L, r0 = threadIdx.x / L;
  const int n = K / 16, np = pitch / 16;
  for (int64_t first = (int64_t)blockIdx.x * RPB; first < rows; first += (int64_t)gridDim.x * RPB) {
    const bool there = first + r0 < rows;
    const int64_t row = there ? first + r0 : rows - 1;  // lanes past the end read the last row and write nothing
    const T *px = x + row * K;
    int8_t *pc = codes + row * pitch;
    float v[REGS ? REGS : 1][2][8];
    uint32_t top = 0;
    if constexpr (REGS > 0) {
#pragma unroll
      for (int i = 0; i < REGS; i++) {
        const int u = l + L * i;
        if (u < n) {
          load8(px + u * 16, v[i][0]);
          load8(px + u * 16 + 8, v[i][1]);
          top = i8_top8(v[i][1], i8_top8(v[i][0], top));
        }
      }
    } else {
      for (int u = l; u < n; u += L) {
        load8(px + u * 16, v[0][0]);
        load8(px + u * 16 + 8, v[0][1]);
        top = i8_top8(v[0][1], i8_top8(v[0][0], top));
      }
    }
#pragma unroll
    for (int o = (L < 64 ? L : 64) / 2; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if constexpr (L > 64) {
      __syncthreads();  // the last row's have been read
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < L / 64; i++) top = max(top, tops[r0 * (L / 64) + i]);
    }
    const I8Row r = i8_row(top);
    if (!there) continue;
    if (l == 0) scales[row] = r.s;
    auto put = [&](int u, const float (&x)[2][8]) {
      const uint2 a = i8_codes8(x[0], r), b = i8_codes8(x[1], r);
      *reinterpret_cast<uint4 *>(pc + u * 16) = make_uint4(a.x, a.y, b.x, b.y);
    };
    if constexpr (REGS > 0) {
#pragma unroll
      for (int i = 0; i < REGS; i++) {
        const int u = l + L * i;
        if (u < n) put(u, v[i]);
      }
    } else {
      for (int u = l; u < n; u += L) {
        load8(px + u * 16, v[0][0]);
        load8(px + u * 16 + 8, v[0][1]);
        put(u, v[0]);
      }
    }
    for (int u = n + l; u < np; u += L) *reinterpret_cast<uint4 *>(pc + u * 16) = make_uint4(0, 0, 0, 0);
  }
}

template <typename T>
static hipError_t launch_q(const T *x, int64_t rows, int K, int pitch, int8_t *codes, float *scales, hipStream_t s) {
  auto go = [&]<int L, int REGS>() {
    const int64_t groups = (rows + 256 / L - 1) / (256 / L);
    hipLaunchKernelGGL((i8_quantize_kernel<T, L, REGS>), dim3((unsigned)(groups < (1 << 23) ? groups : 1 << 23)), dim3(256),
                       0, s, x, rows, K, pitch, codes, scales);
    return hipGetLastError();
  };
  if (K <= 512) return go.template operator()<32, 1>();
  if (K <= 1024) return go.template operator()<64, 1>();
  if (K <= 2048) return go.template operator()<128, 1>();
  if (K <= 4096) return go.template operator()<256, 1>();
  if (K <= 8192) return go.template operator()<256, 2>();
  return go.template operator()<256, 0>();
}

hipError_t launch_i8_quantize(const void *x, int dtype, int64_t rows, int K, int pitch, int8_t *codes, float *scales,
                              hipStream_t s) {
  if (dtype == COLI_F32) return launch_q((const float *)x, rows, K, pitch, codes, scales, s);
  if (dtype == COLI_BF16) return launch_q((const bf16_t *)x, rows, K, pitch, codes, scales, s);
  return launch_q((const f16_t *)x, rows, K, pitch, codes, scales, s);
}

}  // namespace coli
