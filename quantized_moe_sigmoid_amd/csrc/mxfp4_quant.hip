// mxfp4_quant.hip — MXFP4 quantisation of rows of fp32, bf16 or fp16 values, and back.
//
// JustVugg/colibri README, "Other supported models" (MXFP4 experts); encodings and rounding
// of OCP MX v1.0, in mx_quant_half (mxfp4_impl.h).
//
// Bound by memory: a value is read once and 17/32 byte of it written (and the reverse). Two
// lanes own a block, so every load is 16 bytes wide and every store of codes 8 bytes. 49152 x 2048
// bf16 on buffers that no cache holds: 44 us to codes (254 MB, 5.8 TB/s), 46 us back (5.5 TB/s); a
// plain read reaches 6.4 TB/s, a fill 6.9, a copy 5.2. The same buffers again and again, partly
// from the last-level cache: 35 and 38 us. Two or four blocks to a thread: 2 to 5 us slower.
#include "mxfp4_impl.h"

namespace coli {

template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T *__restrict__ x, int64_t nblk,
                                                          uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t blk = gid >> 1;
  const int q = threadIdx.x & 1;
  if (blk >= nblk) return;  // both lanes of a block or neither
  float a[8], b[8];
  load8(x + blk * 32 + 8 * q, a);
  load8(x + blk * 32 + 16 + 8 * q, b);
  uint32_t u;
  const uint2 w = mx_quant_half(a, b, u);
  *reinterpret_cast<uint2 *>(codes + blk * 16 + 8 * q) = w;
  if (q == 0) scales[blk] = (uint8_t)u;
}

template <typename T>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, int64_t nblk,
                                                            T *__restrict__ out) {
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t blk = gid >> 1;
  const int q = threadIdx.x & 1;
  if (blk >= nblk) return;
  const uint2 w = *reinterpret_cast<const uint2 *>(codes + blk * 16 + 8 * q);
  const float s = e8m0_f32(scales[blk]);  // fp32 products: exact, 2^-127 and NaN included
  typedef T v8 __attribute__((ext_vector_type(8)));
  v8 lo, hi;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t c = i ? w.y : w.x;
    auto put = [&](int j, auto p) {
      lo[4 * i + j] = (T)(p[0] * s);
      hi[4 * i + j] = (T)(p[1] * s);
    };
    put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0));
    put(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1));
    put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2));
    put(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3));
  }
  *reinterpret_cast<v8 *>(out + blk * 32 + 8 * q) = lo;
  *reinterpret_cast<v8 *>(out + blk * 32 + 16 + 8 * q) = hi;
}

// The activations of a product: rows of nb blocks, padded to nbp (zero codes, scale 1); fewer than
// 2^31 blocks. Whole rows (nb == nbp) need no place in their row.
template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_rows_kernel(const T *__restrict__ x, uint32_t blocks, uint32_t nb,
                                                               uint32_t nbp, uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scales) {
  const uint32_t blk = blockIdx.x * 128 + (threadIdx.x >> 1);
  const int q = threadIdx.x & 1;
  if (blk >= blocks) return;  // both lanes of a block or neither
  int64_t from = blk;
  bool there = true;
  if (nb != nbp) {
    const uint32_t row = blk / nbp, b0 = blk - row * nbp;
    there = b0 < nb;
    from = (int64_t)row * nb + b0;
  }
  uint2 w = make_uint2(0, 0);
  uint32_t u = 127;
  if (there) {
    float a[8], b[8];
    const T *px = x + from * 32;
    load8(px + 8 * q, a);
    load8(px + 16 + 8 * q, b);
    w = mx_quant_half(a, b, u);
  }
  *reinterpret_cast<uint2 *>(codes + (int64_t)blk * 16 + 8 * q) = w;
  if (q == 0) scales[blk] = (uint8_t)u;
}

__global__ __launch_bounds__(256) void mx_pad_scales_kernel(const uint8_t *__restrict__ scales, int rows, int nb,
                                                            int nbp, uint8_t *__restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // four bytes each
  const int64_t row = i / (nbp / 4);
  const int b0 = (int)(i - row * (nbp / 4)) * 4;
  if (row >= rows) return;
  uint32_t v = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) v |= (b0 + j < nb ? (uint32_t)scales[row * nb + b0 + j] : 127u) << (8 * j);
  reinterpret_cast<uint32_t *>(out)[i] = v;
}

static unsigned grid_of(int64_t nblk) { return (unsigned)((nblk * 2 + 255) / 256); }

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t nblk, uint8_t *codes, uint8_t *scales, hipStream_t s) {
  const dim3 g(grid_of(nblk)), b(256);
  if (dtype == COLI_F32)
    hipLaunchKernelGGL(mx_quantize_kernel<float>, g, b, 0, s, (const float *)x, nblk, codes, scales);
  else if (dtype == COLI_BF16)
    hipLaunchKernelGGL(mx_quantize_kernel<bf16_t>, g, b, 0, s, (const bf16_t *)x, nblk, codes, scales);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<f16_t>, g, b, 0, s, (const f16_t *)x, nblk, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t nblk, void *out, int dtype,
                                hipStream_t s) {
  const dim3 g(grid_of(nblk)), b(256);
  if (dtype == COLI_F32)
    hipLaunchKernelGGL(mx_dequantize_kernel<float>, g, b, 0, s, codes, scales, nblk, (float *)out);
  else if (dtype == COLI_BF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<bf16_t>, g, b, 0, s, codes, scales, nblk, (bf16_t *)out);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<f16_t>, g, b, 0, s, codes, scales, nblk, (f16_t *)out);
  return hipGetLastError();
}

hipError_t launch_mx_quantize_rows(const void *x, int dtype, int64_t rows, int K, uint8_t *codes, uint8_t *scales,
                                   hipStream_t s) {
  const uint32_t nb = K / 32, nbp = mx_padded(K) / 32, n = (uint32_t)(rows * nbp);
  const dim3 g(grid_of(rows * nbp)), b(256);
  if (dtype == COLI_F32)
    hipLaunchKernelGGL(mx_quantize_rows_kernel<float>, g, b, 0, s, (const float *)x, n, nb, nbp, codes, scales);
  else if (dtype == COLI_BF16)
    hipLaunchKernelGGL(mx_quantize_rows_kernel<bf16_t>, g, b, 0, s, (const bf16_t *)x, n, nb, nbp, codes, scales);
  else
    hipLaunchKernelGGL(mx_quantize_rows_kernel<f16_t>, g, b, 0, s, (const f16_t *)x, n, nb, nbp, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_pad_scales(const uint8_t *scales, int rows, int K, uint8_t *out, hipStream_t s) {
  const int nb = K / 32, nbp = mx_padded(K) / 32;
  const int64_t n = (int64_t)rows * (nbp / 4);
  hipLaunchKernelGGL(mx_pad_scales_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, scales, rows, nb, nbp, out);
  return hipGetLastError();
}

}  // namespace coli
