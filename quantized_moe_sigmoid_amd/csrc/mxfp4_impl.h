// mxfp4_impl.h — device code shared by the MXFP4 x MXFP4 operators (mxfp4_*.hip).
//
// MXFP4 (OCP MX v1.0): 32 consecutive values of a row share one E8M0 byte u = 2^(u - 127);
// the values are E2M1 codes, byte j of the 16-byte block = code j | code (j + 16) << 4.
// Expert format named on the JustVugg/colibri README, "Other supported models".
#pragma once

#include "coli_internal.h"
#include "per_device.h"

namespace coli {

// The current device lets `kernel` have `bytes` of LDS (64 KB without asking)
template <typename Kernel>
inline hipError_t allow_lds(PerDevice &done, Kernel kernel, size_t bytes) {
  int device = -1;
  const hipError_t st = hipGetDevice(&device);
  if (st != hipSuccess) return st;
  return done.once(device, [&]() {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
}

typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v4i32 __attribute__((ext_vector_type(4)));
typedef int v8i32 __attribute__((ext_vector_type(8)));

// eight consecutive values as fp32 (p 16-byte aligned)
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16_t *p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const f16_t *p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const f16x2 h = as_f16x2(w[i]);
    v[2 * i] = (float)h.x;
    v[2 * i + 1] = (float)h.y;
  }
}

// Half a block: lanes l and l ^ 1 share one; half q holds a = values 8q .. 8q + 7 and b =
// values 16 + 8q .. 16 + 8q + 7, so its eight bytes hold their codes. u = the block's E8M0
// byte: the exponent of the largest magnitude less 2 (E2M1's largest is 6 = 1.5 * 2^2), 0
// for a block of zeros, 255 (NaN) when it holds an infinity or a NaN, whose codes are 0. The
// product with 2^(127 - u) is exact (or far below the smallest code), so the values are
// rounded once, to nearest even and saturating at 6, by the hardware's fp4 convert.
__device__ __forceinline__ uint2 mx_quant_half(const float (&a)[8], const float (&b)[8], uint32_t &u) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; i++)
    top = max(top, max(__float_as_uint(a[i]) & 0x7FFFFFFFu, __float_as_uint(b[i]) & 0x7FFFFFFFu));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));  // lane ^ 1
  const int e = (int)(top >> 23);
  u = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
  const float up = __uint_as_float(e == 255 ? 0u : (254u - u) << 23);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; i++) {
    w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], a[4 * i] * up, b[4 * i] * up, 1.0f, 0);
    w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], a[4 * i + 1] * up, b[4 * i + 1] * up, 1.0f, 1);
    w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], a[4 * i + 2] * up, b[4 * i + 2] * up, 1.0f, 2);
    w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], a[4 * i + 3] * up, b[4 * i + 3] * up, 1.0f, 3);
  }
  return e == 255 ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
}

// D = A B + C on the scaled matrix instruction with both operands in E2M1 (cbsz = blgp = 4):
// lane l holds row (A) or column (B) l % 16, block l / 16 of the four blocks of a K step of
// 128; byte 0 of its scale register is that block's E8M0 code. Lane l's four results are rows
// 4 (l / 16) .. + 3 of column l % 16. The order of the 32 codes inside a block is the same in
// both operands, so it does not enter.
__device__ __forceinline__ v4f mx_mfma16(uint4 a, uint32_t ua, uint4 b, uint32_t ub, v4f c) {
  const v8i32 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i32 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)ua, 0, (int)ub);
}

// silu in fp32 for the many values of a tile: e^-g = 2^h (1 + l ln 2) with h + l = -g log2(e)
// to about 2^-46, by the hardware's exponential and reciprocal (within 1 ulp each). The clamp
// keeps h + l finite: below it 1 + e^-g is 1, above it infinite. The reciprocal of 1 + e^-g past
// 2^126 would count as 0 while e^-g is still finite (g from -88.7 to -87.3), so 2^-8 of it is taken.
__device__ __forceinline__ float silu_fast(float g) {
  const float x = __builtin_amdgcn_fmed3f(-g, -126.0f, 200.0f);
  const float h = x * 0x1.715476p+0f;
  const float l = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -h));
  const float e = __builtin_amdgcn_exp2f(h) * __builtin_fmaf(l, 0x1.62e430p-1f, 1.0f);
  return g * 0x1p-8f * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0x1p-8f, 0x1p-8f));
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

}  // namespace coli
