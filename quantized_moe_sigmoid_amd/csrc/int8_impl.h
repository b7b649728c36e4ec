// int8_impl.h — device code shared by the int8 products with token and channel scales (int8_*.hip).
//
// Rule of a row x (the Q8_0 rule of colibri-strix README, "What's implemented", integer-dot kernels
// item, with one scale for the whole row): s = max|x| / 127, q = round-half-away(x / s), both fp32
// divisions correctly rounded; s = 0 gives q = 0, an infinity or a NaN s = NaN and codes 0.
#pragma once

#include "mxfp4_impl.h"

namespace coli {

// The scale of a row whose largest magnitude has these bits
__device__ __forceinline__ float i8_scale(uint32_t top) {
  return top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 127.0f;
}

// Code of v; inv is about 1 / s (within 2^-22). |v / s| <= 127, so v inv is within 2^-15 of the
// quotient: away from a half its nearest integer is the quotient's, near one the division decides.
// Scales of 0, below 2^-126 or NaN: inv is infinite or NaN, and so is what follows.
__device__ __forceinline__ int i8_code(float v, float s, float inv) {
  const float r = v * inv;
  float q = __builtin_rintf(r);
  if (__builtin_expect(!(fabsf(r - q) <= 0.4999f), 0)) {
    q = roundf(v / s);
    q = s > 0.0f ? fminf(fmaxf(q, -127.0f), 127.0f) : 0.0f;
  }
  return (int)q;
}

__device__ __forceinline__ uint2 i8_codes8(const float (&v)[8], float s, float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i++) w[i >> 2] |= (uint32_t)(i8_code(v[i], s, inv) & 0xFF) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t i8_top8(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; i++) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return top;
}

__device__ __forceinline__ uint32_t wave_top(uint32_t top) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  return top;
}

// A product that stays a value of its own: fused with what follows (a bias, the rounding to fp16) it
// would be rounded otherwise in one kernel than in another.
__device__ __forceinline__ float i8_product(float a, float b) {
  float y = a * b;
  asm volatile("" : "+v"(y));
  return y;
}

// y of an exact sum
__device__ __forceinline__ float i8_value(int acc, float row, float channel) { return i8_product((float)acc, row * channel); }

// silu(g) = g / (1 + e^-g) from t = e^-|g|, which does not overflow: g / (1 + t), or g t / (1 + t) below
// 0, so that gates down to -103, where g t leaves fp32, count. t = 2^h (1 + l ln 2) with h + l =
// -|g| log2(e) to about 2^-46, by the hardware's exponential and reciprocal (within 1 ulp each); t of
// h below -64 is held times 2^64 (h + 64 is exact). One function for all kernels: the same bits in each.
__device__ __forceinline__ float i8_silu(float g) {
  const float x = fmaxf(-fabsf(g), -200.0f);
  const float h = x * 0x1.715476p+0f;
  const float l = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -h));
  const bool low = h < -64.0f;
  const float unit = low ? 0x1p-64f : 1.0f;
  const float e = __builtin_amdgcn_exp2f(low ? h + 64.0f : h);
  const float t = __builtin_fmaf(e * l, 0x1.62e430p-1f, e);
  const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(t, unit, 1.0f));
  return g >= 0.0f ? g * r : g * t * r * unit;
}

// D = A B + C: lane l holds row (A) or column (B) l % 16, inputs 16 (l / 16) .. + 15 of a K step of 64;
// lane l's four results are rows 4 (l / 16) .. + 3 of column l % 16. The order of the inputs is the
// same in both operands, so it does not enter.
__device__ __forceinline__ v4i32 i8_mfma16(uint4 a, uint4 b, v4i32 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i32, a), __builtin_bit_cast(v4i32, b), c, 0, 0, 0);
}

}  // namespace coli
