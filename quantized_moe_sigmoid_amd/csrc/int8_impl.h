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

// What a row is rounded with: its scale s and about 1 / s (within 2^-23 of it), NaN where s is 0, below
// fp32's normal numbers or NaN.
struct I8Row {
  float s, inv;
};
__device__ __forceinline__ I8Row i8_row(uint32_t top) {
  const float s = i8_scale(top);
  return I8Row{s, s >= 0x1p-126f ? __builtin_amdgcn_rcpf(s) : __uint_as_float(0x7FC00000u)};
}

// The definition: one division, rounded half away from zero
__device__ __forceinline__ uint32_t i8_code(float v, float s) {
  return s > 0.0f ? (uint32_t)(int)fminf(fmaxf(roundf(v / s), -127.0f), 127.0f) : 0u;
}

// Codes of eight values. |v / s| <= 127.001 and v inv is within 2^-15 of the quotient: where it is not
// that near a half, its nearest integer is the code, and the sum with 3 * 2^22 holds it in its low byte.
// Otherwise (one value in 5000) and for scales without an inverse the division decides, for all eight.
__device__ __forceinline__ uint2 i8_codes8(const float (&v)[8], const I8Row &row) {
  constexpr float M = 0x1.8p+23f;
  uint32_t w[8];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float t = __builtin_fmaf(v[i], row.inv, M);
    far = fmaxf(far, fabsf(__builtin_fmaf(v[i], row.inv, M - t)));
    w[i] = __float_as_uint(t);
  }
  if (__builtin_expect(!(far <= 0.4999f && row.inv == row.inv), 0)) {
#pragma unroll
    for (int i = 0; i < 8; i++) w[i] = i8_code(v[i], row.s);
  }
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; i++) h[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x0c0c0400u);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
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

// y of an exact sum, and with a bias (likewise a value of its own)
__device__ __forceinline__ float i8_value(int acc, float row, float channel) { return i8_product((float)acc, row * channel); }
__device__ __forceinline__ float i8_biased(int acc, float row, float channel, float bias) {
  float y = i8_value(acc, row, channel) + bias;
  asm volatile("" : "+v"(y));
  return y;
}

// silu(g) = g / (1 + e^-g) from t = e^-|g|, which does not overflow: g / (1 + t), or g t / (1 + t) below
// 0, so that gates down to -103, where g t leaves fp32, count. t = 2^h (1 + l ln 2) with h + l =
// -|g| log2(e) to about 2^-46, by the hardware's exponential and reciprocal (within 1 ulp each); t of
// h below -64 is held times 2^64 (h + 64 is exact, h being a value of its own: fused into x log2(e) + 64 it would
// lose the rounding that l makes good, up to 46 half steps of t for 2). One function for all kernels: the same
// bits in each.
__device__ __forceinline__ float i8_silu(float g) {
  const float x = fmaxf(-fabsf(g), -200.0f);
  const float h = i8_product(x, 0x1.715476p+0f);
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
