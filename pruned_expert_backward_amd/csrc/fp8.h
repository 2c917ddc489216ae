// Blocks of 128 values in 8 bits: e4m3 (1 sign, 4 exponent, 3 mantissa bits; up to
// 448, steps of 2^-9 below 2^-6, no infinity) with one power-of-two scale, held as
// the exponent byte e + 127 that the scaled matrix instructions read.  The scale is
// the smallest power of two that keeps the block within +-448.  A power of two
// costs e4m3 no accuracy (only the lowest of its 18 binades), makes scaling exact in
// both directions, and leaves the product's scaling to the matrix unit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "row_norm.h"

namespace lrmoe {

constexpr int kFp8Block = 128;

// Bytes of a row of scales: a block each, in whole dwords.
__host__ __device__ inline int fp8_scale_row(int d) {
  return ((d + kFp8Block - 1) / kFp8Block + 3) / 4 * 4;
}

// Bits of |x|, 0 for infinity and NaN: they become NaN codes and leave the block's
// scale to the others.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest of the 16 lanes of a row of lanes.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = umax(v, dpp<0xB1>(v));
  v = umax(v, dpp<0x4E>(v));
  v = umax(v, dpp<0x141>(v));
  return umax(v, dpp<0x140>(v));
}

// Scale byte of a block from the bits of its largest magnitude: 448 = 1.75 * 2^8,
// so the exponent less 8, and one more above 1.75.  A block of zeros has scale 1.
// Between 1 (so that 1 / scale is finite) and 247.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t top) {
  const int b = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return top == 0 ? 127u : (uint32_t)(b < 1 ? 1 : b);
}
__device__ __forceinline__ float fp8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float fp8_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Four values within +-448 (or NaN) to four codes, nearest, ties to even.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ __forceinline__ void fp8_unpack4(uint32_t w, float (&v)[4]) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}

// x / scale, NaN for infinity and NaN.
__device__ __forceinline__ float fp8_scaled(float x, float inverse) {
  return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                                           : x * inverse;
}

}  // namespace lrmoe
