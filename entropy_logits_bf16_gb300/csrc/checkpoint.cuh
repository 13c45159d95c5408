// The arithmetic of the 8-bit activation checkpoints (rlk_checkpoint): blocks
// of 32 columns with a power-of-two step, so everything but the rounding of
// x / step to a whole number is exact.
#pragma once

#include "common.cuh"

namespace rlk {

constexpr int kCkBlock = 32;

// Scale byte of a block from the bits of its largest |x|: k + 127 with k the
// least whole number >= -126 and 127 2^k >= |x|; 255 when that is no number.
// |x| = 1.m 2^e and 127 = 1.984375 2^6, so k = e - 6, one more when the
// mantissa is above 1.984375 (fraction 0x7E0000).
__device__ __forceinline__ uint32_t ck_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int b = (int)(amax_bits >> 23) - 6 + ((amax_bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return b < 1 ? 1u : (uint32_t)b;
}
// 2^k and (byte < 255) 2^-k of a scale byte.  255: the step reads as +inf, and with code 0
// the value is 0 inf = NaN.
__device__ __forceinline__ float ck_step(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float ck_inv_step(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// x / step rounded to nearest even: in [-127, 127]; 0 where the block has no
// step (255); in [-63, 63] at the largest step, 2^122, where 64 steps would be
// 2^128 and overflow.
constexpr uint32_t kCkTop = 249u;
__device__ __forceinline__ int ck_code(float x, uint32_t byte) {
  if (byte == 255u) return 0;
  const int q = __float2int_rn(__fmul_rn(x, ck_inv_step(byte)));
  return byte == kCkTop ? max(-63, min(63, q)) : q;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

}  // namespace rlk
