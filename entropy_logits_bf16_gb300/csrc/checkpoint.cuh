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
// Four codes as the bytes of a word, of finite numbers in blocks with a step
// below the topmost (byte < kCkTop): adding 1.5 2^23 to the exact x / step rounds
// it to nearest even and leaves its low byte in the sum's.
__device__ __forceinline__ uint32_t ck_pack4(float2 a, float2 b, float inv) {
  const float2 magic = both(12582912.f);
  a = fma2(a, both(inv), magic);
  b = fma2(b, both(inv), magic);
  const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ uint32_t ck_pack4_any(float2 a, float2 b, uint32_t byte) {
  return ((uint32_t)ck_code(a.x, byte) & 255u) | ((uint32_t)ck_code(a.y, byte) & 255u) << 8 |
         ((uint32_t)ck_code(b.x, byte) & 255u) << 16 | (uint32_t)ck_code(b.y, byte) << 24;
}
// The four codes of a word as floats: a byte (plus 128) under the exponent of
// 2^23 reads as 2^23 + code + 128.
__device__ __forceinline__ void ck_unpack4(uint32_t w, float2& a, float2& b) {
  w ^= 0x80808080u;
  const float2 off = both(-8388736.f);
  a = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)),
                       __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441))), off);
  b = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)),
                       __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443))), off);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

}  // namespace rlk
