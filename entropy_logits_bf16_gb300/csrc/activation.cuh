// The activations of the linear layers with their slopes, and bf16 stores of a few columns.
#pragma once

#include "common.cuh"
#include "rlk.h"

namespace rlk {
namespace {

// 1 / v to 2^-23 (MUFU; a result below 2^-126 is 0).
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Phi(-|z|), Phi the normal distribution function, two numbers an instruction, to a
// relative (2 z^2 + 24) 2^-24 (half an ulp of z alone moves it by z^2 2^-24):
// Phi(-|z|) = t q(t) exp(-z^2 / 2) with t = 1 / (1 + 0.305 |z|).  t q(t) is half the scaled
// complementary error function erfcx(|z| / sqrt 2); q is its minimax fit in t, by relative
// error (9.4e-8) over |z| <= 13.3, beyond which the exponential is below 2^-126 and is 0.
// `bell`: exp(-z^2 / 2).
__device__ __forceinline__ float2 normal_tail(float2 z, float2& bell) {
  const float2 d = fma2(make_float2(fabsf(z.x), fabsf(z.y)), both(0.305f), both(1.f));
  const float2 t = make_float2(rcp(d.x), rcp(d.y));
  float2 q = fma2(both(0.0366991907f), t, both(-0.1529883f));
  q = fma2(q, t, both(0.185716853f));
  q = fma2(q, t, both(-0.0379767865f));
  q = fma2(q, t, both(0.121021658f));
  q = fma2(q, t, both(0.103420876f));
  q = fma2(q, t, both(0.122466817f));
  q = fma2(q, t, both(0.121639736f));
  const float2 e = mul2(mul2(z, z), both(-0.5f * kLog2e));
  bell = make_float2(ex2(e.x), ex2(e.y));
  return mul2(mul2(q, t), bell);
}
// Phi(z) from Phi(-|z|).
__device__ __forceinline__ float2 normal_below(float2 z, float2 tail) {
  const float2 up = fma2(tail, both(-1.f), both(1.f));
  return make_float2(z.x > 0.f ? up.x : tail.x, z.y > 0.f ? up.y : tail.y);
}
// 1 / (1 + exp(-z)), to a relative (2 |z| + 24) 2^-24.
__device__ __forceinline__ float2 logistic(float2 z) {
  const float2 e = mul2(z, both(-kLog2e)), d = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}
// act of W values; the choice is made once.
template <int W>
__device__ __forceinline__ void activate(float (&v)[W], int act) {
  if (act == RLK_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < W; j += 2) {
      const float2 z = make_float2(v[j], v[j + 1 < W ? j + 1 : j]);
      float2 bell;
      const float2 tail = normal_tail(z, bell), o = mul2(z, normal_below(z, tail));
      v[j] = o.x;
      if (j + 1 < W) v[j + 1] = o.y;
    }
  } else if (act == RLK_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < W; j += 2) {
      const float2 z = make_float2(v[j], v[j + 1 < W ? j + 1 : j]), o = mul2(z, logistic(z));
      v[j] = o.x;
      if (j + 1 < W) v[j + 1] = o.y;
    }
  } else if (act == RLK_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];
  }
}
// act'(z), to the same.
template <int ACT>
__device__ __forceinline__ float2 activation_slope(float2 z) {
  if (ACT == RLK_ACT_GELU) {   // Phi(z) + z phi(z)
    float2 bell;
    const float2 tail = normal_tail(z, bell);
    return fma2(mul2(z, bell), both(0.39894228040143268f), normal_below(z, tail));
  }
  if (ACT == RLK_ACT_SILU) {
    const float2 s = logistic(z);
    return mul2(s, fma2(z, fma2(s, both(-1.f), both(1.f)), both(1.f)));
  }
  auto relu = [](float v) { return v > 0.f ? 1.f : (v != v ? v : 0.f); };
  return make_float2(relu(z.x), relu(z.y));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 columns of one row that starts on a 16-byte boundary there; n of the columns exist.
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], int n) {
  if (n == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                              pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint16_t)pack_bf16(v[j], 0.f);
  }
}

}  // namespace
}  // namespace rlk
