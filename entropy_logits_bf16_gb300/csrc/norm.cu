// rlk_norm_fwd / rlk_norm_bwd: layer and RMS norm.
//
//   m = mean x (RMS: 0),  r = (mean (x - m)^2 + eps)^-1/2,  h = (x - m) r,
//   y = h w + b;
//   g = dy w,  dx = r (g - mean g - h mean(g h))  (RMS: without mean g),
//   dw = sum_t dy h,  db = sum_t dy.
//
// Sums are fp32 in a fixed order; the parameter gradients go through per-part
// partial sums in the workspace that a second kernel adds in part order.

#include <math.h>

#include "checkpoint.cuh"
#include "internal.h"
#include "rlk.h"

namespace rlk {
namespace {

constexpr int kNormParts = 304;   // most row parts of the parameter gradients

__device__ __forceinline__ float ld_elem(const void* p, int dtype, int64_t i) {
  return dtype ? static_cast<const float*>(p)[i]
               : bf16_val(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void st_elem(void* p, int dtype, int64_t i, float v) {
  if (dtype) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float ck_value(const CheckpointView& ck, int64_t t, int64_t c) {
  return __fmul_rn((float)ck.codes[t * ck.ldc + c], ck_step(ck.scales[t * ck.lds + c / kCkBlock]));
}

// Sum over the CTA in a fixed order, on every thread.
template <int NW>
__device__ __forceinline__ float cta_sum(float v, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();   // the last sum's readers are done with s_red
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_red[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) v = __fadd_rn(v, s_red[w]);
  return v;
}

// ------------------------------------------------------------ rows of any width
constexpr int WT = 512;

__global__ void __launch_bounds__(WT) norm_fwd_wide_kernel(NormArgs a) {
  __shared__ float s_red[WT / 32];
  const int tid = threadIdx.x;
  const float inv_h = __fdiv_rn(1.f, (float)a.H);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t x0 = t * a.ldx;
    float m = 0.f, s = 0.f;
    if (!a.rms) {
      for (int64_t c = tid; c < a.H; c += WT) s = __fadd_rn(s, ld_elem(a.x, a.dtype, x0 + c));
      m = __fmul_rn(cta_sum<WT / 32>(s, s_red), inv_h);
      s = 0.f;
    }
    for (int64_t c = tid; c < a.H; c += WT) {
      const float d = __fsub_rn(ld_elem(a.x, a.dtype, x0 + c), m);
      s = __fmaf_rn(d, d, s);
    }
    const float var = __fmul_rn(cta_sum<WT / 32>(s, s_red), inv_h);
    const bool bad = !isfinite(var);
    const float r = bad ? NAN : __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(var, a.eps)));
    if (bad) m = NAN;
    if (tid == 0) {
      if (a.mean && !a.rms) a.mean[t] = m;
      if (a.rstd) a.rstd[t] = r;
      if (bad && a.status) atomicOr(a.status, RLK_STATUS_NONFINITE);
    }
    // whole blocks of 32 columns per warp, for the checkpoint
    for (int64_t c0 = tid & ~31; c0 < a.H; c0 += WT) {
      const int64_t c = c0 + (tid & 31);
      const bool in = c < a.H;
      const float x = in ? ld_elem(a.x, a.dtype, x0 + c) : 0.f;
      if (a.ck.codes) {
        const uint32_t byte = ck_scale_byte(__reduce_max_sync(0xFFFFFFFFu, abs_bits(x)));
        if (in) a.ck.codes[t * a.ck.ldc + c] = (int8_t)ck_code(x, byte);
        if ((tid & 31) == 0) a.ck.scales[t * a.ck.lds + c0 / kCkBlock] = (uint8_t)byte;
      }
      if (!in) continue;
      const float h = __fmul_rn(__fsub_rn(x, m), r);
      const float w = a.weight ? ld_elem(a.weight, a.param_dtype, c) : 1.f;
      const float b = a.bias ? ld_elem(a.bias, a.param_dtype, c) : 0.f;
      st_elem(a.y, a.y_dtype, t * a.ldy + c, __fmaf_rn(h, w, b));
    }
  }
}

__device__ __forceinline__ float bwd_x(const NormBwdArgs& a, int64_t t, int64_t c) {
  return a.x ? ld_elem(a.x, a.dtype, t * a.ldx + c) : ck_value(a.ck, t, c);
}

__global__ void __launch_bounds__(WT) norm_bwd_wide_kernel(NormBwdArgs a) {
  __shared__ float s_red[WT / 32];
  const float inv_h = __fdiv_rn(1.f, (float)a.H);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float m = a.rms ? 0.f : a.mean[t], r = a.rstd[t];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < a.H; c += WT) {
      const float w = a.weight ? ld_elem(a.weight, a.param_dtype, c) : 1.f;
      const float g = __fmul_rn(ld_elem(a.dy, a.dy_dtype, t * a.lddy + c), w);
      const float h = __fmul_rn(__fsub_rn(bwd_x(a, t, c), m), r);
      s1 = __fadd_rn(s1, g);
      s2 = __fmaf_rn(g, h, s2);
    }
    const float mg = a.rms ? 0.f : __fmul_rn(cta_sum<WT / 32>(s1, s_red), inv_h);
    const float mgh = __fmul_rn(cta_sum<WT / 32>(s2, s_red), inv_h);
    for (int64_t c = threadIdx.x; c < a.H; c += WT) {
      const float w = a.weight ? ld_elem(a.weight, a.param_dtype, c) : 1.f;
      const float g = __fmul_rn(ld_elem(a.dy, a.dy_dtype, t * a.lddy + c), w);
      const float h = __fmul_rn(__fsub_rn(bwd_x(a, t, c), m), r);
      st_elem(a.dx, a.dx_dtype, t * a.lddx + c,
              __fmul_rn(r, __fsub_rn(__fsub_rn(g, mg), __fmul_rn(h, mgh))));
    }
  }
}

// Partial dw, db of part blockIdx.y's rows (part p takes rows p, p + parts, ...).
__global__ void __launch_bounds__(256) norm_param_wide_kernel(NormBwdArgs a, int parts) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float dw = 0.f, db = 0.f;
  for (int64_t t = blockIdx.y; t < a.T; t += parts) {
    const float m = a.rms ? 0.f : a.mean[t], r = a.rstd[t];
    const float dy = ld_elem(a.dy, a.dy_dtype, t * a.lddy + c);
    dw = __fmaf_rn(dy, __fmul_rn(__fsub_rn(bwd_x(a, t, c), m), r), dw);
    db = __fadd_rn(db, dy);
  }
  float* p = a.workspace + (int64_t)blockIdx.y * 2 * a.H;
  p[c] = dw;
  p[a.H + c] = db;
}

__global__ void __launch_bounds__(256) norm_param_sum_kernel(NormBwdArgs a, int parts) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float* out = blockIdx.y ? a.db : a.dw;
  if (!out) return;
  float v = 0.f;
  for (int p = 0; p < parts; ++p) v = __fadd_rn(v, a.workspace[((int64_t)p * 2 + blockIdx.y) * a.H + c]);
  out[c] = a.accumulate ? __fadd_rn(out[c], v) : v;
}

int parts_for(int64_t T) { return (int)(T < kNormParts ? T : kNormParts); }

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  return ((size_t)parts_for(T) * 2 * (size_t)H * sizeof(float) + 255) & ~(size_t)255;
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream) {
  const int64_t cap = (int64_t)sm_count() * 4;
  norm_fwd_wide_kernel<<<(unsigned)(a.T < cap ? a.T : cap), WT, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t stream) {
  const int64_t cap = (int64_t)sm_count() * 4;
  if (a.T > 0) {
    norm_bwd_wide_kernel<<<(unsigned)(a.T < cap ? a.T : cap), WT, 0, stream>>>(a);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  if (!a.dw && !a.db) return cudaSuccess;
  const int parts = parts_for(a.T);
  const unsigned cols = (unsigned)((a.H + 255) / 256);
  if (parts > 0) {
    norm_param_wide_kernel<<<dim3(cols, parts), 256, 0, stream>>>(a, parts);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  norm_param_sum_kernel<<<dim3(cols, 2), 256, 0, stream>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace rlk
