// rlk_norm_fwd / rlk_norm_bwd: layer and RMS norm.
//
//   m = mean x (RMS: 0),  r = (mean (x - m)^2 + eps)^-1/2,  h = (x - m) r,
//   y = h w + b;
//   g = dy w,  dx = r (g - mean g - h mean(g h))  (RMS: without mean g),
//   dw = sum_t dy h,  db = sum_t dy.
//
// A few flops an element: bound by memory.  A row of up to 16384 columns lives
// in the registers of a group of threads, 16 or 32 columns a thread (4 to 512
// threads), so each pass reads every element once.  The CTAs are persistent,
// and the next rows are on their way to shared memory (bulk copies) while a group works:
//  * forward: a group has two rows at work (their sums share barriers); the
//    mean first, then the squares of the deviations from it.  w and b stay in registers.
//  * backward: a thread keeps its columns of w and of the partial dw, db over all
//    its rows (dw, db in shared memory where registers are short).  The CTAs'
//    partials go to the workspace and a second kernel adds them in order.
// Columns are taken 8 at a time (16-byte loads) where every row starts on a
// 16-byte boundary and H is a multiple of 8, else one at a time with
// consecutive columns on consecutive threads.  Wider rows
// take the any-width kernels: several passes over the row, and the parameter
// gradients in a pass of their own.
// Sums are fp32 in a fixed order.
//
// Measured, 16384 rows of 4096 bf16: RMS forward 52 us, backward from
// fp32 dy 81 us; layer norm's forward with the checkpoint written 80 us
// (52 M warp instructions against 31 M without it), its backward from the checkpoint
// and bf16 dy 79 us: 4.2 TB/s, half of the issue slots; 16 warps an SM do not
// cover the chains of instructions.  4099 rows of 5003
// (one column at a time): 36 us and 61 us, bound by instructions
// and barriers.  The parameter sums take 7 us.

#include <math.h>

#include <atomic>

#include "checkpoint.cuh"
#include "internal.h"
#include "rlk.h"

namespace rlk {
namespace {

constexpr int kNormParts = 304;   // most row parts of the parameter gradients
// Floats of a part's dw (and db): rows of 16 bytes.
__host__ __device__ __forceinline__ int64_t part_pitch(int64_t H) { return (H + 3) / 4 * 4; }

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

// v^-1/2: the hardware's approximation (about 2^-22) and one Newton step
// r (3 - v r^2) / 2; 0 and infinity as they come from the approximation.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float e = __fmaf_rn(__fmul_rn(-v, r), r, 1.f);   // 1 - v r^2
  return isfinite(e) ? __fmaf_rn(__fmul_rn(0.5f, r), e, r) : r;
}

// sum / n by the rounded reciprocal and one correction: the nearest fp32, or next to it,
// and exact where the quotient is.  (The product alone may be an ulp off the mean of a
// constant row, which eps then divides: y of +-0.5 where 29952 fills 1000 columns.)
__device__ __forceinline__ float mean_of(float sum, float n, float inv_n) {
  const float q = __fmul_rn(sum, inv_n);
  return __fmaf_rn(__fmaf_rn(-q, n, sum), inv_n, q);
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
      m = mean_of(cta_sum<WT / 32>(s, s_red), (float)a.H, inv_h);
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
  float* p = a.workspace + (int64_t)blockIdx.y * 2 * part_pitch(a.H);
  p[c] = dw;
  p[part_pitch(a.H) + c] = db;
}

// ------------------------------------------------------------ rows on chip
// A thread has E = 16 columns, or 32 in rows of over 8192 columns.
constexpr int kMaxGroup = 512;       // threads of a row, at most
// Registers of a thread.  The VW = 1 path (below) has longer chains of instructions
// to hide and takes fewer, so that two CTAs of up to 320 threads share an SM.
template <int VW, int E>
constexpr int regs_of() { return VW == 1 && E == 16 ? 96 : 128; }
// Where the backward's partial dw, db are: in shared memory when there are no
// registers for them.
template <int VW, int E>
constexpr bool sums_in_smem() { return VW == 1 || E == 32; }
constexpr int64_t kOnChip = 32 * kMaxGroup;

// The thread's E columns go VW at a time, consecutive threads on consecutive ones
// (col_of).  They are held as pairs, so that most of the arithmetic goes two
// elements an instruction (these kernels would otherwise be bound by issue).
// FULL (VW = 8): the threads' columns are exactly the row's, and nothing needs a
// bounds check.  VW = 1: that holds for every warp but the last (whole_warp).
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// element e of a thread's pairs
template <int E>
__device__ __forceinline__ float& elem(float2 (&v)[E / 2], int e) {
  return e % 2 ? v[e / 2].y : v[e / 2].x;
}

// The threads of a row: n of them, either a power of two up to 128 with several
// rows a CTA, or any multiple of 32 with one.
struct Group {
  int n, t, index, count;   // size, this thread, this group, groups of the CTA
  __device__ __forceinline__ explicit Group(int size)
      : n(size), t(size > 128 ? (int)threadIdx.x : (int)threadIdx.x & (size - 1)),
        index(size > 128 ? 0 : (int)threadIdx.x / size), count((int)blockDim.x / size) {}
  // all threads of the group (and of the CTA's other groups, where that takes a barrier)
  __device__ __forceinline__ void sync() const {
    if (n > 32) __syncthreads();
    else __syncwarp();
  }
};

// First of the k-th VW columns of the thread.  VW = 8: the group's threads side by
// side.  VW = 1: a warp has 32 E columns of its own, so that a thread's lie at
// distances known when this is compiled, and addresses take no arithmetic (with
// the group side by side, at multiples of its size, 16 columns took a warp
// some 700 instructions: 46 and 60 us forward and backward on 4099 rows of 5003).
template <int VW, int E>
__device__ __forceinline__ int col_of(int k, const Group& g) {
  return VW == 8 ? (k * g.n + g.t) * 8 : (g.t >> 5) * (32 * E) + (g.t & 31) + 32 * k;
}
template <int E>
__device__ __forceinline__ bool whole_warp(int H, const Group& g) { return ((g.t >> 5) + 1) * (32 * E) <= H; }

// Sums of NV values over the group, in a fixed order, on every thread.  `buf`
// alternates between two halves of s_red, so one barrier a sum is enough.
template <int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], const Group& g, float* s_red, int& buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (g.n >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int k = 0; k < NV; ++k) v[k] = __fadd_rn(v[k], __shfl_xor_sync(0xFFFFFFFFu, v[k], o));
    }
  } else {
    for (int o = g.n / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int k = 0; k < NV; ++k) v[k] = __fadd_rn(v[k], __shfl_xor_sync(0xFFFFFFFFu, v[k], o));
    }
  }
  if (g.n <= 32) return;
  float* s = s_red + buf;
  buf ^= 64;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) s[warp * NV + k] = v[k];
  }
  __syncthreads();
  const int nw = g.n / 32, at = lane & 15;   // at most 16 warps
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = at < nw ? s[(g.index * nw + at) * NV + k] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = __fadd_rn(v[k], __shfl_xor_sync(0xFFFFFFFFu, v[k], o));
  }
}

// A thread's columns of a row or of a parameter vector (0 past the end).
template <int VW, int E, bool FULL>
__device__ __forceinline__ void load_cols(const void* p, int dtype, int64_t at, int H, const Group& g,
                                          float2 (&v)[E / 2]) {
  if (VW == 8) {
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      const int c = col_of<8, E>(k, g);
      float2* o = v + k * 4;
      if (FULL || c + 8 <= H) {
        if (dtype) {
          const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + c);
          const float4 a = q[0], b = q[1];
          o[0] = make_float2(a.x, a.y); o[1] = make_float2(a.z, a.w);
          o[2] = make_float2(b.x, b.y); o[3] = make_float2(b.z, b.w);
        } else {
          const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at + c);
          o[0] = bf16x2_to_f2(q.x); o[1] = bf16x2_to_f2(q.y); o[2] = bf16x2_to_f2(q.z); o[3] = bf16x2_to_f2(q.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) elem<E>(v, 8 * k + j) = c + j < H ? ld_elem(p, dtype, at + c + j) : 0.f;
      }
    }
  } else {
    const int c = col_of<1, E>(0, g), left = H - c;
    if (dtype) {
      const float* q = static_cast<const float*>(p) + at + c;
#pragma unroll
      for (int e = 0; e < E; ++e) elem<E>(v, e) = 32 * e < left ? q[32 * e] : 0.f;
    } else {
      const uint16_t* q = static_cast<const uint16_t*>(p) + at + c;
#pragma unroll
      for (int e = 0; e < E; ++e) elem<E>(v, e) = 32 * e < left ? bf16_val(q[32 * e]) : 0.f;
    }
  }
}
template <int E, bool ALL>
__device__ __forceinline__ void store_single(void* p, int dtype, int64_t at, int left, float2 (&v)[E / 2]) {
  if (dtype) {
    float* q = static_cast<float*>(p) + at;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (ALL || 32 * e < left) q[32 * e] = elem<E>(v, e);
  } else {
    __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + at;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (ALL || 32 * e < left) q[32 * e] = __float2bfloat16_rn(elem<E>(v, e));
  }
}
template <int VW, int E, bool FULL>
__device__ __forceinline__ void store_cols(void* p, int dtype, int64_t at, int H, const Group& g, float2 (&v)[E / 2]) {
  if (VW == 8) {
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      const int c = col_of<8, E>(k, g);
      const float2* o = v + k * 4;
      if (FULL || c + 8 <= H) {
        if (dtype) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at + c);
          d[0] = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
          d[1] = make_float4(o[2].x, o[2].y, o[3].x, o[3].y);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at + c) =
              make_uint4(pack_bf16(o[0]), pack_bf16(o[1]), pack_bf16(o[2]), pack_bf16(o[3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < H) st_elem(p, dtype, at + c + j, elem<E>(v, 8 * k + j));
      }
    }
  } else {
    const int c = col_of<1, E>(0, g);
    if (whole_warp<E>(H, g)) store_single<E, true>(p, dtype, at + c, 0, v);
    else store_single<E, false>(p, dtype, at + c, H - c, v);
  }
}

// The thread's columns of the row's checkpoint.  VW = 8: a block of 32 columns
// is 4 neighbouring threads'; VW = 1: a warp's.  `finite`: the whole row is.
template <int VW, int E, bool FULL>
__device__ __forceinline__ void write_checkpoint(const CheckpointView& ck, int64_t row, bool live, bool finite, int H,
                                                 const Group& g, float2 (&x)[E / 2]) {
  int8_t* codes = ck.codes + row * ck.ldc;
  uint8_t* scales = ck.scales + row * ck.lds;
#pragma unroll
  for (int k = 0; k < E / VW; ++k) {
    uint32_t amax = 0u;
    if (finite) {
      float f = 0.f;
#pragma unroll
      for (int j = 0; j < VW; ++j) f = fmaxf(f, fabsf(elem<E>(x, k * VW + j)));
      amax = __float_as_uint(f);
    } else {
#pragma unroll
      for (int j = 0; j < VW; ++j) amax = max(amax, abs_bits(elem<E>(x, k * VW + j)));
    }
    if (VW == 8) {
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    } else {
      amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    }
    const uint32_t byte = ck_scale_byte(amax);
    const int c = col_of<VW, E>(k, g);
    if (!live || (!FULL && c >= H)) continue;
    if constexpr (VW == 8) {
      uint2 q;
      if (byte < kCkTop) {
        const float inv = ck_inv_step(byte);
        q = make_uint2(ck_pack4(x[4 * k], x[4 * k + 1], inv), ck_pack4(x[4 * k + 2], x[4 * k + 3], inv));
      } else {
        q = make_uint2(ck_pack4_any(x[4 * k], x[4 * k + 1], byte), ck_pack4_any(x[4 * k + 2], x[4 * k + 3], byte));
      }
      if (FULL || c + 8 <= H) {
        *reinterpret_cast<uint2*>(codes + c) = q;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < H) codes[c + j] = (int8_t)((j < 4 ? q.x : q.y) >> (8 * (j % 4)));
      }
    } else {
      codes[c] = (int8_t)ck_code(elem<E>(x, k), byte);
    }
    if (c % kCkBlock == 0) scales[c / kCkBlock] = (uint8_t)byte;
  }
}

// ---- rows on their way to shared memory
// Bulk copies: one thread of a group asks for whole rows, which keeps more bytes
// on their way than loads or cp.async did (reading fp32 dy and bf16 x by cp.async the
// backward stayed at 3.6 TB/s of reads whatever the depth: 108 us on 16384 rows of
// 4096; now 81 us).  A place has an mbarrier; every wait on one is
// bounded, and a row that did not come in time is NaN.
// Types: 0 bf16, 1 fp32, 2 checkpoint codes.
constexpr int kFromCk = 2;
constexpr int bytes_of(int type) { return type == 1 ? 4 : (type == 0 ? 2 : 1); }
constexpr int kMaxDepth = 4;

// The mbarriers of a group's places, and where its copies stand.
struct Places {
  uint32_t bar;     // the first barrier
  int depth, shift, issued;
  volatile int* abort;
  long long limit;  // clock cycles a wait may take
  // withheld: debug, the place of the first group whose barrier waits for an arrival that never comes (-1: none)
  __device__ __forceinline__ Places(uint64_t* bars, const Group& g, int d, volatile int* flag, long long wait_limit,
                                    long long withheld)
      : bar(smem_u32(bars + g.index * kMaxDepth)), depth(d), shift(d == 4 ? 2 : (d == 2 ? 1 : 0)), issued(0), abort(flag),
        limit(wait_limit) {
    if (threadIdx.x == 0) *abort = 0;
    if (g.t == 0) {
      for (int k = 0; k < depth; ++k) mbar_init(bar + 8 * k, 1 + (k == withheld && g.index == 0 && blockIdx.x == 0));
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncthreads();
  }
  __device__ __forceinline__ int of(int i) const { return i & (depth - 1); }
  __device__ __forceinline__ uint32_t bar_of(int i) const { return bar + 8 * of(i); }
  __device__ __forceinline__ bool came(int i) const { return mbar_try_wait(bar_of(i), (uint32_t)(i >> shift) & 1u); }
  // False when the limit ran out, or did for a row before: no copies are asked for
  // after that, and a barrier's parity says nothing about rows that were not.
  __device__ __forceinline__ bool wait(int i) const {
    if (i >= issued) return false;
    if (came(i)) return true;
    const long long t0 = clock64();
    for (;;) {
      if (*abort) return false;
      if (came(i)) return true;
      if (clock64() - t0 > limit) {
        *abort = 1;
        return false;
      }
    }
  }
  // after a wait has run out: lets the copies already asked for land
  __device__ __forceinline__ void drain() const {
    if (!*abort) return;
    const long long t0 = clock64();
    for (int i = issued > depth ? issued - depth : 0; i < issued; ++i)
      while (!came(i) && clock64() - t0 <= limit) {}
  }
};

// Bytes of a row's place in shared memory.  VW = 8: the threads' columns; VW = 1: the row's bytes at its own distance from a 16-byte boundary,
// and zeros up to the threads' last column (and the distance).
template <int TYPE, int VW, int E>
__host__ __device__ __forceinline__ int place_bytes(int H, int n) {
  return E * n * bytes_of(TYPE) + (VW == 8 ? 0 : 32);
}

// VW = 1: the element of a row that a thread carries to shared memory itself,
// being outside the whole 16-byte units of the bulk copy: threads 0..7 those
// before the first boundary, 8..15 those after the last.  -1: none.
template <int TYPE>
__device__ __forceinline__ int edge_byte(int to_boundary, int row_bytes, int t) {
  constexpr int es = bytes_of(TYPE);
  if (TYPE == kFromCk) return -1;   // rows of codes start on boundaries and are padded to whole units
  const int head = to_boundary < row_bytes ? to_boundary : row_bytes;
  if (t < 8) return t * es < head ? t * es : -1;
  const int at = head + ((row_bytes - head) & ~15) + (t - 8) * es;
  return t < 16 && at < row_bytes ? at : -1;
}
__device__ __forceinline__ int to_boundary(const void* p) { return (int)(-reinterpret_cast<uintptr_t>(p) & 15u); }

// The 16-byte units of a row (at element `at` of p) that a bulk copy brings, and
// where they go in its place.
struct Body {
  const char* src;
  int offset, bytes;
};
template <int TYPE, int VW>
__device__ __forceinline__ Body body_of(const void* p, int64_t at, int H) {
  constexpr int es = bytes_of(TYPE);
  const char* src = static_cast<const char*>(p) + at * es;
  const int row_bytes = H * es;
  if (VW == 8 || TYPE == kFromCk) return Body{src, 0, (row_bytes + 15) & ~15};   // whole units: see rows16
  const int gap = to_boundary(src), head = gap < row_bytes ? gap : row_bytes;
  return Body{src + head, (int)(reinterpret_cast<uintptr_t>(src) & 15u) + head, (row_bytes - head) & ~15};
}
// VW = 1: the edge element of a row that this thread has to store when the row is used.
template <int TYPE>
__device__ __forceinline__ uint32_t load_edge(const void* p, int64_t at, int H, const Group& g) {
  constexpr int es = bytes_of(TYPE);
  if (g.t >= 16) return 0u;
  const char* src = static_cast<const char*>(p) + at * es;
  const int e = edge_byte<TYPE>(to_boundary(src), H * es, g.t);
  if (e < 0) return 0u;
  return TYPE == 1 ? *reinterpret_cast<const uint32_t*>(src + e) : *reinterpret_cast<const uint16_t*>(src + e);
}
// VW = 1: stores the edge element of the row that started `at` there, and the
// zeros behind the row where an earlier one may have ended later.
template <int TYPE>
__device__ __forceinline__ void store_edge(uint8_t* place, const void* p, int64_t at, int H, const Group& g, uint32_t v) {
  constexpr int es = bytes_of(TYPE);
  if (TYPE == kFromCk || g.t >= 32) return;   // the codes past a row meet a dy of 0
  const char* src = static_cast<const char*>(p) + at * es;
  const int z = H * es + (g.t - 16) * es;
  if (g.t >= 16 && (g.t - 16) * es < 16) {
    uint8_t* d = place + (reinterpret_cast<uintptr_t>(src) & 15u) + z;
    if (TYPE == 1) *reinterpret_cast<uint32_t*>(d) = 0u;
    else *reinterpret_cast<uint16_t*>(d) = 0;
  }
  const int e = edge_byte<TYPE>(to_boundary(src), H * es, g.t);
  if (e < 0) return;
  uint8_t* d = place + (reinterpret_cast<uintptr_t>(src) & 15u) + e;
  if (TYPE == 1) *reinterpret_cast<uint32_t*>(d) = v;
  else *reinterpret_cast<uint16_t*>(d) = (uint16_t)v;
}

// A thread's columns of a row in shared memory (0 past the end; codes times
// their steps).
template <int TYPE, int VW, int E, bool FULL>
__device__ __forceinline__ void take_row(const uint8_t* place, const void* p, int64_t at, int H, const Group& g,
                                         const float (&step)[VW == 8 ? E / 8 : E], float2 (&v)[E / 2]) {
  constexpr int es = bytes_of(TYPE);
  if constexpr (VW == 8) {
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      const int c = col_of<8, E>(k, g);
      const uint8_t* s = place + c * es;
      float2* o = v + 4 * k;
      if (TYPE == 1) {
        const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
        o[0] = make_float2(a.x, a.y); o[1] = make_float2(a.z, a.w);
        o[2] = make_float2(b.x, b.y); o[3] = make_float2(b.z, b.w);
      } else if (TYPE == 0) {
        const uint4 q = *reinterpret_cast<const uint4*>(s);
        o[0] = bf16x2_to_f2(q.x); o[1] = bf16x2_to_f2(q.y); o[2] = bf16x2_to_f2(q.z); o[3] = bf16x2_to_f2(q.w);
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(s);
        ck_unpack4(q.x, o[0], o[1]);
        ck_unpack4(q.y, o[2], o[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = mul2(o[j], both(step[k]));
      }
      if (!FULL && c + 8 > H) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j >= H) elem<E>(v, 8 * k + j) = 0.f;
      }
    }
  } else {
    const uint8_t* s = place + ((reinterpret_cast<uintptr_t>(p) + at * es) & 15u) + col_of<1, E>(0, g) * es;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint8_t* q = s + 32 * e * es;
      float f;
      if (TYPE == 1) f = *reinterpret_cast<const float*>(q);
      else if (TYPE == 0) f = bf16_val(*reinterpret_cast<const uint16_t*>(q));
      else f = __fmul_rn((float)*reinterpret_cast<const int8_t*>(q), step[e]);
      elem<E>(v, e) = f;
    }
  }
}
// VW = 1: zeros in the places of `depth` rows, before the first copy.
__device__ __forceinline__ void clear_places(uint8_t* mine, int bytes, const Group& g) {
  for (int o = g.t * 16; o < bytes; o += g.n * 16) *reinterpret_cast<uint4*>(mine + o) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();   // before the copies into them
  g.sync();
}

template <int E>
__device__ __forceinline__ void fill(float2 (&v)[E / 2], float f) {
#pragma unroll
  for (int j = 0; j < E / 2; ++j) v[j] = both(f);
}

// ---- forward
// Persistent: a group takes rows index, + stride, ..., `depth` of them (1, 2, 4) on
// their way to shared memory ahead of the one at work.  E = 16 keeps its columns of
// weight and bias in registers.  R rows are at work together (their sums share
// barriers); depth >= R.
template <int XT, int VW, int E, bool FULL>
__global__ void __maxnreg__((regs_of<VW, E>())) norm_fwd_kernel(NormArgs a, int n, int depth) {
  constexpr int R = VW == 8 && E == 16 ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_red[128];
  int buf = 0;
  const Group g(n);
  const int H = (int)a.H;
  const int64_t stride = (int64_t)gridDim.x * g.count, row0 = (int64_t)blockIdx.x * g.count;
  const int iters = row0 < a.T ? (int)((a.T - row0 + stride - 1) / stride) : 0;
  const int size = place_bytes<XT, VW, E>(H, n);
  uint8_t* mine = smem + (size_t)g.index * depth * size;
  const float inv_h = __fdiv_rn(1.f, (float)H);
  const float none[VW == 8 ? E / 8 : E] = {};

  __shared__ uint64_t s_bars[kMaxDepth * 64];
  __shared__ int s_abort;
  Places places(s_bars, g, depth, &s_abort, a.wait_limit, a.withhold);
  if (VW == 1) clear_places(mine, depth * size, g);
  pdl_wait();   // the rows may come from the kernel before
  uint32_t edge[2] = {0u, 0u};   // VW = 1: depth is at most 2
  auto start = [&](int i) -> uint32_t {
    const int64_t row = row0 + g.index + i * stride;
    if (i >= iters || row >= a.T || *places.abort) return 0u;
    places.issued = i + 1;
    if (g.t == 0) {
      const Body b = body_of<XT, VW>(a.x, row * a.ldx, H);
      fence_proxy_async_smem();   // the place was read
      mbar_expect_tx(places.bar_of(i), b.bytes);
      if (b.bytes > 0) bulk_copy_g2s(smem_u32(mine + places.of(i) * size + b.offset), b.src, b.bytes, places.bar_of(i));
    }
    return VW == 1 ? load_edge<XT>(a.x, row * a.ldx, H, g) : 0u;
  };
  edge[0] = start(0);
  if (depth > 1) edge[1] = start(1);
  for (int i = 2; i < depth; ++i) start(i);

  constexpr bool KEEP = E == 16;
  float2 w[KEEP ? E / 2 : 1], b[KEEP ? E / 2 : 1];
  if constexpr (KEEP) {
    if (a.weight) load_cols<VW, E, FULL>(a.weight, a.param_dtype, 0, H, g, w);
    else fill<E>(w, 1.f);
    if (a.bias) load_cols<VW, E, FULL>(a.bias, a.param_dtype, 0, H, g, b);
    else fill<E>(b, 0.f);
  }

  for (int i = 0; i < iters; i += R) {
    float2 x[R][E / 2];
    float m[R], v[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t row = row0 + g.index + (i + q) * stride;
      const bool live = i + q < iters && row < a.T;
      uint8_t* place = mine + places.of(i + q) * size;
      if (VW == 1 && live) store_edge<XT>(place, a.x, row * a.ldx, H, g, edge[0]);
      const bool came = !live || places.wait(i + q);
      if (VW == 1) g.sync();
      if (!live) {
        fill<E>(x[q], 0.f);
      } else if (came) {
        take_row<XT, VW, E, FULL>(place, a.x, row * a.ldx, H, g, none, x[q]);
      } else {
        fill<E>(x[q], NAN);
        if (a.status) atomicOr(a.status, RLK_STATUS_TIMEOUT);
      }
      m[q] = 0.f;
    }
    if (!a.rms) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        float2 s = x[q][0];
#pragma unroll
        for (int j = 1; j < E / 2; ++j) s = add2(s, x[q][j]);
        m[q] = __fadd_rn(s.x, s.y);
      }
      group_sum(m, g, s_red, buf);
#pragma unroll
      for (int q = 0; q < R; ++q) m[q] = mean_of(m[q], (float)H, inv_h);
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 s = both(0.f);
      if (VW == 8 ? FULL || a.rms : a.rms || whole_warp<E>(H, g)) {   // with m = 0 the zeros past the end add nothing
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const float2 d = add2(x[q][j], both(-m[q]));
          s = fma2(d, d, s);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = col_of<VW, E>(e / VW, g) + e % VW < H ? __fsub_rn(elem<E>(x[q], e), m[q]) : 0.f;
          if (e % 2) s.y = __fmaf_rn(d, d, s.y);
          else s.x = __fmaf_rn(d, d, s.x);
        }
      }
      v[q] = __fadd_rn(s.x, s.y);
    }
    group_sum(v, g, s_red, buf);
    // the sum's barrier: every thread has read the places
    if (n <= 32) __syncwarp();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t e = start(i + q + depth);
      edge[0] = depth == 2 ? edge[1] : e;
      edge[1] = e;
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t row = row0 + g.index + (i + q) * stride;
      const bool live = i + q < iters && row < a.T;
      const float var = __fmul_rn(v[q], inv_h);
      const bool bad = !isfinite(var);
      const float r = bad ? NAN : inv_sqrt(__fadd_rn(var, a.eps));
      if (bad) m[q] = NAN;
      if (live && g.t == 0) {
        if (a.mean && !a.rms) a.mean[row] = m[q];
        if (a.rstd) a.rstd[row] = r;
        if (bad && a.status) atomicOr(a.status, RLK_STATUS_NONFINITE);
      }
      if (a.ck.codes) write_checkpoint<VW, E, FULL>(a.ck, row, live, !bad, H, g, x[q]);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        x[q][j] = mul2(add2(x[q][j], both(-m[q])), both(r));
        if constexpr (KEEP) x[q][j] = fma2(x[q][j], w[j], b[j]);
      }
      if constexpr (!KEEP) {
        float2 p[E / 2];
        if (a.weight) {
          load_cols<VW, E, FULL>(a.weight, a.param_dtype, 0, H, g, p);
#pragma unroll
          for (int j = 0; j < E / 2; ++j) x[q][j] = mul2(x[q][j], p[j]);
        }
        if (a.bias) {
          load_cols<VW, E, FULL>(a.bias, a.param_dtype, 0, H, g, p);
#pragma unroll
          for (int j = 0; j < E / 2; ++j) x[q][j] = add2(x[q][j], p[j]);
        }
      }
      if (live) store_cols<VW, E, FULL>(a.y, a.y_dtype, row * a.ldy, H, g, x[q]);
    }
  }
  if (g.t == 0) places.drain();
}

// ---- backward
// XT: type of x, 2: from its checkpoint; DT: type of dy.  Rows as in the
// forward; `depth` 0: a row is loaded when its turn comes (rows that do not fit).
template <int XT, int DT, int VW, int E, bool FULL>
__global__ void __maxnreg__((regs_of<VW, E>())) norm_bwd_kernel(NormBwdArgs a, int n, int depth) {
  constexpr bool SACC = sums_in_smem<VW, E>(), KEEP = E == 16;
  constexpr int STEPS = VW == 8 ? E / 8 : E;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_red[128];
  int buf = 0;
  const Group g(n);
  const int H = (int)a.H;
  const float inv_h = __fdiv_rn(1.f, (float)H);
  float2* s_acc = reinterpret_cast<float2*>(smem);   // SACC: [groups][2][E / 2][n]
  const int dy_size = place_bytes<DT, VW, E>(H, n), size = dy_size + place_bytes<XT, VW, E>(H, n);
  uint8_t* mine = smem + (SACC ? g.count * 2 * E * n * 4 : 0) + (size_t)g.index * depth * size;
  if (SACC) s_acc += g.index * E * n;
  const int64_t stride = (int64_t)gridDim.x * g.count, row0 = (int64_t)blockIdx.x * g.count;
  const int iters = row0 < a.T ? (int)((a.T - row0 + stride - 1) / stride) : 0;
  const void* xp = XT == kFromCk ? static_cast<const void*>(a.ck.codes) : a.x;
  const int64_t ldx = XT == kFromCk ? a.ck.ldc : a.ldx;

  __shared__ uint64_t s_bars[kMaxDepth * 64];
  __shared__ int s_abort;
  Places places(s_bars, g, depth, &s_abort, a.wait_limit, a.withhold);
  if (VW == 1) clear_places(mine, depth * size, g);
  pdl_wait();
  uint2 edge[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};   // VW = 1: depth is at most 2
  auto place = [&](int i) { return mine + places.of(i) * size; };
  auto start = [&](int i) -> uint2 {
    const int64_t row = row0 + g.index + i * stride;
    uint2 e = make_uint2(0u, 0u);
    if (i >= iters || row >= a.T || *places.abort) return e;
    places.issued = i + 1;
    if (g.t == 0) {
      const Body y = body_of<DT, VW>(a.dy, row * a.lddy, H), x = body_of<XT, VW>(xp, row * ldx, H);
      fence_proxy_async_smem();   // the place was read
      const uint32_t bar = places.bar_of(i);
      mbar_expect_tx(bar, y.bytes + x.bytes);
      if (y.bytes > 0) bulk_copy_g2s(smem_u32(place(i) + y.offset), y.src, y.bytes, bar);
      if (x.bytes > 0) bulk_copy_g2s(smem_u32(place(i) + dy_size + x.offset), x.src, x.bytes, bar);
    }
    if (VW == 1) {
      e.x = load_edge<DT>(a.dy, row * a.lddy, H, g);
      e.y = load_edge<XT>(xp, row * ldx, H, g);
    }
    return e;
  };
  if (depth > 0) edge[0] = start(0);
  if (depth > 1) edge[1] = start(1);
  for (int i = 2; i < depth; ++i) start(i);
  // a row's statistics and checkpoint steps, read one row ahead
  float m1 = 0.f, r1 = 0.f;
  uint32_t byte1[STEPS];
  auto ahead = [&](int i) {
    const int64_t row = row0 + g.index + i * stride;
    const bool in = i < iters && row < a.T;
    m1 = in && !a.rms ? a.mean[row] : 0.f;
    r1 = in ? a.rstd[row] : 0.f;
    if (XT == kFromCk) {
      const uint8_t* sc = a.ck.scales + row * a.ck.lds;
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        const int c = col_of<VW, E>(k, g);
        byte1[k] = in && (FULL || c < H) ? sc[c / kCkBlock] : 1u;
      }
    }
  };
  ahead(0);

  float2 w[E / 2], dw[SACC ? 1 : E / 2], db[SACC ? 1 : E / 2];
  auto load_w = [&]() {
    if (a.weight) load_cols<VW, E, FULL>(a.weight, a.param_dtype, 0, H, g, w);
    else fill<E>(w, 1.f);
  };
  if (KEEP) load_w();   // else with each row: there are no registers to keep it in
#pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    if (SACC) s_acc[j * n + g.t] = s_acc[(E / 2 + j) * n + g.t] = both(0.f);
    else dw[j] = db[j] = both(0.f);
  }

  for (int i = 0; i < iters; ++i) {
    const int64_t row = row0 + g.index + i * stride;
    const bool live = row < a.T;
    const float m = m1, r = r1;
    float step[STEPS];
    if (XT == kFromCk) {
#pragma unroll
      for (int k = 0; k < STEPS; ++k) step[k] = ck_step(byte1[k]);
    }
    float2 dy[E / 2], h[E / 2];
    if (!live) {
      fill<E>(dy, 0.f);
      fill<E>(h, 0.f);
    }
    if (depth > 0) {
      if (VW == 1 && live) {
        store_edge<DT>(place(i), a.dy, row * a.lddy, H, g, edge[0].x);
        store_edge<XT>(place(i) + dy_size, xp, row * ldx, H, g, edge[0].y);
      }
      const bool came = !live || places.wait(i);
      if (VW == 1) g.sync();
      if (live && came) {
        take_row<DT, VW, E, FULL>(place(i), a.dy, row * a.lddy, H, g, step, dy);
        take_row<XT, VW, E, FULL>(place(i) + dy_size, xp, row * ldx, H, g, step, h);
      } else if (live) {
        fill<E>(dy, NAN);
        fill<E>(h, NAN);
      }
    } else if (live) {
      load_cols<VW, E, FULL>(a.dy, DT, row * a.lddy, H, g, dy);
      if (XT == kFromCk) {
        const int8_t* q = a.ck.codes + row * a.ck.ldc;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = col_of<VW, E>(e / VW, g) + e % VW;
          elem<E>(h, e) = c < H ? __fmul_rn((float)q[c], step[VW == 8 ? e / 8 : e]) : 0.f;
        }
      } else {
        load_cols<VW, E, FULL>(a.x, XT, row * a.ldx, H, g, h);
      }
    }
    ahead(i + 1);
    if (!KEEP) load_w();
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {   // past the row dy is 0, and h does not matter
      h[j] = mul2(add2(h[j], both(-m)), both(r));
      const float2 gr = mul2(dy[j], w[j]);
      s1 = add2(s1, gr);
      s2 = fma2(gr, h[j], s2);
      if (SACC) {
        s_acc[j * n + g.t] = fma2(dy[j], h[j], s_acc[j * n + g.t]);
        s_acc[(E / 2 + j) * n + g.t] = add2(s_acc[(E / 2 + j) * n + g.t], dy[j]);
      } else {
        dw[j] = fma2(dy[j], h[j], dw[j]);
        db[j] = add2(db[j], dy[j]);
      }
      dy[j] = gr;
    }
    float v[2] = {__fadd_rn(s2.x, s2.y), __fadd_rn(s1.x, s1.y)};
    group_sum(v, g, s_red, buf);
    if (depth > 0) {   // the sum's barrier: every thread has read the place
      if (n <= 32) __syncwarp();
      const uint2 e = start(i + depth);
      edge[0] = depth == 2 ? edge[1] : e;
      edge[1] = e;
    }
    const float mg = a.rms ? 0.f : __fmul_rn(v[1], inv_h), mgh = __fmul_rn(v[0], inv_h);
#pragma unroll
    for (int j = 0; j < E / 2; ++j)
      h[j] = mul2(both(r), fma2(h[j], both(-mgh), add2(dy[j], both(-mg))));
    if (live) store_cols<VW, E, FULL>(a.dx, a.dx_dtype, row * a.lddx, H, g, h);
  }
  if (g.t == 0) places.drain();
  if (!a.workspace) return;
  float* part = a.workspace + (int64_t)blockIdx.x * 2 * part_pitch(a.H);
  if constexpr (SACC) {
    if (g.count > 1) __syncthreads();
    if (g.index > 0) return;
    float2 v[E / 2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {   // the CTA's groups, added in order
        v[j] = s_acc[(k * E / 2 + j) * n + g.t];
        for (int q = 1; q < g.count; ++q) v[j] = add2(v[j], s_acc[q * E * n + (k * E / 2 + j) * n + g.t]);
      }
      store_cols<VW, E, FULL>(part + k * part_pitch(a.H), 1, 0, H, g, v);
    }
  } else {
    // the CTA's groups, added in order (every copy has landed: the shared memory is free again)
    if (g.count > 1) {
      for (int k = 0; k < g.count; ++k) {
        __syncthreads();
        if (g.index != k) continue;
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          float2* p = s_acc + j * n + g.t;
          float2* q = s_acc + (E / 2 + j) * n + g.t;
          *p = dw[j] = k ? add2(*p, dw[j]) : dw[j];
          *q = db[j] = k ? add2(*q, db[j]) : db[j];
        }
      }
      if (g.index != g.count - 1) return;
    }
    store_cols<VW, E, FULL>(part, 1, 0, H, g, dw);
    store_cols<VW, E, FULL>(part + part_pitch(a.H), 1, 0, H, g, db);
  }
}

// Adds the parts in order: 32 columns a CTA, warp w takes parts w, w + 8, ...,
// 20 of them on their way together.
__global__ void __launch_bounds__(256) norm_param_sum_kernel(NormBwdArgs a, int parts) {
  pdl_wait();
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* out = blockIdx.y ? a.db : a.dw;
  if (!out) return;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane, pitch = 2 * part_pitch(a.H);
  const float* p = a.workspace + blockIdx.y * part_pitch(a.H) + c;
  float v = 0.f;
  for (int k0 = warp; k0 < parts; k0 += 160) {
    float x[20];
#pragma unroll
    for (int u = 0; u < 20; ++u) x[u] = c < a.H && k0 + 8 * u < parts ? p[(k0 + 8 * u) * pitch] : 0.f;
#pragma unroll
    for (int u = 0; u < 20; ++u) v = __fadd_rn(v, x[u]);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < a.H) {
    for (int k = 1; k < 8; ++k) v = __fadd_rn(v, s[k][lane]);
    out[c] = a.accumulate ? __fadd_rn(out[c], v) : v;
  }
}

// ------------------------------------------------------------ host side
int parts_for(int64_t T) { return (int)(T < kNormParts ? T : kNormParts); }

// Columns of a thread, and threads of a row on chip: a power of two up to 128,
// then whole warps.  One column at a time (vec false) takes at least a warp.
int cols_for(int64_t H) { return H > 16 * kMaxGroup ? 32 : 16; }
int group_for(int64_t H, bool vec) {
  const int64_t want = (H + cols_for(H) - 1) / cols_for(H);
  if (want > 128) return (int)((want + 31) / 32 * 32);
  int n = vec ? 4 : 32;
  while (n < want) n *= 2;
  return n;
}
constexpr size_t kSmemMost = 223 * 1024;   // dynamic, beside the kernels' own 3 KB
bool rows16(const void* p, int dtype, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (dtype ? 4 : 8) == 0;
}
bool base16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <class K>
cudaError_t allow_smem(K kernel, std::atomic<int>* done) {
  const int ds = device_slot();
  if (ds >= 0 && done[ds].load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
  if (e == cudaSuccess && ds >= 0) done[ds].store(1);
  return e;
}
// CTAs an SM: by the registers, two at most (three, with 80 registers and a row at a
// time in the forward: 67 us on 16384 rows of 4096, layer norm; two, with two rows: 58).
template <int VW, int E>
int ctas_for(int block) { return 2 * block * regs_of<VW, E>() <= 65536 ? 2 : 1; }
// Rows on their way, as many (a power of two) as leave room for the SM's CTAs.
int depth_for(size_t row, size_t fixed, int ctas, int most) {
  const size_t room = ctas == 1 ? kSmemMost : 110 * 1024;
  int d = most;
  while (d > 0 && fixed + d * row > room) d /= 2;
  return d;
}

template <int XT, int VW, int E, bool FULL = false>
cudaError_t fwd(const NormArgs& a, cudaStream_t stream) {
  auto kernel = norm_fwd_kernel<XT, VW, E, FULL>;
  static std::atomic<int> done[64];
  if (cudaError_t e = allow_smem(kernel, done); e != cudaSuccess) return e;
  const int n = group_for(a.H, VW == 8), block = n > 128 ? n : 256, groups = block / n;
  const size_t row = (size_t)groups * place_bytes<XT, VW, E>((int)a.H, n);
  const int ctas = ctas_for<VW, E>(block), depth = depth_for(row, 0, ctas, VW == 8 ? 4 : 2);
  const int64_t want = (a.T + groups - 1) / groups, cap = (int64_t)sm_count() * ctas;
  const cudaError_t e = launch_after(kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(block), depth * row, stream, a, n, depth);
  return e != cudaSuccess ? e : cudaGetLastError();
}
// FULL of the kernels for VW = 8.
bool full_row(int64_t H) { return group_for(H, true) * cols_for(H) == H; }

template <int XT>
cudaError_t fwd_for(const NormArgs& a, bool vec, cudaStream_t stream) {
  const bool wide = cols_for(a.H) == 32;
  if (!vec) return wide ? fwd<XT, 1, 32>(a, stream) : fwd<XT, 1, 16>(a, stream);
  if (full_row(a.H)) return wide ? fwd<XT, 8, 32, true>(a, stream) : fwd<XT, 8, 16, true>(a, stream);
  return wide ? fwd<XT, 8, 32>(a, stream) : fwd<XT, 8, 16>(a, stream);
}

template <int XT, int DT, int VW, int E, bool FULL = false>
cudaError_t bwd(const NormBwdArgs& a, int& parts, cudaStream_t stream) {
  auto kernel = norm_bwd_kernel<XT, DT, VW, E, FULL>;
  static std::atomic<int> done[64];
  if (cudaError_t e = allow_smem(kernel, done); e != cudaSuccess) return e;
  const int n = group_for(a.H, VW == 8), block = n > 128 ? n : 256, groups = block / n;
  constexpr bool SACC = sums_in_smem<VW, E>();
  const size_t acc = (size_t)2 * E * n * sizeof(float) * (SACC ? groups : 1);
  const size_t row = (size_t)groups * (place_bytes<XT, VW, E>((int)a.H, n) + place_bytes<DT, VW, E>((int)a.H, n));
  const int ctas = ctas_for<VW, E>(block), depth = depth_for(row, SACC ? acc : 0, ctas, VW == 8 ? 4 : 2);
  size_t smem = depth * row;
  if (SACC) smem += acc;
  else if (groups > 1 && smem < acc) smem = acc;
  const int64_t want = (a.T + groups - 1) / groups, cap = kNormParts / 2 * ctas;
  parts = (int)(want < cap ? want : cap);
  const cudaError_t e = launch_after(kernel, dim3(parts), dim3(block), smem, stream, a, n, depth);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int XT, int DT>
cudaError_t bwd_for(const NormBwdArgs& a, bool vec, int& parts, cudaStream_t stream) {
  const bool wide = cols_for(a.H) == 32;
  if (!vec) return wide ? bwd<XT, DT, 1, 32>(a, parts, stream) : bwd<XT, DT, 1, 16>(a, parts, stream);
  if (full_row(a.H)) return wide ? bwd<XT, DT, 8, 32, true>(a, parts, stream) : bwd<XT, DT, 8, 16, true>(a, parts, stream);
  return wide ? bwd<XT, DT, 8, 32>(a, parts, stream) : bwd<XT, DT, 8, 16>(a, parts, stream);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  return ((size_t)parts_for(T) * 2 * (size_t)part_pitch(H) * sizeof(float) + 255) & ~(size_t)255;
}

cudaError_t launch_norm_fwd(const NormArgs& args, cudaStream_t stream) {
  NormArgs a = args;
  if (a.H <= kOnChip) {
    a.wait_limit = debug_wait_limit();
    a.withhold = debug_take_withheld();
    const bool vec = a.H % 8 == 0 && rows16(a.x, a.dtype, a.ldx) && rows16(a.y, a.y_dtype, a.ldy) && base16(a.weight) && base16(a.bias);
    return a.dtype ? fwd_for<1>(a, vec, stream) : fwd_for<0>(a, vec, stream);
  }
  const int64_t cap = (int64_t)sm_count() * 4;
  norm_fwd_wide_kernel<<<(unsigned)(a.T < cap ? a.T : cap), WT, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormBwdArgs& args, cudaStream_t stream) {
  NormBwdArgs a = args;
  if (!a.dw && !a.db) a.workspace = nullptr;
  int parts = 0;
  if (a.T > 0 && a.H <= kOnChip) {
    a.wait_limit = debug_wait_limit();
    a.withhold = debug_take_withheld();
    const bool vec = a.H % 8 == 0 && rows16(a.dy, a.dy_dtype, a.lddy) && rows16(a.dx, a.dx_dtype, a.lddx) && base16(a.weight) &&
                     (!a.x || rows16(a.x, a.dtype, a.ldx));
    const int type = !a.x ? kFromCk : a.dtype;
    cudaError_t e;
    if (a.dy_dtype == 0)
      e = type == 0 ? bwd_for<0, 0>(a, vec, parts, stream) : type == 1 ? bwd_for<1, 0>(a, vec, parts, stream)
                                                                    : bwd_for<kFromCk, 0>(a, vec, parts, stream);
    else
      e = type == 0 ? bwd_for<0, 1>(a, vec, parts, stream) : type == 1 ? bwd_for<1, 1>(a, vec, parts, stream)
                                                                    : bwd_for<kFromCk, 1>(a, vec, parts, stream);
    if (e != cudaSuccess) return e;
  } else if (a.T > 0) {
    const int64_t cap = (int64_t)sm_count() * 4;
    norm_bwd_wide_kernel<<<(unsigned)(a.T < cap ? a.T : cap), WT, 0, stream>>>(a);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (a.workspace) {
      parts = parts_for(a.T);
      norm_param_wide_kernel<<<dim3((unsigned)((a.H + 255) / 256), parts), 256, 0, stream>>>(a, parts);
      if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
  }
  if (!a.workspace) return cudaSuccess;
  const cudaError_t e = launch_after(norm_param_sum_kernel, dim3((unsigned)((a.H + 31) / 32), 2), dim3(256), 0, stream, a, parts);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rlk
