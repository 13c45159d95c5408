// rlk_checkpoint_pack / rlk_checkpoint_unpack: an activation as 8-bit codes
// with a power-of-two step per 32 columns, and back.
//
// A maximum, a multiplication and a conversion an element against 3 to 5 bytes of
// traffic: bound by memory.  Measured on 55296 rows of 4096 bf16: pack 109 us,
// unpack 108 us.  Rows that start on 16-byte boundaries go 16
// columns a thread (two threads share a block, and each has the loads of several rows
// in flight); others one column a lane, a block a warp, four blocks in flight.

#include "checkpoint.cuh"
#include "internal.h"
#include "rlk.h"

namespace rlk {
namespace {

constexpr int CT = 256;
// Rows a thread has in flight (16 columns a thread): 128 bytes of them.
constexpr int pack_rows(int dtype) { return dtype ? 2 : 4; }
constexpr int UNPACK_ROWS = 2;   // 4: 114 us on 55296 rows of 4096 instead of 107
constexpr int BLOCKS = 4;   // blocks a warp has in flight (one column a lane)

__device__ __forceinline__ float ld_elem(const void* p, int dtype, int64_t i) {
  return dtype ? static_cast<const float*>(p)[i]
               : bf16_val(static_cast<const uint16_t*>(p)[i]);
}

// 16 columns as they lie in memory, and as pairs.
template <int DT>
struct Raw {
  uint4 q[DT ? 4 : 2];
};
// From column c on (0 past the row).
template <int DT>
__device__ __forceinline__ void load16(const void* p, int64_t at, int c, int H, Raw<DT>& r) {
  constexpr int N = DT ? 4 : 2;
  if (c + 16 <= H) {
    const uint4* q = DT ? reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at + c)
                        : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at + c);
#pragma unroll
    for (int k = 0; k < N; ++k) r.q[k] = q[k];
  } else {
    uint32_t w[4 * N];
#pragma unroll
    for (int k = 0; k < 4 * N; ++k) {
      if (DT) {
        w[k] = c + k < H ? static_cast<const uint32_t*>(p)[at + c + k] : 0u;
      } else {
        const uint16_t* e = static_cast<const uint16_t*>(p) + at + c + 2 * k;
        w[k] = (c + 2 * k < H ? e[0] : 0u) | (c + 2 * k + 1 < H ? (uint32_t)e[1] << 16 : 0u);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) r.q[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}
template <int DT>
__device__ __forceinline__ void as_pairs(const Raw<DT>& r, float2 (&v)[8]) {
#pragma unroll
  for (int k = 0; k < (DT ? 4 : 2); ++k) {
    const uint32_t w[4] = {r.q[k].x, r.q[k].y, r.q[k].z, r.q[k].w};
    if (DT) {
      v[2 * k] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      v[(2 * k + 1) % 8] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[(4 * k + j) % 8] = bf16x2_to_f2(w[j]);
    }
  }
}

// n threads a row (a power of two up to CT), ROWS rows a thread.
template <int DT>
__global__ void __launch_bounds__(CT) checkpoint_pack_kernel(CheckpointArgs a, int n) {
  constexpr int ROWS = pack_rows(DT);
  const int t = threadIdx.x & (n - 1), H = (int)a.H, per = CT / n;
  const int64_t r0 = (int64_t)blockIdx.x * per * ROWS + threadIdx.x / n;
  bool bad = false;
  // every thread of a pair makes every step: the shuffle needs both
  for (int c0 = 0; c0 < H; c0 += n * 16) {
    const int c = c0 + t * 16;
    Raw<DT> raw[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
      if (r0 + k * per < a.T) load16<DT>(a.x, (r0 + k * per) * a.ldx, c, H, raw[k]);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r0 + k * per;
      float2 v[8];
      as_pairs(raw[k], v);
      // fmaxf passes over a NaN; 0 x is one where x is a NaN or an infinity
      float2 nan = both(0.f);
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top = fmaxf(top, fmaxf(fabsf(v[j].x), fabsf(v[j].y)));
        nan = fma2(v[j], both(0.f), nan);
      }
      uint32_t amax = nan.x + nan.y == 0.f ? __float_as_uint(top) : 0x7FC00000u;
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      const uint32_t byte = ck_scale_byte(amax);
      if (row >= a.T || c >= H) continue;
      bad = bad || byte == 255u;
      uint32_t q[4];
      const float inv = ck_inv_step(byte);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[j] = byte < kCkTop ? ck_pack4(v[2 * j], v[2 * j + 1], inv) : ck_pack4_any(v[2 * j], v[2 * j + 1], byte);
      int8_t* dst = a.ck.codes + row * a.ck.ldc + c;
      if (c + 16 <= H) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < H) dst[j] = (int8_t)(q[j / 4] >> (8 * (j % 4)));
      }
      if ((t & 1) == 0) a.ck.scales[row * a.ck.lds + c / kCkBlock] = (uint8_t)byte;
    }
  }
  if (bad && a.status) atomicOr(a.status, RLK_STATUS_NONFINITE);
}

template <int DT>
__global__ void __launch_bounds__(CT) checkpoint_unpack_kernel(CheckpointArgs a, int n) {
  const int t = threadIdx.x & (n - 1), H = (int)a.H, per = CT / n;
  const int64_t r0 = (int64_t)blockIdx.x * per * UNPACK_ROWS + threadIdx.x / n;
  for (int c = t * 16; c < H; c += n * 16) {
    uint4 q[UNPACK_ROWS];
    float step[UNPACK_ROWS];
#pragma unroll
    for (int k = 0; k < UNPACK_ROWS; ++k) {
      const int64_t row = r0 + k * per;
      if (row >= a.T) continue;
      q[k] = *reinterpret_cast<const uint4*>(a.ck.codes + row * a.ck.ldc + c);   // ld_codes is a multiple of 16
      step[k] = ck_step(a.ck.scales[row * a.ck.lds + c / kCkBlock]);
    }
#pragma unroll
    for (int k = 0; k < UNPACK_ROWS; ++k) {
      const int64_t row = r0 + k * per;
      if (row >= a.T) continue;
      const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
      float2 v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ck_unpack4(w[j], v[2 * j], v[2 * j + 1]);
        v[2 * j] = mul2(v[2 * j], both(step[k]));
        v[2 * j + 1] = mul2(v[2 * j + 1], both(step[k]));
      }
      if (c + 16 <= H) {
        if (DT) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.x) + row * a.ldx + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
        } else {
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[j].x, v[j].y);
            o[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x) + row * a.ldx + c);
          d[0] = make_uint4(o[0], o[1], o[2], o[3]);
          d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (c + j >= H) continue;
          const float f = j % 2 ? v[j / 2].y : v[j / 2].x;
          if (DT) static_cast<float*>(a.x)[row * a.ldx + c + j] = f;
          else static_cast<__nv_bfloat16*>(a.x)[row * a.ldx + c + j] = __float2bfloat16_rn(f);
        }
      }
    }
  }
}

// Any layout: a block a warp, `wpr` warps a row (a power of two up to 8).
template <int DT>
__global__ void __launch_bounds__(CT) checkpoint_pack_any_kernel(CheckpointArgs a, int wpr) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = CT / 32 / wpr;
  const int H = (int)a.H, nb = (H + kCkBlock - 1) / kCkBlock;
  bool bad = false;
  for (int64_t row = (int64_t)blockIdx.x * per + warp / wpr; row < a.T; row += (int64_t)gridDim.x * per) {
    for (int b0 = (warp & (wpr - 1)) * BLOCKS; b0 < nb; b0 += wpr * BLOCKS) {
      float x[BLOCKS];
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        const int c = (b0 + k) * kCkBlock + lane;
        x[k] = c < H ? ld_elem(a.x, DT, row * a.ldx + c) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        const int c = (b0 + k) * kCkBlock + lane;
        const uint32_t byte = ck_scale_byte(__reduce_max_sync(0xFFFFFFFFu, abs_bits(x[k])));
        bad = bad || byte == 255u;
        if (c < H) a.ck.codes[row * a.ck.ldc + c] = (int8_t)ck_code(x[k], byte);
        if (lane == 0 && c < H) a.ck.scales[row * a.ck.lds + b0 + k] = (uint8_t)byte;
      }
    }
  }
  if (bad && lane == 0 && a.status) atomicOr(a.status, RLK_STATUS_NONFINITE);
}

template <int DT>
__global__ void __launch_bounds__(CT) checkpoint_unpack_any_kernel(CheckpointArgs a, int wpr) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = CT / 32 / wpr;
  const int H = (int)a.H, nb = (H + kCkBlock - 1) / kCkBlock;
  for (int64_t row = (int64_t)blockIdx.x * per + warp / wpr; row < a.T; row += (int64_t)gridDim.x * per) {
    for (int b0 = (warp & (wpr - 1)) * BLOCKS; b0 < nb; b0 += wpr * BLOCKS) {
      float v[BLOCKS];
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        const int c = (b0 + k) * kCkBlock + lane;
        v[k] = c < H ? __fmul_rn((float)a.ck.codes[row * a.ck.ldc + c], ck_step(a.ck.scales[row * a.ck.lds + b0 + k])) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        const int c = (b0 + k) * kCkBlock + lane;
        if (c >= H) continue;
        if (DT) static_cast<float*>(a.x)[row * a.ldx + c] = v[k];
        else static_cast<__nv_bfloat16*>(a.x)[row * a.ldx + c] = __float2bfloat16_rn(v[k]);
      }
    }
  }
}

// Whether every row of x starts on a 16-byte boundary.
bool rows16(const CheckpointArgs& a) {
  return reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % (a.dtype ? 4 : 8) == 0;
}
int pow2_up_to(int64_t want, int most) {
  int n = 1;
  while (n < most && n < want) n *= 2;
  return n;
}

cudaError_t launch(const CheckpointArgs& a, void (*vec)(CheckpointArgs, int), int vec_rows,
                   void (*any)(CheckpointArgs, int), cudaStream_t stream) {
  if (rows16(a)) {
    const int n = a.H <= 32 ? 2 : pow2_up_to((a.H + 15) / 16, CT);   // whole pairs
    const int64_t rows = CT / n * vec_rows, grid = (a.T + rows - 1) / rows;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    vec<<<(unsigned)grid, CT, 0, stream>>>(a, n);
  } else {
    const int wpr = pow2_up_to((a.H + kCkBlock * BLOCKS - 1) / (kCkBlock * BLOCKS), CT / 32);
    const int64_t rows = CT / 32 / wpr, want = (a.T + rows - 1) / rows, cap = (int64_t)sm_count() * 64;
    any<<<(unsigned)(want < cap ? want : cap), CT, 0, stream>>>(a, wpr);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CheckpointArgs& a, cudaStream_t stream) {
  return a.dtype ? launch(a, checkpoint_pack_kernel<1>, pack_rows(1), checkpoint_pack_any_kernel<1>, stream)
                 : launch(a, checkpoint_pack_kernel<0>, pack_rows(0), checkpoint_pack_any_kernel<0>, stream);
}

cudaError_t launch_checkpoint_unpack(const CheckpointArgs& a, cudaStream_t stream) {
  return a.dtype ? launch(a, checkpoint_unpack_kernel<1>, UNPACK_ROWS, checkpoint_unpack_any_kernel<1>, stream)
                 : launch(a, checkpoint_unpack_kernel<0>, UNPACK_ROWS, checkpoint_unpack_any_kernel<0>, stream);
}

}  // namespace rlk
