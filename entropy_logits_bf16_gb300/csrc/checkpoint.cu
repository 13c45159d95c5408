// rlk_checkpoint_pack / rlk_checkpoint_unpack: an activation as 8-bit codes
// with a power-of-two step per 32 columns, and back.

#include "checkpoint.cuh"
#include "internal.h"
#include "rlk.h"

namespace rlk {
namespace {

constexpr int CT = 256;

__device__ __forceinline__ float ld_elem(const void* p, int dtype, int64_t i) {
  return dtype ? static_cast<const float*>(p)[i]
               : bf16_val(static_cast<const uint16_t*>(p)[i]);
}

// One warp per block of 32 columns, any layout.
__global__ void __launch_bounds__(CT) checkpoint_pack_kernel(CheckpointArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.H + kCkBlock - 1) / kCkBlock;
  const int64_t n = a.T * nb;
  bool bad = false;
  for (int64_t u = (int64_t)blockIdx.x * (CT / 32) + (threadIdx.x >> 5); u < n;
       u += (int64_t)gridDim.x * (CT / 32)) {
    const int64_t t = u / nb, b = u - t * nb, c = b * kCkBlock + lane;
    const float x = c < a.H ? ld_elem(a.x, a.dtype, t * a.ldx + c) : 0.f;
    const uint32_t byte = ck_scale_byte(__reduce_max_sync(0xFFFFFFFFu, abs_bits(x)));
    bad = bad || byte == 255u;
    if (c < a.H) a.ck.codes[t * a.ck.ldc + c] = (int8_t)ck_code(x, byte);
    if (lane == 0) a.ck.scales[t * a.ck.lds + b] = (uint8_t)byte;
  }
  if (bad && lane == 0 && a.status) atomicOr(a.status, RLK_STATUS_NONFINITE);
}

__global__ void __launch_bounds__(CT) checkpoint_unpack_kernel(CheckpointArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.H + kCkBlock - 1) / kCkBlock;
  const int64_t n = a.T * nb;
  for (int64_t u = (int64_t)blockIdx.x * (CT / 32) + (threadIdx.x >> 5); u < n;
       u += (int64_t)gridDim.x * (CT / 32)) {
    const int64_t t = u / nb, b = u - t * nb, c = b * kCkBlock + lane;
    if (c >= a.H) continue;
    const float v = __fmul_rn((float)a.ck.codes[t * a.ck.ldc + c], ck_step(a.ck.scales[t * a.ck.lds + b]));
    if (a.dtype) static_cast<float*>(a.x)[t * a.ldx + c] = v;
    else static_cast<__nv_bfloat16*>(a.x)[t * a.ldx + c] = __float2bfloat16_rn(v);
  }
}

unsigned grid_for(int64_t units) {
  const int64_t want = (units + CT / 32 - 1) / (CT / 32), cap = (int64_t)sm_count() * 8;
  return (unsigned)(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CheckpointArgs& a, cudaStream_t stream) {
  const int64_t units = a.T * ((a.H + kCkBlock - 1) / kCkBlock);
  checkpoint_pack_kernel<<<grid_for(units), CT, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const CheckpointArgs& a, cudaStream_t stream) {
  const int64_t units = a.T * ((a.H + kCkBlock - 1) / kCkBlock);
  checkpoint_unpack_kernel<<<grid_for(units), CT, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rlk
