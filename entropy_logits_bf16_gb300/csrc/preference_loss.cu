// rlk_preference_loss kernels: paired preference loss over packed
// log-probabilities, with its gradient.
//
//   D_s = sum_t m_t (logp_t - ref_t) [/ sum_t m_t],  r_s = beta D_s,
//   h_i = r_2i - r_2i+1 - margin,  L = (1 / P) sum_i l(h_i),
//   dL/dlogp_t = +-l'(h_i) beta m_t / P [/ sum m].
//
// 13 bytes a token and a handful of flops: the floor of an ordinary batch
// (half a million tokens) is about 1 us, so the time is that of launches and
// of the dependent loads (offsets, then tokens).  Two launches, the second a
// programmatic dependent of the first:
//  1. pref_sum_kernel: a CTA sums a sequence.  It is cut into segments of kSeg
//     tokens from its own start; a warp sums a segment (each lane its tokens in
//     order, then a tree, as double-floats) and one thread adds the segments in
//     order.  The cut depends on the sequence alone, so its sum's bits do too,
//     whatever the number of warps (one for thousands of sequences, up to 32 for
//     a few long ones: about 24 warps an SM in all).  A few more CTAs check
//     the offsets and leave a flag each.
//  2. pref_grad_kernel: a CTA reads its pair's two sums, forms l'(h) and writes the
//     gradient of up to 2048 tokens; one more CTA sums the pairs' losses and
//     statistics in a fixed order.
// No atomics, and no CTA waits for another of the same launch.
// Measured: 2048 pairs, 4.7 M tokens with reference and mask, 25.5 us in all (sum 17,
// gradient 17 when timed alone); 4 pairs of up to 256 tokens 5 us, the time of two
// launches.

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "rlk.h"

namespace rlk {
namespace {

constexpr int kSeg = 512;            // tokens of one segment: 16 a lane
constexpr int kSumWarps = 32;        // warps that sum a sequence, at most
constexpr int kChecks = 32;          // CTAs that check the offsets, at most
constexpr int PT = 128;              // threads of a CTA of the gradient
constexpr int kGradToks = 16 * PT;   // tokens whose gradient a CTA writes at a time

// Sequence s's tokens, clamped to the n_tok packed ones; false: offsets that
// decrease or leave them.
__device__ __forceinline__ bool seq_range(const PrefArgs& a, int64_t s, int64_t& t0, int64_t& t1) {
  t0 = a.seq_offsets[s];
  t1 = a.seq_offsets[s + 1];
  const bool ok = t0 >= 0 && t1 >= t0 && t1 <= a.n_tok;
  t0 = t0 < 0 ? 0 : (t0 > a.n_tok ? a.n_tok : t0);
  t1 = t1 < t0 ? t0 : (t1 > a.n_tok ? a.n_tok : t1);
  return ok;
}

__device__ __forceinline__ DF warp_sum_df(DF v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = df_add(v, DF{shfl_down(v.hi, o), shfl_down(v.lo, o)});
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, shfl_down(v, o));
  return v;
}
// The double-float sum, or the plain one where that is no number (the error
// terms are inf - inf there).
__device__ __forceinline__ float sum_value(DF v, float plain) {
  return isfinite(plain) ? __fadd_rn(v.hi, v.lo) : plain;
}

__global__ void __launch_bounds__(32 * kSumWarps) pref_sum_kernel(PrefArgs a) {
  pdl_trigger();
  pdl_wait();   // the log-probabilities may come from the kernel before
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if ((int)blockIdx.x < a.checks) {   // this share of the offsets valid?
    const int64_t n = 2 * (int64_t)a.n_pairs;
    const int64_t s0 = n * blockIdx.x / a.checks, s1 = n * (blockIdx.x + 1) / a.checks;
    bool bad = false;
    for (int64_t s = s0 + tid; s < s1; s += blockDim.x) {
      int64_t t0, t1;
      bad = !seq_range(a, s, t0, t1) || bad;
    }
    const int any = __syncthreads_or(bad);
    if (tid == 0) a.flags[blockIdx.x] = any ? 1u : 0u;
    return;
  }
  __shared__ DF s_sum[kSumWarps];
  __shared__ float s_plain[kSumWarps];
  __shared__ int s_cnt[kSumWarps];
  const int64_t s = (int64_t)blockIdx.x - a.checks;
  int64_t t0, t1;
  seq_range(a, s, t0, t1);
  const int nseg = (int)((t1 - t0 + kSeg - 1) / kSeg);
  DF total{0.f, 0.f};
  float total_plain = 0.f;
  int64_t count = 0;
  for (int j0 = 0; j0 < nseg; j0 += nw) {
    const int64_t b = t0 + (int64_t)(j0 + warp) * kSeg;
    const int left = (int)(t1 - b < kSeg ? t1 - b : kSeg);   // may be negative: no such segment
    constexpr int U = kSeg / 32;
    float x[U], r[U];
    uint32_t on[U];   // the loads of all 16 tokens are on their way together
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int t = k * 32 + lane;
      const bool in = t < left;
      x[k] = in ? a.logp[b + t] : 0.f;
      r[k] = in & (a.logp_ref != nullptr) ? a.logp_ref[b + t] : 0.f;
      on[k] = in & (a.mask != nullptr) ? a.mask[b + t] : (in ? 1u : 0u);
    }
    DF acc{0.f, 0.f};
    int cnt = 0;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float v = on[k] ? __fsub_rn(x[k], r[k]) : 0.f;
      float e;
      two_sum(acc.hi, v, acc.hi, e);   // the errors are added beside the chain of the sums
      acc.lo = __fadd_rn(acc.lo, e);
      cnt += on[k] ? 1 : 0;
    }
    float plain = acc.hi;   // the sum without its errors: no number where that is right
    acc = df_add(acc, DF{0.f, 0.f});
    acc = warp_sum_df(acc);
    plain = warp_sum(plain);
    cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
    if (lane == 0) {
      s_sum[warp] = acc;
      s_plain[warp] = plain;
      s_cnt[warp] = cnt;
    }
    __syncthreads();
    if (tid == 0) {
      const int n = nseg - j0 < nw ? nseg - j0 : nw;
      for (int w = 0; w < n; ++w) {
        total = df_add(total, s_sum[w]);
        total_plain = __fadd_rn(total_plain, s_plain[w]);
        count += s_cnt[w];
      }
    }
    __syncthreads();
  }
  if (tid == 0) a.sums[s] = make_float2(sum_value(total, total_plain), (float)count);
}

// Whether some offsets are invalid.
__device__ __forceinline__ bool bad_offsets(const PrefArgs& a) {
  const int lane = threadIdx.x & 31;
  return __any_sync(0xFFFFFFFFu, lane < a.checks && a.flags[lane] != 0u);
}

// A sequence's reward.
__device__ __forceinline__ float reward_of(const PrefArgs& a, float sum, float count) {
  return __fmul_rn(a.beta, a.mean && count > 0.f ? __fdiv_rn(sum, count) : sum);
}

// ln(1 + e^v)
__device__ __forceinline__ float softplus(float v) {
  return __fadd_rn(fmaxf(v, 0.f), log1pf(expf(-fabsf(v))));
}
__device__ __forceinline__ float sigmoid(float v) { return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-v))); }

// l(h) and l'(h)
__device__ __forceinline__ float pref_value(const PrefArgs& a, float h) {
  if (a.type == RLK_PREF_HINGE) return h != h ? h : fmaxf(__fsub_rn(1.f, h), 0.f);
  if (a.type == RLK_PREF_IPO) {
    const float d = __fdiv_rn(__fsub_rn(h, 0.5f), a.beta);
    return __fmul_rn(d, d);
  }
  if (a.smoothing == 0.f) return h != h ? h : softplus(-h);
  return __fmaf_rn(__fsub_rn(1.f, a.smoothing), softplus(-h), __fmul_rn(a.smoothing, softplus(h)));
}
__device__ __forceinline__ float pref_slope(const PrefArgs& a, float h) {
  if (a.type == RLK_PREF_HINGE) return h != h ? h : (h < 1.f ? -1.f : 0.f);
  if (a.type == RLK_PREF_IPO)
    return __fdiv_rn(__fmul_rn(2.f, __fdiv_rn(__fsub_rn(h, 0.5f), a.beta)), a.beta);
  const float down = __fmul_rn(__fsub_rn(1.f, a.smoothing), sigmoid(-h));
  return __fsub_rn(__fmul_rn(a.smoothing, sigmoid(h)), down);
}

__global__ void __launch_bounds__(PT) pref_grad_kernel(PrefArgs a) {
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float4* pairs = reinterpret_cast<const float4*>(a.sums);   // (sum, count) of both sequences
  if (blockIdx.x == 0) {   // the loss and the statistics; the gradient of a batch without pairs
    pdl_wait();   // the sequences' sums
    const bool bad = bad_offsets(a);
    if (a.n_pairs == 0 && a.out_grad)
      for (int64_t t = tid; t < a.n_tok; t += PT) a.out_grad[t] = 0.f;
    __shared__ DF s_red[PT / 32][RLK_PREF_NSTATS];
    __shared__ float s_plain[PT / 32][RLK_PREF_NSTATS];
    DF acc[RLK_PREF_NSTATS];
    float plain[RLK_PREF_NSTATS];
#pragma unroll
    for (int k = 0; k < RLK_PREF_NSTATS; ++k) {
      acc[k] = DF{0.f, 0.f};
      plain[k] = 0.f;
    }
    for (int64_t i0 = tid; i0 < a.n_pairs && !bad; i0 += 8 * PT) {
      float4 p[8];   // on their way together
#pragma unroll
      for (int u = 0; u < 8; ++u) p[u] = i0 + u * PT < a.n_pairs ? pairs[i0 + u * PT] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (!(p[u].y > 0.f && p[u].w > 0.f)) continue;
        const float c = reward_of(a, p[u].x, p[u].y), r = reward_of(a, p[u].z, p[u].w);
        const float diff = __fsub_rn(c, r);
        const float v[RLK_PREF_NSTATS] = {pref_value(a, __fsub_rn(diff, a.margin)), 1.f, diff > 0.f ? 1.f : 0.f, diff, c, r};
#pragma unroll
        for (int k = 0; k < RLK_PREF_NSTATS; ++k) {
          acc[k] = df_add_f(acc[k], v[k]);
          plain[k] = __fadd_rn(plain[k], v[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < RLK_PREF_NSTATS; ++k) {
      acc[k] = warp_sum_df(acc[k]);
      plain[k] = warp_sum(plain[k]);
      if (lane == 0) {
        s_red[warp][k] = acc[k];
        s_plain[warp][k] = plain[k];
      }
    }
    __syncthreads();
    if (tid != 0) return;
    float v[RLK_PREF_NSTATS];
#pragma unroll
    for (int k = 0; k < RLK_PREF_NSTATS; ++k) {
      for (int w = 1; w < PT / 32; ++w) {
        acc[k] = df_add(acc[k], s_red[w][k]);
        plain[k] = __fadd_rn(plain[k], s_plain[w][k]);
      }
      v[k] = bad ? NAN : sum_value(acc[k], plain[k]);
    }
    const float L = a.n_pairs > 0 ? __fdiv_rn(v[RLK_PREF_STAT_LOSS], (float)a.n_pairs) : 0.f;
    *a.out_loss = L;
    if (a.out_stats) {
      const float n = v[RLK_PREF_STAT_PAIRS], d = n > 0.f ? n : (bad ? NAN : 1.f);
      a.out_stats[RLK_PREF_STAT_LOSS] = L;
      a.out_stats[RLK_PREF_STAT_PAIRS] = n;
      for (int k = RLK_PREF_STAT_ACCURACY; k < RLK_PREF_NSTATS; ++k) a.out_stats[k] = __fdiv_rn(v[k], d);
    }
    return;
  }
  const int64_t unit = (int64_t)blockIdx.x - 1;
  const int64_t s = unit / a.split, j0 = unit - s * a.split;
  pdl_wait();   // the sequences' sums (and, through that kernel, the caller's offsets and mask)
  int64_t t0, t1;
  seq_range(a, s, t0, t1);
  const float4 p = pairs[s / 2];
  const bool bad = bad_offsets(a);
  if (bad) {   // offsets that do not describe the batch: everything is NaN
    const int64_t step = ((int64_t)gridDim.x - 1) * PT;
    for (int64_t i = unit * PT + tid; i < a.n_tok && a.out_grad; i += step) a.out_grad[i] = NAN;
    for (int64_t i = unit * PT + tid; i < 2 * (int64_t)a.n_pairs && a.out_reward; i += step) a.out_reward[i] = NAN;
    return;
  }
  const float c = reward_of(a, p.x, p.y), r = reward_of(a, p.z, p.w);
  if (j0 == 0 && tid == 0 && a.out_reward) a.out_reward[s] = (s & 1) ? r : c;
  if (!a.out_grad) return;
  float g = 0.f;
  if (p.y > 0.f && p.w > 0.f) {
    g = pref_slope(a, __fsub_rn(__fsub_rn(c, r), a.margin));
    g = __fdiv_rn(__fmul_rn((s & 1) ? -g : g, a.beta), (float)a.n_pairs);
    if (a.mean) g = __fdiv_rn(g, (s & 1) ? p.w : p.y);
  }
  for (int64_t b = t0 + j0 * kGradToks; b < t1; b += (int64_t)a.split * kGradToks) {
    const int left = (int)(t1 - b < kGradToks ? t1 - b : kGradToks);
    // four tokens a thread at a time: their mask bytes are on their way together
    for (int k0 = 0; k0 < left; k0 += 4 * PT) {
      uint32_t on[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = k0 + k * PT + tid;
        on[k] = (t < left) & (a.mask != nullptr) ? a.mask[b + t] : 1u;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = k0 + k * PT + tid;
        if (t < left) a.out_grad[b + t] = on[k] ? g : 0.f;
      }
    }
  }
  // tokens before the first sequence and after the last
  if (j0 == 0 && s == 0)
    for (int64_t t = tid; t < t0; t += PT) a.out_grad[t] = 0.f;
  if (j0 == 0 && s == 2 * (int64_t)a.n_pairs - 1)
    for (int64_t t = t1 + tid; t < a.n_tok; t += PT) a.out_grad[t] = 0.f;
}

}  // namespace

size_t pref_workspace_bytes(int64_t n_tok, int64_t n_pairs) {
  (void)n_tok;
  return (kChecks * sizeof(uint32_t) + (size_t)(2 * n_pairs) * sizeof(float2) + 255) & ~(size_t)255;
}

cudaError_t launch_preference_loss(PrefArgs a, void* workspace, cudaStream_t stream) {
  a.flags = static_cast<uint32_t*>(workspace);
  a.sums = reinterpret_cast<float2*>(a.flags + kChecks);
  const int64_t n_seq = 2 * (int64_t)a.n_pairs, mean_len = n_seq > 0 ? a.n_tok / n_seq : 0;
  // warps of a sequence: what its mean length takes at once, if the SMs have room
  const int64_t room = (int64_t)sm_count() * 24;
  int warps = 1;
  while (warps < kSumWarps && warps * kSeg < mean_len && n_seq * warps * 2 <= room) warps *= 2;
  a.checks = (int)(n_seq / 64 + 1 < kChecks ? n_seq / 64 + 1 : kChecks);
  // CTAs that write a sequence's gradient: what its mean length takes, and half as much for uneven ones
  int64_t split = (mean_len + mean_len / 2 + kGradToks - 1) / kGradToks;
  if (split < 1) split = 1;
  if (split > 64) split = 64;
  a.split = (int)split;
  cudaError_t e = launch_after(pref_sum_kernel, dim3((unsigned)(n_seq + a.checks)), dim3(32 * warps), 0, stream, a);
  if (e == cudaSuccess)
    e = launch_after(pref_grad_kernel, dim3((unsigned)(n_seq * split + 1)), dim3(PT), 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rlk
