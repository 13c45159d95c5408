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
//  1. pref_sum_kernel: a sequence is cut into segments of kSeg tokens from its
//     own start; a CTA sums a segment (each thread its tokens in order, then a
//     tree, as double-floats) into the segment's slot of the workspace.  The
//     cut depends on the sequence alone, so its sum's bits do too.  One more
//     CTA checks all offsets and leaves a flag.
//  2. pref_grad_kernel: every CTA joins its pair's slots in order (a few loads),
//     forms l'(h) and writes its segments' gradients; one more CTA sums the
//     pairs' losses and statistics in a fixed order.
// No atomics, and no CTA waits for another of the same launch.

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "rlk.h"

namespace rlk {
namespace {

constexpr int PT = 256;
constexpr int PWARP = PT / 32;
constexpr int kSeg = 8 * PT;   // tokens of one segment

// Slot of segment j of sequence s: unique for valid offsets, since a sequence
// that starts at t0 and has n tokens takes ceil(n / kSeg) slots from
// s + t0 / kSeg on and the next one starts at s + 1 + (t0 + n) / kSeg.  Clamped
// ranges keep it below 2 n_pairs + n_tok / kSeg + 1 whatever the offsets.
__device__ __forceinline__ int64_t slot_of(int64_t s, int64_t t0, int64_t j) {
  return s + t0 / kSeg + j;
}

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

// A non-finite sum keeps its value: the error terms of the double-float sum
// are inf - inf there.
__device__ __forceinline__ float df_value(DF v) { return isfinite(v.hi) ? __fadd_rn(v.hi, v.lo) : v.hi; }

__global__ void __launch_bounds__(PT) pref_sum_kernel(PrefArgs a) {
  pdl_trigger();
  pdl_wait();   // the log-probabilities may come from the kernel before
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0) {   // all offsets valid?
    bool bad = false;
    for (int64_t s = tid; s < 2 * (int64_t)a.n_pairs; s += PT) {
      int64_t t0, t1;
      bad = !seq_range(a, s, t0, t1) || bad;
    }
    const int any = __syncthreads_or(bad);
    if (tid == 0) *a.flag = any ? 1u : 0u;
    return;
  }
  __shared__ DF s_sum[PWARP];
  __shared__ int s_cnt[PWARP];
  const int64_t unit = (int64_t)blockIdx.x - 1;
  const int64_t s = unit / a.split;
  int64_t t0, t1;
  seq_range(a, s, t0, t1);
  for (int64_t j = unit - s * a.split; j * kSeg < t1 - t0; j += a.split) {
    const int64_t b = t0 + j * kSeg;
    const int64_t e = t1 < b + kSeg ? t1 : b + kSeg;
    DF acc{0.f, 0.f};
    float plain = 0.f;   // carries infinities and NaN
    int cnt = 0;
#pragma unroll
    for (int k = 0; k < kSeg / PT; ++k) {
      const int64_t t = b + k * PT + tid;
      if (t < e && (!a.mask || a.mask[t])) {
        const float d = a.logp_ref ? __fsub_rn(a.logp[t], a.logp_ref[t]) : a.logp[t];
        acc = df_add_f(acc, d);
        plain = __fadd_rn(plain, d);
        ++cnt;
      }
    }
    if (!isfinite(plain)) acc = DF{plain, 0.f};
    acc = warp_sum_df(acc);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) plain = __fadd_rn(plain, shfl_down(plain, o));
    cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
    if (lane == 0) {
      s_sum[warp] = isfinite(plain) ? acc : DF{plain, 0.f};
      s_cnt[warp] = cnt;
    }
    __syncthreads();
    if (tid == 0) {
      DF v = s_sum[0];
      float p = s_sum[0].hi;
      int n = s_cnt[0];
      for (int w = 1; w < PWARP; ++w) {
        v = df_add(v, s_sum[w]);
        p = __fadd_rn(p, s_sum[w].hi);
        n += s_cnt[w];
      }
      if (!isfinite(p)) v = DF{p, 0.f};
      a.slots[slot_of(s, t0, j)] = make_float4(v.hi, v.lo, __int_as_float(n), 0.f);
    }
    __syncthreads();
  }
}

// A sequence's reward and token count, its segments joined in order.
struct SeqSum {
  float reward;
  float count;
};
__device__ __forceinline__ SeqSum join_sequence(const PrefArgs& a, int64_t s) {
  int64_t t0, t1;
  seq_range(a, s, t0, t1);
  const int64_t nseg = (t1 - t0 + kSeg - 1) / kSeg, first = slot_of(s, t0, 0);
  DF sum{0.f, 0.f};
  float plain = 0.f;
  int64_t n = 0;
  for (int64_t j = 0; j < nseg; ++j) {
    const float4 p = a.slots[first + j];
    sum = df_add(sum, DF{p.x, p.y});
    plain = __fadd_rn(plain, p.x);
    n += __float_as_int(p.z);
  }
  SeqSum r;
  r.count = (float)n;
  float d = isfinite(plain) ? __fadd_rn(sum.hi, sum.lo) : plain;
  if (a.mean && n > 0) d = __fdiv_rn(d, r.count);
  r.reward = __fmul_rn(a.beta, d);
  return r;
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
  pdl_wait();   // the segments' sums
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool bad = *a.flag != 0u;
  if (blockIdx.x == 0) {   // the loss and the statistics; the gradient of a batch without pairs
    if (a.n_pairs == 0 && a.out_grad)
      for (int64_t t = tid; t < a.n_tok; t += PT) a.out_grad[t] = 0.f;
    __shared__ DF s_red[PWARP][RLK_PREF_NSTATS];
    DF acc[RLK_PREF_NSTATS];
#pragma unroll
    for (int k = 0; k < RLK_PREF_NSTATS; ++k) acc[k] = DF{0.f, 0.f};
    float plain = 0.f;
    for (int64_t i = tid; i < a.n_pairs && !bad; i += PT) {
      const SeqSum c = join_sequence(a, 2 * i), r = join_sequence(a, 2 * i + 1);
      if (!(c.count > 0.f && r.count > 0.f)) continue;
      const float diff = __fsub_rn(c.reward, r.reward);
      const float l = pref_value(a, __fsub_rn(diff, a.margin));
      plain = __fadd_rn(plain, l);
      acc[RLK_PREF_STAT_LOSS] = df_add_f(acc[RLK_PREF_STAT_LOSS], l);
      acc[RLK_PREF_STAT_PAIRS] = df_add_f(acc[RLK_PREF_STAT_PAIRS], 1.f);
      acc[RLK_PREF_STAT_ACCURACY] = df_add_f(acc[RLK_PREF_STAT_ACCURACY], diff > 0.f ? 1.f : 0.f);
      acc[RLK_PREF_STAT_MARGIN] = df_add_f(acc[RLK_PREF_STAT_MARGIN], diff);
      acc[RLK_PREF_STAT_CHOSEN] = df_add_f(acc[RLK_PREF_STAT_CHOSEN], c.reward);
      acc[RLK_PREF_STAT_REJECTED] = df_add_f(acc[RLK_PREF_STAT_REJECTED], r.reward);
    }
#pragma unroll
    for (int k = 0; k < RLK_PREF_NSTATS; ++k) acc[k] = warp_sum_df(acc[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) plain = __fadd_rn(plain, shfl_down(plain, o));
    if (lane == 0) {
      if (!isfinite(plain)) acc[RLK_PREF_STAT_LOSS] = DF{plain, 0.f};
#pragma unroll
      for (int k = 0; k < RLK_PREF_NSTATS; ++k) s_red[warp][k] = acc[k];
    }
    __syncthreads();
    if (tid != 0) return;
    float v[RLK_PREF_NSTATS];
#pragma unroll
    for (int k = 0; k < RLK_PREF_NSTATS; ++k) {
      DF t = s_red[0][k];
      float p = t.hi;
      for (int w = 1; w < PWARP; ++w) {
        t = df_add(t, s_red[w][k]);
        p = __fadd_rn(p, s_red[w][k].hi);
      }
      v[k] = bad ? NAN : (isfinite(p) ? df_value(t) : p);
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
  if (bad) {   // offsets that do not describe the batch: everything is NaN
    const int64_t step = ((int64_t)gridDim.x - 1) * PT;
    for (int64_t i = unit * PT + tid; i < a.n_tok && a.out_grad; i += step) a.out_grad[i] = NAN;
    for (int64_t i = unit * PT + tid; i < 2 * (int64_t)a.n_pairs && a.out_reward; i += step) a.out_reward[i] = NAN;
    return;
  }
  const int64_t s = unit / a.split, j0 = unit - s * a.split;
  const SeqSum c = join_sequence(a, s & ~(int64_t)1), r = join_sequence(a, s | 1);
  const float own_reward = (s & 1) ? r.reward : c.reward, own_count = (s & 1) ? r.count : c.count;
  if (j0 == 0 && tid == 0 && a.out_reward) a.out_reward[s] = own_reward;
  if (!a.out_grad) return;
  float g = 0.f;
  if (c.count > 0.f && r.count > 0.f) {
    g = pref_slope(a, __fsub_rn(__fsub_rn(c.reward, r.reward), a.margin));
    g = __fdiv_rn(__fmul_rn((s & 1) ? -g : g, a.beta), (float)a.n_pairs);
    if (a.mean) g = __fdiv_rn(g, own_count);
  }
  int64_t t0, t1;
  seq_range(a, s, t0, t1);
  for (int64_t j = j0; j * kSeg < t1 - t0; j += a.split) {
    const int64_t b = t0 + j * kSeg;
#pragma unroll
    for (int k = 0; k < kSeg / PT; ++k) {
      const int64_t t = b + k * PT + tid;
      if (t < t1) a.out_grad[t] = (!a.mask || a.mask[t]) ? g : 0.f;
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
  const size_t slots = (size_t)(2 * n_pairs + n_tok / kSeg + 1);
  return (slots * sizeof(float4) + 16 + 255) & ~(size_t)255;
}

cudaError_t launch_preference_loss(PrefArgs a, void* workspace, cudaStream_t stream) {
  a.flag = static_cast<uint32_t*>(workspace);
  a.slots = reinterpret_cast<float4*>(static_cast<char*>(workspace) + 16);
  // CTAs a sequence: its mean number of segments, twice over for uneven lengths
  const int64_t n_seq = 2 * (int64_t)a.n_pairs;
  int64_t split = n_seq > 0 ? (2 * a.n_tok + n_seq * kSeg - 1) / (n_seq * kSeg) : 1;
  if (split < 1) split = 1;
  if (split > 64) split = 64;
  a.split = (int)split;
  const dim3 grid((unsigned)(n_seq * split + 1));
  cudaError_t e = launch_after(pref_sum_kernel, grid, dim3(PT), 0, stream, a);
  if (e == cudaSuccess) e = launch_after(pref_grad_kernel, grid, dim3(PT), 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rlk
