// rlk_token_logprobs_fwd / rlk_token_logprobs_bwd: log-probabilities of any number of given
// tokens a row, the entropy, and the row's top alternatives, over the whole vocabulary.
//
//   forward   M = max z,  S = sum e^((z - M) / T),  logprob_c = (z_c - M) / T - ln S,
//             H = ln S - (1 / S) sum e^d d,  d = (z - M) / T;
//             the K largest logits, equal ones by the lower index
//   backward  dz_i = (1 / T) [ sum of the gradients of what names i - p_i (G + g_H (ln p_i + H)) ],
//             G the sum of all of them, p_i = e^((z_i - M) / T) / S
//
// Forward: one read of the row.  A row is cut into groups of 16 bytes by index, 32 groups a
// chunk; chunk c belongs to virtual warp c mod 32, whose lanes keep a running reference, S and
// sum w d each and are joined in a fixed order.  A row is worked on by a cluster of 1, 2 or 4 CTAs
// (few rows: more of them, so that every SM reads), which only changes which CTA holds which
// virtual warps, so a row's bits do not depend on the batch.  Rows that start off 16-byte
// boundaries are read as aligned words and shifted, into the same groups.
// The alternatives need no second pass: each lane keeps the largest logit of each of its
// virtual warps (a unit: V / 1024 logits).  The K-th largest of the threads' maxima is a lower bound
// of the K-th largest logit, nearly tight for logits in any order that is not sorted; only
// the units that reach it are read again (about K of 1024), and what is at or above it is
// sorted by (logit, index).  Rows that put too many logits there (long ties) take a bisection
// over the logits' order instead, with one read of the row a step.
//
// Measured: 4096 x 151936 bf16 197 us (6.3 TB/s, 0.93 of the copy rate) without alternatives, 227 with
// 20: what follows the pass takes about a fifth of a row's time on its CTA (a third of that the second
// look, which waits for memory), and the others of the SM do not quite fill in.  (A sketch of all
// groups' maxima in shared memory made the second look small, and took the L1 cache that the loads
// pass through: 262 us.)  777 x 50021 fp32, rows off 16 bytes, 50 alternatives 50 us (3.1 TB/s): 5.1
// rows an SM, the last of them alone.  Backward, 4096 x 151936 bf16 with 64 tokens a row 383 to 391 us
// (6.4 TB/s); 777 x 50021 fp32 55 us, to bf16 43 (floors 46 and 34), to rows that start elsewhere on 16 bytes
// than the logits' 175 (one element a thread).
#include <float.h>
#include <math.h>

#include <atomic>

#include "internal.h"
#include "rlk.h"
#include "tensor_core.cuh"

namespace rlk {
namespace {

constexpr int MAX_VW = 32;        // most virtual warps of a row
constexpr int MAX_TOP = RLK_MAX_ALTERNATIVES;
// Rows of up to kShortRow bytes are cut into 16 virtual warps (half the threads a row); few rows
// of kLongRow and more are shared by CTAs.
constexpr int64_t kShortRow = 32768, kLongRow = 131072;
constexpr int CAP = 1024;         // candidates that are sorted
constexpr int MAX_UNITS = 512;    // units that are read again
constexpr float CLAMP = -200.f;   // 2^-200 is 0 in fp32, and 0 x -200 is 0 (0 x -inf would be NaN)

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Barriers of the NT threads that work on a row (another warp may fetch for them).
template <int NT>
__device__ __forceinline__ void sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
}
template <int NT>
__device__ __forceinline__ int sync_count(bool p) {
  int n;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n bar.red.popc.u32 %0, 1, %2, p;\n}\n" : "=r"(n) : "r"((int)p), "n"(NT) : "memory");
  return n;
}

// One 16-byte group of a row as floats; DT 0 bf16 (8 logits), 1 fp32 (4).
template <int DT>
struct Group;
template <>
struct Group<0> {
  static constexpr int E = 8;
  using elem = uint16_t;
  static __device__ __forceinline__ float value(uint16_t b) { return bf16_val(b); }
  static __device__ __forceinline__ void floats(const uint4& q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(u[j]);
      v[2 * j + 1] = bf16_hi(u[j]);
    }
  }
  static __device__ __forceinline__ float largest(const uint4& q) {   // NaN if one is
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(bf2(q.x), bf2(q.y)), __hmax2_nan(bf2(q.z), bf2(q.w)));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
    return max_nan(bf16_lo(w), bf16_hi(w));
  }
  static __device__ __forceinline__ uint32_t key(float v) { return okey16(__float_as_uint(v) >> 16); }
  static __device__ __forceinline__ float of_key(uint32_t k) { return bf16_val(okey16_inverse(k)); }
  static constexpr uint32_t kLowest = 0x0080u;   // key of the least finite value
  static constexpr int BITS = 16, SHIFT = 0;
};
template <>
struct Group<1> {
  static constexpr int E = 4;
  using elem = uint32_t;
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b); }
  static __device__ __forceinline__ void floats(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ float largest(const uint4& q) {
    return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                   max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
  static __device__ __forceinline__ uint32_t key(float v) { return okey32(__float_as_uint(v)); }
  static __device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(okey32_inverse(k)); }
  static constexpr uint32_t kLowest = 0x00800000u;
  static constexpr int BITS = 32, SHIFT = 16;   // the threads' maxima are compared by the upper 16 bits
};

// A row of logits, read in groups.  ALIGNED: it starts on a 16-byte boundary.
template <int DT, bool ALIGNED>
struct Row {
  using G = Group<DT>;
  using elem = typename G::elem;
  const elem* p;
  int V;
  uint32_t sh;   // bytes of the row's start past a 16-byte boundary

  __device__ __forceinline__ Row(const void* logits, int64_t row, int64_t ld, int64_t V_)
      : p(static_cast<const elem*>(logits) + row * ld), V((int)V_) {
    sh = ALIGNED ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  }
  __device__ __forceinline__ int groups() const { return (V + G::E - 1) / G::E; }
  // element by element, -inf past the end
  static __device__ __noinline__ uint4 edge(const elem* p, int V, int g) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (DT == 0) {
        const int e = g * 8 + 2 * j;
        const uint32_t lo = e < V ? (uint32_t)p[e] : 0xFF80u, hi = e + 1 < V ? (uint32_t)p[e + 1] : 0xFF80u;
        w[j] = lo | hi << 16;
      } else {
        const int e = g * 4 + j;
        w[j] = e < V ? (uint32_t)p[e] : 0xFF800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // INNER: a group after this one exists
  template <bool INNER = false>
  __device__ __forceinline__ uint4 load(int g) const {
    const int64_t at = (int64_t)g * 16, end = (int64_t)V * (int)sizeof(elem);
    if (ALIGNED) {
      if (!INNER && at + 16 > end) return edge(p, V, g);
      return __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + at));
    }
    // the two aligned words that the group lies in, where both are inside the row
    if ((g == 0 && sh) || at + 32 - (int)sh > end) return edge(p, V, g);
    const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + at - sh);
    return shifted(__ldg(a), __ldg(a + 1));
  }
  // The same from the copy of the row's whole aligned words, of which group g's first is at `at`.
  // INNER: not the first of the row, and two groups after this one exist
  template <bool INNER = false>
  __device__ __forceinline__ uint4 from_copy(const uint8_t* at, int g) const {
    if (!INNER && ((g == 0 && sh) || (int64_t)g * 16 + 32 - (int)sh > (int64_t)V * (int)sizeof(elem))) return edge(p, V, g);
    return shifted(*reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + 16));
  }
  __device__ __forceinline__ uint4 shifted(const uint4& x, const uint4& y) const {
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (sh & 8u) {
#pragma unroll
      for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
    }
    if (sh & 4u) {
#pragma unroll
      for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
    }
    const uint32_t b = (sh & 3u) * 8u;
    return make_uint4(__funnelshift_r(w[0], w[1], b), __funnelshift_r(w[1], w[2], b), __funnelshift_r(w[2], w[3], b),
                      __funnelshift_r(w[3], w[4], b));
  }
};

// A lane's share of a virtual warp: sums relative to a reference m that trails the largest
// logit seen (`top`) by at most `slack`, 16 powers of two, so that it hardly ever moves.
// (Temperatures over 3.8e36: less, so that z - m stays in fp32 from the first reference on, -FLT_MAX.)
struct Sums {
  float m = -FLT_MAX, top = -INFINITY;
  float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
};

template <int DT>
__device__ __forceinline__ void absorb(Sums& a, const uint4& q, float c, float slack) {
  using G = Group<DT>;
  const float gm = G::largest(q);
  a.top = max_nan(a.top, gm);
  if (!(gm <= __fadd_rn(a.m, slack))) {   // also a NaN, which the sums then carry on
    const float d = max_nan(__fmul_rn(__fsub_rn(a.m, gm), c), CLAMP), f = ex2(d);
    a.t = mul2(fma2(a.s, both(d), a.t), both(f));
    a.s = mul2(a.s, both(f));
    a.m = gm;
  }
  float v[G::E];
  G::floats(q, v);
#pragma unroll
  for (int j = 0; j < G::E; j += 2) {
    float2 d = mul2(add2(make_float2(v[j], v[j + 1]), both(-a.m)), both(c));
    d.x = max_nan(d.x, CLAMP);
    d.y = max_nan(d.y, CLAMP);
    const float2 w = make_float2(ex2(d.x), ex2(d.y));
    a.s = add2(a.s, w);
    a.t = fma2(w, d, a.t);
  }
}

struct Part {   // largest logit, sum 2^d, sum 2^d d with d = (z - top) c
  float top, s, t;
};
// Joins what the lanes hold, each with sums relative to its own m <= top.
__device__ __forceinline__ Part join(float m, float top, float s, float t, float c) {
  float M = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  // (no finite logit yet: M is -inf, m -FLT_MAX, both sums 0)
  const float d = M == -INFINITY ? 0.f : max_nan(__fmul_rn(__fsub_rn(m, M), c), CLAMP), f = ex2(d);
  t = __fmul_rn(__fmaf_rn(s, d, t), f);
  s = __fmul_rn(s, f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    t = __fadd_rn(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  }
  return Part{M, s, t};
}

struct Shared {
  Part part[MAX_VW];
  float M, lnS;
  int bad;
  int n_units, n_cand;
  uint32_t units[MAX_UNITS];
  unsigned long long cand[CAP];
  unsigned long long sorted[MAX_TOP];
  int n_sorted;
  int scan[32];
};

// key of (logit, index): larger is better, unique
__device__ __forceinline__ unsigned long long rank_key(uint32_t k, int i) {
  return (unsigned long long)k << 32 | (0xFFFFFFFFu - (uint32_t)i);
}

// The K largest of sh.cand[0, n) in order to sh.sorted, n <= CAP.
template <int NT>
__device__ void sort_candidates(Shared& sh, int n, int K) {
  if (n <= 256) {
    for (int i = threadIdx.x; i < n; i += NT) {
      const unsigned long long mine = sh.cand[i];
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) r += sh.cand[j] > mine;
      if (r < K) sh.sorted[r] = mine;
    }
  } else {   // bitonic, descending
    int P = 512;
    while (P < n) P *= 2;
    for (int i = n + threadIdx.x; i < P; i += NT) sh.cand[i] = 0ull;
    sync<NT>();
    for (int k = 2; k <= P; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = threadIdx.x; i < P / 2; i += NT) {
          const int a = 2 * i - (i & (j - 1)), b = a + j;
          const unsigned long long x = sh.cand[a], y = sh.cand[b];
          if ((x < y) == ((a & k) == 0)) {
            sh.cand[a] = y;
            sh.cand[b] = x;
          }
        }
        sync<NT>();
      }
    for (int i = threadIdx.x; i < K && i < n; i += NT) sh.sorted[i] = sh.cand[i];
  }
  if (threadIdx.x == 0) sh.n_sorted = n < K ? n : K;
  sync<NT>();
}

// The CTA's share of a row: nv of its VW virtual warps, from v0 on.  `f(group)` for each of its
// groups, any order over the threads.
template <int NT, int VW, class F>
__device__ __forceinline__ void each_group(int groups, int v0, int nv, F f) {
  const int per = nv * 32;   // groups of the CTA in a round of VW chunks of the row
  for (int i = threadIdx.x;; i += NT) {
    const int g = i / per * (VW * 32) + v0 * 32 + i % per;
    if (i / per * (VW * 32) >= groups) break;
    if (g < groups) f(g);
  }
}

// The CTA's K largest logits when the fast way found too many candidates: the K-th largest
// logit by bisection over its bits, then what is above it, then the first of its ties.
template <int NT, int VW, int DT, bool ALIGNED>
__device__ void select_by_bisection(Shared& sh, const Row<DT, ALIGNED>& row, int v0, int nv, int K) {
  using G = Group<DT>;
  const int groups = row.groups();
  auto count = [&](uint32_t least) {   // logits of the CTA at or above
    int n = 0;
    each_group<NT, VW>(groups, v0, nv, [&](int g) {
      float v[G::E];
      G::floats(row.load(g), v);
#pragma unroll
      for (int j = 0; j < G::E; ++j) n += G::key(v[j]) >= least;
    });
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    sync<NT>();
    if ((threadIdx.x & 31) == 0) sh.scan[threadIdx.x >> 5] = n;
    sync<NT>();
    n = 0;
    for (int w = 0; w < NT / 32; ++w) n += sh.scan[w];
    return n;
  };
  uint32_t kth = 0u;
  for (int b = G::BITS - 1; b >= 0; --b) {
    const uint32_t c = kth | 1u << b;
    if (count(c) >= K) kth = c;
  }
  if (kth < G::kLowest) kth = G::kLowest;
  sync<NT>();
  if (threadIdx.x == 0) sh.n_cand = 0;
  sync<NT>();
  each_group<NT, VW>(groups, v0, nv, [&](int g) {   // fewer than K of them
    float v[G::E];
    G::floats(row.load(g), v);
#pragma unroll
    for (int j = 0; j < G::E; ++j)
      if (G::key(v[j]) > kth) {
        const int at = atomicAdd(&sh.n_cand, 1);
        if (at < CAP) sh.cand[at] = rank_key(G::key(v[j]), g * G::E + j);
      }
  });
  sync<NT>();
  int have = sh.n_cand;
  sync<NT>();
  // ties in the order of their index: NT groups at a time, the counts before a thread's by a scan
  const int per = nv * 32;
  for (int i0 = 0; have < K; i0 += NT) {
    if (i0 / per * (VW * 32) >= groups) break;
    const int i = i0 + threadIdx.x, g = i / per * (VW * 32) + v0 * 32 + i % per;
    uint32_t mask = 0u;
    if (g < groups) {
      float v[G::E];
      G::floats(row.load(g), v);
#pragma unroll
      for (int j = 0; j < G::E; ++j)
        if (G::key(v[j]) == kth && g * G::E + j < row.V) mask |= 1u << j;
    }
    int before = __popc(mask);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += up;
    }
    if (lane == 31) sh.scan[threadIdx.x >> 5] = before;
    before -= __popc(mask);
    sync<NT>();
    int all = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < (int)(threadIdx.x >> 5)) before += sh.scan[w];
      all += sh.scan[w];
    }
    for (int j = 0, at = have + before; mask && at < K; ++j)
      if (mask >> j & 1u) {
        mask &= ~(1u << j);
        sh.cand[at++] = rank_key(kth, g * G::E + j);
      }
    have += all;
    sync<NT>();
  }
  if (threadIdx.x == 0) sh.n_cand = have < K ? have : K;
  sync<NT>();
}

// Thread's largest logits (`tops`, one a virtual warp of its warp) -> the CTA's K largest in
// sh.sorted.  `meanwhile` is run by all threads while the units that are read again are on
// their way.
template <int NT, int VW, int DT, bool ALIGNED, int S, class F>
__device__ __forceinline__ void select_top(Shared& sh, const Row<DT, ALIGNED>& row, int v0, int nv, const float (&tops)[S], int K,
                                           F meanwhile) {
  using G = Group<DT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float mine = tops[0];
#pragma unroll
  for (int j = 1; j < S; ++j) mine = max_nan(mine, tops[j]);
  const uint32_t key = G::key(mine) >> G::SHIFT;
  // a value that K threads reach, and not many more: by bisection over its upper 16 bits
  uint32_t least = 0u;
#pragma unroll 1
  for (int b = 15; b >= 0; --b) {
    const uint32_t c = least | 1u << b;
    const int n = sync_count<NT>(key >= c);
    if (n < K) continue;
    least = c;
    if (n <= K + 1) break;
  }
  least <<= G::SHIFT;
  if (least < G::kLowest) least = G::kLowest;
  if (threadIdx.x == 0) sh.n_units = sh.n_cand = 0;
  sync<NT>();
#pragma unroll
  for (int j = 0; j < S; ++j)
    if (G::key(tops[j]) >= least) {
      const int at = atomicAdd(&sh.n_units, 1);
      if (at < MAX_UNITS) sh.units[at] = (uint32_t)((v0 + warp + j * (NT / 32)) * 32 + lane);
    }
  sync<NT>();
  const int groups = row.groups(), units = sh.n_units;
  const int rounds = (groups + VW * 32 - 1) / (VW * 32);   // groups of a unit
  bool many = units > MAX_UNITS;
  if (!many) {
    constexpr int R = 2;
    const int total = units * rounds;
    int base = 0;
    do {   // all threads together
      uint4 q[R];
      int g[R];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const int i = base + (int)threadIdx.x + u * NT;
        g[u] = i < total ? i / units * (VW * 32) + (int)sh.units[i % units] : groups;
        if (g[u] < groups) q[u] = row.load(g[u]);
      }
      if (base == 0) meanwhile();
#pragma unroll
      for (int u = 0; u < R; ++u) {
        if (g[u] >= groups || !(G::key(G::largest(q[u])) >= least)) continue;   // (a NaN's key is above or below all)
        float v[G::E];
        G::floats(q[u], v);
#pragma unroll
        for (int j = 0; j < G::E; ++j)
          if (G::key(v[j]) >= least) {
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < CAP) sh.cand[at] = rank_key(G::key(v[j]), g[u] * G::E + j);
          }
      }
      base += R * NT;
    } while (base < total);
    sync<NT>();
    many = sh.n_cand > CAP;
  } else {
    meanwhile();
  }
  if (many) select_by_bisection<NT, VW, DT, ALIGNED>(sh, row, v0, nv, K);
  sort_candidates<NT>(sh, sh.n_cand, K);
}

// C CTAs a row of VW virtual warps; a warp holds S of them.
template <int C, int VW>
struct Cut {
  static constexpr int NT = VW == 16 ? 128 : 256, WARPS = NT / 32, NV = VW / C, S = NV / WARPS;
  static_assert(S >= 1 && S * WARPS * C == VW, "every warp has the same share");
};

// The given tokens of a row, a thread's first asked for while the row is read.
template <int DT>
struct Given {
  int id = -1;
  float z = 0.f;
  bool bad = false;
  __device__ __forceinline__ void ask(const TokenArgs& a, int64_t t, const typename Group<DT>::elem* row, int64_t i) {
    id = a.ids[t * a.C + i];
    if (id < -1 || id >= a.V) bad = true;
    z = id >= 0 && id < a.V ? Group<DT>::value(row[id]) : 0.f;
  }
};

// What follows the pass over a row: the CTA's sums joined, the alternatives, the outputs (by
// the cluster's first CTA).
template <int DT, bool ALIGNED, int C, int VW>
__device__ __forceinline__ void end_of_row(Shared& sh, const TokenArgs& a, int64_t t, const Row<DT, ALIGNED>& row, int rank,
                                           const Sums (&sums)[Cut<C, VW>::S], Given<DT>& given, float c, float inv_t) {
  using G = Group<DT>;
  constexpr int NT = Cut<C, VW>::NT, WARPS = Cut<C, VW>::WARPS, NV = Cut<C, VW>::NV, S = Cut<C, VW>::S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, v0 = rank * NV;
  float tops[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    tops[j] = sums[j].top;
    const Part p = join(sums[j].m, sums[j].top, __fadd_rn(sums[j].s.x, sums[j].s.y), __fadd_rn(sums[j].t.x, sums[j].t.y), c);
    if (lane == 0) sh.part[v0 + warp + j * WARPS] = p;
  }
  sync<NT>();
  // the row's sums, from all its virtual warps, by the last warp
  auto conclude = [&] {
    if (warp != WARPS - 1) return;
    const Part p = lane < VW ? sh.part[lane] : Part{-INFINITY, 0.f, 0.f};
    const Part all = join(p.top, p.top, p.s, p.t, c);
    const bool bad = !(all.top > -INFINITY && all.top < INFINITY) || all.s != all.s;
    if (lane == 0) {
      sh.M = bad ? NAN : all.top;
      sh.lnS = bad ? NAN : logf(all.s);
      sh.bad = bad;
      const float H = bad ? NAN : __fmaf_rn(-kLn2, __fdiv_rn(all.t, all.s), sh.lnS);
      if (a.out_entropy) a.out_entropy[t] = H;
      if (a.state) *reinterpret_cast<float4*>(a.state + 4 * t) = make_float4(sh.M, bad ? NAN : log2f(all.s), H, a.temperature);
      if (bad && a.status) atomicOr(a.status, RLK_STATUS_NONFINITE);
    }
  };
  if (a.top > 0)
    select_top<NT, VW, DT, ALIGNED, S>(sh, row, v0, NV, tops, a.top, [&] {
      if (C == 1) {
        __syncwarp();
        conclude();
      }
    });
  if (C > 1) {
    tc::cluster_sync();
    if (rank != 0) {
      tc::cluster_leave();   // rank 0 has read what this CTA holds
      return;
    }
    // the other CTAs' parts and alternatives
    for (int i = threadIdx.x; i < VW; i += NT) {
      const int from = i / NV;
      if (from == 0) continue;
      const uint32_t at = tc::peer_addr(smem_u32(&sh.part[i]), (uint32_t)from);
      sh.part[i] = Part{tc::ld_peer_f32(at), tc::ld_peer_f32(at + 4), tc::ld_peer_f32(at + 8)};
    }
    if (a.top > 0) {
      for (int i = threadIdx.x; i < sh.n_sorted; i += NT) sh.cand[i] = sh.sorted[i];
      int base = sh.n_sorted;
      for (int k = 1; k < C; ++k) {
        const int n = (int)tc::ld_peer_u32(tc::peer_addr(smem_u32(&sh.n_sorted), (uint32_t)k));
        for (int i = threadIdx.x; i < n; i += NT) {
          const uint32_t at = tc::peer_addr(smem_u32(&sh.sorted[i]), (uint32_t)k);
          sh.cand[base + i] = (unsigned long long)tc::ld_peer_u32(at + 4) << 32 | tc::ld_peer_u32(at);
        }
        base += n;
      }
      sync<NT>();
      sort_candidates<NT>(sh, base, a.top);
    }
    sync<NT>();
    tc::cluster_leave();
  }
  if (C > 1 || a.top == 0) {
    conclude();
    sync<NT>();
  }
  const float M = sh.M, lnS = sh.lnS;
  auto logprob = [&](float z) { return __fsub_rn(__fmul_rn(__fsub_rn(z, M), inv_t), lnS); };
  for (int64_t i = threadIdx.x; i < a.C; i += NT) {
    if (i >= NT) given.ask(a, t, row.p, i);
    a.out_logprob[t * a.C + i] = given.id == -1 ? 0.f : (given.id < 0 || given.id >= a.V ? NAN : logprob(given.z));
  }
  if (given.bad && a.status) atomicOr(a.status, RLK_STATUS_BAD_TOKEN_ID);
  for (int i = threadIdx.x; i < a.top; i += NT) {
    int id = -1;
    float lp = sh.bad ? NAN : -INFINITY;
    if (!sh.bad && i < sh.n_sorted) {
      const unsigned long long k = sh.sorted[i];
      id = (int)(0xFFFFFFFFu - (uint32_t)k);
      lp = logprob(G::of_key((uint32_t)(k >> 32)));
    }
    a.out_top_ids[t * a.top + i] = id;
    a.out_top_logprob[t * a.top + i] = lp;
  }
}

// A row to each cluster of C CTAs, read straight into registers.
template <int DT, bool ALIGNED, int C, int VW>
__global__ void __launch_bounds__(Cut<C, VW>::NT, 1024 / Cut<C, VW>::NT) token_forward_kernel(TokenArgs a, float c, float inv_t) {
  using K = Cut<C, VW>;
  constexpr int WARPS = K::WARPS, S = K::S;
  pdl_wait();
  __shared__ Shared sh;
  const int rank = C == 1 ? 0 : (int)tc::cluster_rank();
  const int64_t t = blockIdx.x / C;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Row<DT, ALIGNED> row(a.logits, t, a.ld, a.V);
  const int groups = row.groups();
  const float slack = fminf(__fdiv_rn(16.f, c), 0x1p125f);
  Given<DT> given;
  if (rank == 0 && (int)threadIdx.x < a.C) given.ask(a, t, row.p, threadIdx.x);

  Sums sums[S];
  constexpr int U = S == 4 ? 1 : (S == 2 ? 2 : 4);   // rounds (of VW chunks of the row) in flight together
  const int g0 = (rank * K::NV + warp) * 32 + lane;
  int r = 0;
  const int whole = (groups - 1) / (VW * 32);          // rounds in which every lane has a group
  for (; r + U <= whole; r += U) {
    uint4 q[U][S];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < S; ++j) q[u][j] = row.template load<true>((r + u) * (VW * 32) + g0 + j * (WARPS * 32));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < S; ++j) absorb<DT>(sums[j], q[u][j], c, slack);
  }
  for (; r * (VW * 32) < groups; ++r) {
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int g = r * (VW * 32) + g0 + j * (WARPS * 32);
      if (g < groups) absorb<DT>(sums[j], row.load(g), c, slack);
    }
  }
  end_of_row<DT, ALIGNED, C, VW>(sh, a, t, row, rank, sums, given, c, inv_t);
}

// Many rows off 16-byte boundaries: persistent CTAs, each with a ring of shared memory that one more warp keeps
// full by bulk copies, also with the next row while this one's alternatives are selected.  A
// stage is a round (32 chunks, 16 KB).
constexpr int RING = 3, ROUND = 32 * 32 * 16, SLOT = ROUND + 16;   // (+ the word that an unaligned round's last group ends in)
constexpr int RING_CTAS = 3;   // of an SM
template <int DT>
__global__ void __launch_bounds__(Cut<1, 32>::NT + 32, RING_CTAS)
    token_stream_kernel(TokenArgs a, float c, float inv_t, long long limit, int withhold) {
  using K = Cut<1, 32>;
  constexpr int NT = K::NT, WARPS = K::WARPS, S = K::S;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ Shared sh;
  __shared__ uint64_t s_bars[2 * RING];
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full = smem_u32(s_bars), empty = full + 8 * RING;
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(full + 8 * i, 1 + (i == withhold && blockIdx.x == 0));
      mbar_init(empty + 8 * i, WARPS);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  __syncthreads();
  const int groups = Row<DT, false>(a.logits, 0, a.ld, a.V).groups(), rounds = (groups + 1023) / 1024;
  const int64_t bytes = a.V * (DT ? 4 : 2);
  if (warp == WARPS) {
    if (lane == 0) {
      uint32_t slot = 0, phase = 0, used = 0u, parity = 0u;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < a.T && ok; t += gridDim.x) {
        const Row<DT, false> row(a.logits, t, a.ld, a.V);
        // the row's whole aligned words, by their distance from the word that it starts in
        const char* word0 = reinterpret_cast<const char*>(row.p) - row.sh;
        const int64_t first = row.sh ? 16 : 0, last = (row.sh + bytes) & ~(int64_t)15;
        for (int r = 0; r < rounds; ++r) {
          if (!tc::wait(empty + 8 * slot, phase ^ 1u, &s_abort, limit)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();   // the slot was read before
          int64_t from = (int64_t)r * ROUND, to = from + SLOT;
          const uint32_t dst = smem_u32(ring) + slot * SLOT + (from < first ? (uint32_t)(first - from) : 0u);
          from = from < first ? first : from;
          to = to < last ? to : last;
          if (to > from) {
            mbar_expect_tx(full + 8 * slot, (uint32_t)(to - from));
            bulk_copy_g2s(dst, word0 + from, (uint32_t)(to - from), full + 8 * slot);
            used |= 1u << slot;
            parity = (parity & ~(1u << slot)) | (phase << slot);
          } else {
            mbar_arrive(full + 8 * slot);
          }
          if (++slot == RING) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      const long long t0 = clock64();   // every copy lands before the CTA exits (within the limit)
      for (int i = 0; i < RING; ++i)
        while ((used >> i & 1u) && !mbar_try_wait(full + 8 * i, parity >> i & 1u) && clock64() - t0 <= limit) {}
    }
    return;
  }
  const float slack = fminf(__fdiv_rn(16.f, c), 0x1p125f);
  const int inner = (groups - 2) / 1024;   // rounds whose groups all have two after them
  uint32_t slot = 0, phase = 0;
  bool ok = true;   // once a wait has run out, no later one counts (a barrier's parity could pass for it)
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const Row<DT, false> row(a.logits, t, a.ld, a.V);
    Given<DT> given;
    if ((int)threadIdx.x < a.C) given.ask(a, t, row.p, threadIdx.x);
    Sums sums[S];
    for (int r = 0; r < rounds && ok; ++r) {
      ok = __all_sync(0xFFFFFFFFu, tc::wait(full + 8 * slot, phase, &s_abort, limit));
      if (!ok) break;
      uint4 q[S];
      const int g0 = r * 1024 + warp * 32 + lane;
      const uint8_t* at = ring + slot * SLOT + (warp * 32 + lane) * 16;
      const uint32_t done = empty + 8 * slot;
      if (++slot == RING) {
        slot = 0;
        phase ^= 1u;
      }
      if (r < inner && r > 0) {
#pragma unroll
        for (int j = 0; j < S; ++j) q[j] = row.template from_copy<true>(at + j * (WARPS * 512), g0 + j * (WARPS * 32));
        __syncwarp();
        if (lane == 0) mbar_arrive(done);
#pragma unroll
        for (int j = 0; j < S; ++j) absorb<DT>(sums[j], q[j], c, slack);
      } else {
#pragma unroll
        for (int j = 0; j < S; ++j)
          if (g0 + j * (WARPS * 32) < groups) q[j] = row.from_copy(at + j * (WARPS * 512), g0 + j * (WARPS * 32));
        __syncwarp();
        if (lane == 0) mbar_arrive(done);
#pragma unroll
        for (int j = 0; j < S; ++j)
          if (g0 + j * (WARPS * 32) < groups) absorb<DT>(sums[j], q[j], c, slack);
      }
    }
    if (!ok) {   // a wait ran out: this row and the CTA's later ones are NaN
      sums[0].top = NAN;
      if (lane == 0 && a.status) atomicOr(a.status, RLK_STATUS_TIMEOUT);
    }
    end_of_row<DT, false, 1, 32>(sh, a, t, row, 0, sums, given, c, inv_t);
    sync<NT>();   // the next row's parts go where this one's were
  }
}

// ------------------------------------------------------------ backward
// A CTA writes a run of a row's gradient and then, over it, the places that the given tokens
// and the alternatives name (each by the thread of the first that names it, with the sum of
// all that do), so nothing is added with atomics.  Memory bounds it: one read, one write.
constexpr int BT = 256;
constexpr int MAX_NAMED = RLK_MAX_TOKENS + MAX_TOP;

template <int OT>
__device__ __forceinline__ void store_one(void* out, int64_t i, float v) {
  if (OT == 0) static_cast<uint16_t*>(out)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else static_cast<float*>(out)[i] = v;
}

template <int DT, int OT>
__global__ void __launch_bounds__(BT, 4) token_backward_kernel(TokenBwdArgs a, float c, float inv_t, int run) {
  using G = Group<DT>;
  constexpr int E = G::E;
  pdl_wait();
  __shared__ float s_red[BT / 32];
  __shared__ int s_bad;
  __shared__ int s_id[MAX_NAMED];
  __shared__ float s_g[MAX_NAMED];
  const int64_t t = blockIdx.y;
  const int V = (int)a.V, first = (int)blockIdx.x * run, last = V - first < run ? V : first + run;
  const typename G::elem* z = static_cast<const typename G::elem*>(a.logits) + t * a.ld;
  char* out = static_cast<char*>(a.grad) + t * a.ldg * (OT ? 4 : 2);
  const float4 st = *reinterpret_cast<const float4*>(a.state + 4 * t);
  const float M = st.x, log2S = st.y, H = st.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // where 16-byte groups of the run start, and whether the gradient's groups can be stored whole there
  const uintptr_t za = reinterpret_cast<uintptr_t>(z + first), oa = reinterpret_cast<uintptr_t>(out) + (uintptr_t)first * (OT ? 4 : 2);
  int head = (int)((16u - (za & 15u)) & 15u) / (int)sizeof(*z);
  const bool vec = (oa + (uintptr_t)head * (OT ? 4 : 2)) % (OT ? 16 : 2 * E) == 0;   // the size of its stores
  if (head > last - first) head = last - first;
  const int body = vec ? (last - first - head) / E : 0;   // whole groups
  const uint4* zg = reinterpret_cast<const uint4*>(z + first + head);
  constexpr int U = 4;
  uint4 q[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if ((int)threadIdx.x + u * BT < body) q[u] = __ldg(zg + threadIdx.x + u * BT);

  // what is named, with its gradient, and the sum of it all
  const int n = (int)a.C + (int)a.top;
  if (threadIdx.x == 0) {
    s_bad = !(M == M) || st.w != a.temperature;
    if (M == M && s_bad && a.status) atomicOr(a.status, RLK_STATUS_BAD_PARAM);
  }
  __syncthreads();
  float sum = 0.f;
  for (int i = threadIdx.x; i < n; i += BT) {
    const bool given = i < a.C;
    int id = given ? a.ids[t * a.C + i] : a.top_ids[t * a.top + i - a.C];
    float g = given ? (a.grad_logprob ? a.grad_logprob[t * a.C + i] : 0.f) : (a.grad_top ? a.grad_top[t * a.top + i - a.C] : 0.f);
    if (id < -1 || id >= V) {
      s_bad = 1;
      if (a.status) atomicOr(a.status, RLK_STATUS_BAD_TOKEN_ID);
      id = -1;
    }
    if (id < 0 || G::value(z[id < 0 ? 0 : id]) == -INFINITY) {   // no such log-probability
      id = -1;
      g = 0.f;
    }
    s_id[i] = id;
    s_g[i] = g;
    sum = __fadd_rn(sum, g);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, o));
  if (lane == 0) s_red[warp] = sum;
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int w = 0; w < BT / 32; ++w) total = __fadd_rn(total, s_red[w]);
  const bool bad = s_bad != 0;
  const float gH = a.grad_entropy ? a.grad_entropy[t] : 0.f;
  // -dz T = p (G + gH (ln2 d + H)), d = log2 p
  const float k0 = __fmaf_rn(gH, H, total), k1 = __fmul_rn(gH, kLn2), scale = bad ? NAN : -inv_t;
  auto pair = [&](float2 v) {
    float2 d = add2(mul2(add2(v, both(-M)), both(c)), both(-log2S));
    d.x = max_nan(d.x, CLAMP);
    d.y = max_nan(d.y, CLAMP);
    const float2 p = make_float2(ex2(d.x), ex2(d.y));
    return mul2(mul2(p, both(scale)), fma2(d, both(k1), both(k0)));
  };
  for (int i0 = threadIdx.x; i0 < body; i0 += U * BT) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * BT;
      if (i >= body) break;
      float v[E], o[E];
      G::floats(q[u], v);
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        const float2 d = pair(make_float2(v[j], v[j + 1]));
        o[j] = d.x;
        o[j + 1] = d.y;
      }
      char* to = out + (int64_t)(first + head + i * E) * (OT ? 4 : 2);
      if (i + U * BT < body) q[u] = __ldg(zg + i + U * BT);
      if (OT == 0) {
        uint32_t w[E / 2];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if constexpr (E == 8) __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[1], w[2], w[3]));
        else __stcs(reinterpret_cast<uint2*>(to), make_uint2(w[0], w[1]));
      } else {
#pragma unroll
        for (int j = 0; j < E; j += 4)
          __stcs(reinterpret_cast<float4*>(to + 4 * j), make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]));
      }
    }
  }
  // what lies in no group
  const int from = first + head + body * E;
  auto single = [&](int e) { store_one<OT>(out, e, pair(both(G::value(z[e]))).x); };
  for (int e = first + threadIdx.x; e < first + head; e += BT) single(e);
  for (int e = from + threadIdx.x; e < last; e += BT) single(e);
  if (bad) return;
  __syncthreads();   // the places below are written over
  for (int i = threadIdx.x; i < n; i += BT) {
    const int id = s_id[i];
    if (id < first || id >= last) continue;
    float g = 0.f;
    bool earlier = false;
    for (int j = 0; j < n; ++j) {
      if (s_id[j] != id) continue;
      if (j < i) earlier = true;
      g = __fadd_rn(g, s_g[j]);
    }
    if (earlier) continue;
    const float rest = pair(both(G::value(z[id]))).x;
    store_one<OT>(out, id, __fmaf_rn(g, inv_t, rest));
  }
}

template <int DT, bool ALIGNED, int C, int VW>
cudaError_t launch_forward(const TokenArgs& a, float c, float inv_t, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.T * C));
  cfg.blockDim = dim3(Cut<C, VW>::NT);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, token_forward_kernel<DT, ALIGNED, C, VW>, a, c, inv_t);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int DT>
cudaError_t launch_stream(const TokenArgs& a, float c, float inv_t, cudaStream_t stream) {
  static std::atomic<int> done[64];
  const auto kernel = token_stream_kernel<DT>;
  const int ds = device_slot();
  if (ds < 0 || !done[ds].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING * SLOT);
    if (e != cudaSuccess) return e;
    if (ds >= 0) done[ds].store(1);
  }
  const int64_t most = (int64_t)sm_count() * RING_CTAS;
  const cudaError_t e = launch_after(kernel, dim3((unsigned)(a.T < most ? a.T : most)), dim3(Cut<1, 32>::NT + 32), RING * SLOT, stream,
                                     a, c, inv_t, debug_wait_limit(), (int)debug_take_withheld());
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int DT, bool ALIGNED>
cudaError_t forward_by_rows(const TokenArgs& a, float c, float inv_t, cudaStream_t stream) {
  const int64_t sms = sm_count(), bytes = a.V * (a.dtype ? 4 : 2);
  if (bytes <= kShortRow) return launch_forward<DT, ALIGNED, 1, 16>(a, c, inv_t, stream);
  if (bytes >= kLongRow && a.T * 4 <= sms) return launch_forward<DT, ALIGNED, 4, 32>(a, c, inv_t, stream);
  if (bytes >= kLongRow && a.T <= 2 * sms) return launch_forward<DT, ALIGNED, 2, 32>(a, c, inv_t, stream);
  // Rows off 16-byte boundaries go through the ring (their groups span two words, of which few
  // fit into registers on their way): 777 x 50021 fp32 with 50 alternatives 51 us, 78 straight;
  // aligned ones straight into registers with a third more warps: 4096 x 151936 bf16 195 us, 214
  // through the ring.
  if (ALIGNED || a.T <= 2 * sms) return launch_forward<DT, ALIGNED, 1, 32>(a, c, inv_t, stream);
  return launch_stream<DT>(a, c, inv_t, stream);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenArgs& a, cudaStream_t stream) {
  const float c = (float)(1.4426950408889634 / (double)a.temperature), inv_t = (float)(1.0 / (double)a.temperature);
  const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && (a.T == 1 || a.ld % (a.dtype ? 4 : 8) == 0);
  if (a.dtype == 0) return aligned ? forward_by_rows<0, true>(a, c, inv_t, stream) : forward_by_rows<0, false>(a, c, inv_t, stream);
  return aligned ? forward_by_rows<1, true>(a, c, inv_t, stream) : forward_by_rows<1, false>(a, c, inv_t, stream);
}

cudaError_t launch_token_logprobs_backward(const TokenBwdArgs& a, cudaStream_t stream) {
  const float c = (float)(1.4426950408889634 / (double)a.temperature), inv_t = (float)(1.0 / (double)a.temperature);
  // a run of a row for each CTA: long ones (the named places are looked up once a run), but
  // eight CTAs an SM where the rows are few
  int64_t run = 32768;
  while (run > 4096 && a.T * ((a.V + run - 1) / run) < 8 * (int64_t)sm_count()) run /= 2;
  // grid.y holds 65535 rows at most
  for (int64_t t0 = 0; t0 < a.T; t0 += 65535) {
    TokenBwdArgs b = a;
    const int64_t rows = a.T - t0 < 65535 ? a.T - t0 : 65535;
    b.logits = static_cast<const char*>(a.logits) + t0 * a.ld * (a.dtype ? 4 : 2);
    b.grad = static_cast<char*>(a.grad) + t0 * a.ldg * (a.grad_dtype ? 4 : 2);
    b.state = a.state + 4 * t0;
    b.ids = a.ids ? a.ids + t0 * a.C : nullptr;
    b.top_ids = a.top_ids ? a.top_ids + t0 * a.top : nullptr;
    b.grad_logprob = a.grad_logprob ? a.grad_logprob + t0 * a.C : nullptr;
    b.grad_top = a.grad_top ? a.grad_top + t0 * a.top : nullptr;
    b.grad_entropy = a.grad_entropy ? a.grad_entropy + t0 : nullptr;
    const dim3 grid((unsigned)((a.V + run - 1) / run), (unsigned)rows);
    const auto kernel = a.dtype == 0 ? (a.grad_dtype == 0 ? token_backward_kernel<0, 0> : token_backward_kernel<0, 1>)
                                     : (a.grad_dtype == 0 ? token_backward_kernel<1, 0> : token_backward_kernel<1, 1>);
    const cudaError_t e = launch_after(kernel, grid, dim3(BT), 0, stream, b, c, inv_t, (int)run);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace rlk
