// rlk_gated_linear_fwd / rlk_gated_linear_bwd: the gated half of a feed-forward block.
//
//   forward   g = x w_gate^T + b_gate,  u = x w_up^T + b_up,  y = act(g) u
//   backward  dg = dy u act'(g),  du = dy act(g),
//             dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x,  sums of dg and du
//
// Forward: one kernel.  A tile of B is half rows of w_gate and half the same rows of w_up, so
// one tile of accumulators holds both projections of 128 columns (a pair of CTAs: one stages
// the gate's weights, the other the other's), x is read once for both, and the epilogue joins
// column c with column c + 128.  Up to four rows take dot products instead, as the weights'
// bytes bound them.
// Backward: one pass forms dg and du and their sums; dx is one product whose K runs over both
// halves, so it is rounded once; both weights' gradients are one launch.
//
// Measured: 8192 x 14336 x 4096 with SiLU, projections kept, 1010 to 1090 us (1.76 to 1.9 PFLOP/s; tensor
// pipe 88 % of its cycles), 1160 to 1210 in a loop under the power cap; backward of 8192 x 8192 x 4096 1340 to
// 1440 us (dx 93 %, both dW 85 %, dg and du 110 us), fp32 weight gradients 1465, accumulated 1520, x from its
// checkpoint 1440; one row of 14336 x 4096 35 us (6.66 TB/s); 8 rows 48, 64 rows 50 to 51, 128 rows 55 (224 tiles
// on 152 SMs: 72 of them work on two); 1531 x 2731 x 1001 off 16 bytes with GELU 33 to 37 (17 of them copies; 1536 x
// 2736 x 1008 22.5), its backward 94 (74).
//
// dg and du are rounded to bf16 for the products, as the tensor cores need (relative 2^-8 a
// term, of either sign); the bias gradients sum them unrounded.
#include <math.h>

#include "activation.cuh"
#include "checkpoint.cuh"
#include "gemm.cuh"

namespace rlk {
namespace {

using gemm::Loop;
using gemm::Maps;
using gemm::Operand;
using gemm::Tile;

bool rows16(const void* p, int dtype, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (dtype ? 4 : 8) == 0;
}
bool tma_rows(const void* p, int64_t ld) { return rows16(p, 0, ld); }
bool rows4(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0; }
int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t copy_bytes(int64_t rows, int64_t cols) { return pad256((size_t)rows * pad8(cols) * 2); }

// ------------------------------------------------------------ forward
struct GatedOut {
  const void* bias[2];     // gate, up: [N] or NULL
  int bias_dtype;
  int act;
  void* y;
  int y_dtype;
  int64_t ldy;
  uint16_t* z[2];          // the pre-activations, or NULL
  int64_t ldz;
};

__device__ __forceinline__ float gated_bias(const GatedOut& o, int which, int64_t col) {
  return o.bias_dtype ? static_cast<const float*>(o.bias[which])[col]
                      : bf16_val(static_cast<const uint16_t*>(o.bias[which])[col]);
}
// One column of R rows `step` apart, of which those up to n rows on exist.
template <int R>
__device__ __forceinline__ void gated_column(const GatedOut& o, int64_t row, int step, int n, int64_t col, float (&g)[R], float (&u)[R]) {
  if (o.bias[0]) {
    const float b = gated_bias(o, 0, col);
#pragma unroll
    for (int k = 0; k < R; ++k) g[k] = __fadd_rn(g[k], b);
  }
  if (o.bias[1]) {
    const float b = gated_bias(o, 1, col);
#pragma unroll
    for (int k = 0; k < R; ++k) u[k] = __fadd_rn(u[k], b);
  }
  if (o.z[0]) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (k * step >= n) continue;
      const int64_t at = (row + k * step) * o.ldz + col;
      o.z[0][at] = (uint16_t)pack_bf16(g[k], 0.f);
      o.z[1][at] = (uint16_t)pack_bf16(u[k], 0.f);
    }
  }
  activate(g, o.act);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (k * step >= n) continue;
    const float y = __fmul_rn(g[k], u[k]);
    const int64_t at = (row + k * step) * o.ldy + col;
    if (o.y_dtype) static_cast<float*>(o.y)[at] = y;
    else static_cast<uint16_t*>(o.y)[at] = (uint16_t)pack_bf16(y, 0.f);
  }
}

struct ForwardOp {
  static constexpr bool A_MN = false, B_MN = false, F16 = false, DUAL = true, STACKED = false, TRI_A = false, TRI_B = false;
  struct Params {
    Loop loop;
    int64_t M, N;
    int n_mt, n_nt, vec;
    GatedOut out;
  };
  static __device__ __forceinline__ Tile tile(const Params& p, int t, int tm, int bn) {
    int mt, nt;
    gemm::grouped(t, p.n_mt, p.n_nt, mt, nt);
    return Tile{mt * tm, nt * bn, (int64_t)mt * tm, (int64_t)nt * bn, p.M, p.N, 0};
  }
  static __device__ __forceinline__ void source(const Tile&, int, int&, int&) {}
  static __device__ __forceinline__ bool vec(const Params& p) { return p.vec != 0; }
  struct Aux {};
  static __device__ __forceinline__ void aux8(const Params&, const Tile&, int64_t, int64_t, int, Aux&) {}
  struct Cols {
    float g[8], u[8];
  };
  static __device__ __forceinline__ void cols8(const Params& p, const Tile&, int64_t col, int n, Cols& c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c.g[j] = p.out.bias[0] && j < n ? gated_bias(p.out, 0, col + j) : 0.f;
      c.u[j] = p.out.bias[1] && j < n ? gated_bias(p.out, 1, col + j) : 0.f;
    }
  }
  static __device__ __forceinline__ void finish8(const Params& p, const Tile&, int64_t row, int64_t col, int n, float (&g)[8],
                                                 float (&u)[8], const Aux&, const Cols& c) {
    const GatedOut& o = p.out;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 a = add2(make_float2(g[j], g[j + 1]), make_float2(c.g[j], c.g[j + 1]));
      const float2 b = add2(make_float2(u[j], u[j + 1]), make_float2(c.u[j], c.u[j + 1]));
      g[j] = a.x;
      g[j + 1] = a.y;
      u[j] = b.x;
      u[j + 1] = b.y;
    }
    if (o.z[0]) {
      store8(o.z[0] + row * o.ldz + col, g, n);
      store8(o.z[1] + row * o.ldz + col, u, n);
    }
    activate(g, o.act);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 a = mul2(make_float2(g[j], g[j + 1]), make_float2(u[j], u[j + 1]));
      g[j] = a.x;
      g[j + 1] = a.y;
    }
    if (o.y_dtype == 0) {
      store8(static_cast<uint16_t*>(o.y) + row * o.ldy + col, g, n);
      return;
    }
    float* y = static_cast<float*>(o.y) + row * o.ldy + col;
    if (n == 8) {
      reinterpret_cast<float4*>(y)[0] = make_float4(g[0], g[1], g[2], g[3]);
      reinterpret_cast<float4*>(y)[1] = make_float4(g[4], g[5], g[6], g[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) y[j] = g[j];
    }
  }
  static __device__ __forceinline__ void column8(const Params& p, const Tile&, int64_t row, int step, int n, int64_t col,
                                                 float (&g)[8], float (&u)[8]) {
    gated_column<8>(p.out, row, step, n, col, g, u);
  }
};

// ------------------------------------------------------------ backward products
struct StoreOut {
  void* y;
  int64_t ld;
};
// D to memory as it is; KCAT: one product whose second half of K takes the second maps;
// else two products (of which the second takes a[1]), one after the other in the tiles' order.
template <bool A_MN_, bool KCAT>
struct StoreOp {
  static constexpr bool A_MN = A_MN_, B_MN = true, F16 = false, DUAL = false, STACKED = false, TRI_A = false, TRI_B = false;
  struct Params {
    Loop loop;
    int64_t M, N;
    int n_mt, n_nt, vec;
    int y_dtype, accumulate;
    StoreOut out[2];
  };
  static __device__ __forceinline__ Tile tile(const Params& p, int t, int tm, int bn) {
    const int which = KCAT ? 0 : t / (p.n_mt * p.n_nt);
    int mt, nt;
    gemm::grouped(t - which * p.n_mt * p.n_nt, p.n_mt, p.n_nt, mt, nt);
    return Tile{mt * tm, nt * bn, (int64_t)mt * tm, (int64_t)nt * bn, p.M, p.N, which};
  }
  static __device__ __forceinline__ void source(const Tile& tl, int part, int& ia, int& ib) {
    if (KCAT) ia = ib = part;
    else ia = tl.which;
  }
  static __device__ __forceinline__ bool vec(const Params& p) { return p.vec != 0; }
  struct Aux {};
  static __device__ __forceinline__ void aux8(const Params&, const Tile&, int64_t, int64_t, int, Aux&) {}
  struct Cols {};
  static __device__ __forceinline__ void cols8(const Params&, const Tile&, int64_t, int, Cols&) {}
  static __device__ __forceinline__ void finish8(const Params& p, const Tile& tl, int64_t row, int64_t col, int n, float (&v)[8],
                                                 float (&)[8], const Aux&, const Cols&) {
    const StoreOut& o = p.out[tl.which];
    if (p.y_dtype == 0) {
      store8(static_cast<uint16_t*>(o.y) + row * o.ld + col, v, n);
      return;
    }
    float* y = static_cast<float*>(o.y) + row * o.ld + col;
    if (n == 8) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float4 w = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        if (p.accumulate) {
          const float4 old = reinterpret_cast<const float4*>(y)[k];
          w = make_float4(__fadd_rn(old.x, w.x), __fadd_rn(old.y, w.y), __fadd_rn(old.z, w.z), __fadd_rn(old.w, w.w));
        }
        reinterpret_cast<float4*>(y)[k] = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) y[j] = p.accumulate ? __fadd_rn(y[j], v[j]) : v[j];
    }
  }
  static __device__ __forceinline__ void column8(const Params& p, const Tile& tl, int64_t row, int step, int n, int64_t col,
                                                 float (&v)[8], float (&)[8]) {
    const StoreOut& o = p.out[tl.which];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k * step >= n) continue;
      const int64_t at = (row + k * step) * o.ld + col;
      if (p.y_dtype == 0) {
        static_cast<uint16_t*>(o.y)[at] = (uint16_t)pack_bf16(v[k], 0.f);
      } else {
        float* y = static_cast<float*>(o.y) + at;
        *y = p.accumulate ? __fadd_rn(*y, v[k]) : v[k];
      }
    }
  }
};

// 128 x 128 tiles, K split over a cluster while SMs are left, when there is an SM for each
// (or there are no rows for a pair); else pairs' tiles: the linear layer's rule.  `products`
// of M x N; out: D's columns of a small tile.
template <class Op>
cudaError_t run_tiles(const Maps& maps, typename Op::Params& p, int products, int out, bool few, cudaStream_t stream) {
  const int tm = few ? 128 : 256, tn = few ? out : 2 * out;
  p.n_mt = (int)((p.M + tm - 1) / tm);
  p.n_nt = (int)((p.N + tn - 1) / tn);
  const int64_t tiles = (int64_t)products * p.n_mt * p.n_nt;
  if (tiles > (1 << 30)) return cudaErrorInvalidValue;
  p.loop.n_tiles = (int)tiles;
  return few ? gemm::launch<Op, true>(maps, p, stream) : gemm::launch<Op, false>(maps, p, stream);
}
bool few_tiles(int64_t M, int64_t N, int products, int out) {
  return M <= 128 || (int64_t)products * ((M + 127) / 128) * ((N + out - 1) / out) <= sm_count();
}

// ------------------------------------------------------------ a few rows
// Each column of y is two dot products; a warp takes a column (or `wpf` warps share one, each
// a run of K), U loads of each weight in flight a lane, at distances known when this is
// compiled.  W columns a load: 8, 2 or 1 by the alignment of the rows of x and the weights.
// Their sums are joined in a fixed order.
// Up to four rows whatever the weights, as in the linear layer (us, this and tiles: 14336 x 4096 1 row
// 36 and 47, 2 rows 39 and 47; 2048 x 1024 4 rows 5.2 and 6.9.  3 and 4 rows of large weights would be faster as tiles,
// 52 and 54 here and 47 there, 4096 x 14336 75 and 78 and 48: the converted weights meet each row's loads of x.)
constexpr int FEW_ROWS = 4, FEW_T = 256;
template <int W>
struct Word;
template <>
struct Word<8> {
  using type = uint4;
  static __device__ __forceinline__ void floats(const uint4& q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(u[j]);
      v[2 * j + 1] = bf16_hi(u[j]);
    }
  }
};
template <>
struct Word<2> {
  using type = uint32_t;
  static __device__ __forceinline__ void floats(uint32_t q, float (&v)[2]) {
    v[0] = bf16_lo(q);
    v[1] = bf16_hi(q);
  }
};
template <>
struct Word<1> {
  using type = uint16_t;
  static __device__ __forceinline__ void floats(uint16_t q, float (&v)[1]) { v[0] = bf16_val(q); }
};

struct FewRows {
  const uint16_t *x, *wg, *wu;
  int64_t ldx, ldwg, ldwu, N;
  int K, wpf;
  GatedOut out;
};
template <int R, int W>
__global__ void __launch_bounds__(FEW_T, R <= 2 ? 4 : 3) gated_few_rows_kernel(const FewRows a) {
  pdl_wait();
  __shared__ float s_part[FEW_T / 32][2 * R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & (a.wpf - 1);
  const int64_t f = (int64_t)blockIdx.x * (FEW_T / 32 / a.wpf) + warp / a.wpf;
  float2 acc[2 * R];
#pragma unroll
  for (int m = 0; m < 2 * R; ++m) acc[m] = make_float2(0.f, 0.f);
  if (f < a.N) {
    const uint16_t *wg = a.wg + f * a.ldwg, *wu = a.wu + f * a.ldwu;
    using T = typename Word<W>::type;
    constexpr int U = W == 8 ? (R <= 2 ? 4 : 2) : 8, STEP = 32 * W;
    const int share = (a.K + a.wpf * STEP - 1) / (a.wpf * STEP) * STEP, whole = a.K / W * W;   // a warp's columns: whole loads
    const int end = min(whole, (part + 1) * share);
    auto add = [&](const T& g, const T& u, int k) {
      float gv[W], uv[W];
      Word<W>::floats(g, gv);
      Word<W>::floats(u, uv);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        float xv[W];
        Word<W>::floats(*reinterpret_cast<const T*>(a.x + m * a.ldx + k), xv);
        if constexpr (W == 1) {
          acc[2 * m].x = __fmaf_rn(gv[0], xv[0], acc[2 * m].x);
          acc[2 * m + 1].x = __fmaf_rn(uv[0], xv[0], acc[2 * m + 1].x);
        } else {
#pragma unroll
          for (int j = 0; j < W; j += 2) {
            const float2 x2 = make_float2(xv[j], xv[j + 1]);
            acc[2 * m] = fma2(make_float2(gv[j], gv[j + 1]), x2, acc[2 * m]);
            acc[2 * m + 1] = fma2(make_float2(uv[j], uv[j + 1]), x2, acc[2 * m + 1]);
          }
        }
      }
    };
    int k0 = part * share + lane * W;
    for (; k0 - lane * W + STEP * U <= end; k0 += STEP * U) {
      T g[U], u[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        g[i] = __ldcs(reinterpret_cast<const T*>(wg + k0 + i * STEP));
        u[i] = __ldcs(reinterpret_cast<const T*>(wu + k0 + i * STEP));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) add(g[i], u[i], k0 + i * STEP);
    }
    for (; k0 < end; k0 += STEP)
      add(__ldcs(reinterpret_cast<const T*>(wg + k0)), __ldcs(reinterpret_cast<const T*>(wu + k0)), k0);
    const int k = whole + lane;   // the last K % W columns
    if (part == 0 && k < a.K) {
#pragma unroll
      for (int m = 0; m < R; ++m) {
        const float xv = bf16_val(a.x[m * a.ldx + k]);
        acc[2 * m].x = __fmaf_rn(bf16_val(wg[k]), xv, acc[2 * m].x);
        acc[2 * m + 1].x = __fmaf_rn(bf16_val(wu[k]), xv, acc[2 * m + 1].x);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 2 * R; ++m) {
    float v = __fadd_rn(acc[m].x, acc[m].y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (lane == 0) s_part[warp][m] = v;
  }
  __syncthreads();
  if (part != 0 || f >= a.N || lane >= R) return;
  float g[1] = {0.f}, u[1] = {0.f};
  for (int k = 0; k < a.wpf; ++k) {
    g[0] = __fadd_rn(g[0], s_part[warp + k][2 * lane]);
    u[0] = __fadd_rn(u[0], s_part[warp + k][2 * lane + 1]);
  }
  gated_column<1>(a.out, lane, 1, 1, f, g, u);
}

template <int R>
cudaError_t few_rows(const GatedArgs& a, const GatedOut& out, cudaStream_t stream) {
  const bool vec = tma_rows(a.x, a.ldx) && tma_rows(a.w[0], a.ldw[0]) && tma_rows(a.w[1], a.ldw[1]);
  const bool even = rows4(a.x, a.ldx) && rows4(a.w[0], a.ldw[0]) && rows4(a.w[1], a.ldw[1]);
  // warps of a column: to 32 warps an SM, while each has a few whole loads of K
  const int64_t warps = (int64_t)sm_count() * 32, least = vec ? 512 : (even ? 128 : 64);
  int wpf = 1;
  while (wpf < FEW_T / 32 && a.N * wpf * 2 <= warps && a.K >= least * wpf * 2) wpf *= 2;
  FewRows p{static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.w[0]), static_cast<const uint16_t*>(a.w[1]), a.ldx,
            a.ldw[0], a.ldw[1], a.N, (int)a.K, wpf, out};
  const dim3 grid((unsigned)((a.N * wpf + FEW_T / 32 - 1) / (FEW_T / 32)));
  const auto kernel = vec ? gated_few_rows_kernel<R, 8> : (even ? gated_few_rows_kernel<R, 2> : gated_few_rows_kernel<R, 1>);
  const cudaError_t e = launch_after(kernel, grid, dim3(FEW_T), 0, stream, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------ dg and du
// act(z) and act'(z), to the bounds that the linear layer's have.
template <int ACT>
__device__ __forceinline__ void act_and_slope(float2 z, float2& value, float2& slope) {
  if (ACT == RLK_ACT_GELU) {
    float2 bell;
    const float2 tail = normal_tail(z, bell), phi = normal_below(z, tail);
    value = mul2(z, phi);
    slope = fma2(mul2(z, bell), both(0.39894228040143268f), phi);
  } else if (ACT == RLK_ACT_SILU) {
    const float2 s = logistic(z);
    value = mul2(z, s);
    slope = mul2(s, fma2(z, fma2(s, both(-1.f), both(1.f)), both(1.f)));
  } else if (ACT == RLK_ACT_RELU) {
    slope = activation_slope<RLK_ACT_RELU>(z);
    value = make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);
  } else {
    value = z;
    slope = both(1.f);
  }
}

// A thread takes W columns (8 where every row of the three inputs starts on a 16-byte
// boundary, else 1) of rows blockIdx.y, + parts, ..., DZ_ROWS of them in flight, and keeps
// their sums.  Bound by memory: 10 bytes an element.
constexpr int DT = 128, DZ_ROWS = 2;
template <int W, int ACT>
__global__ void __launch_bounds__(DT) gated_dz_kernel(GatedBwdArgs a, uint16_t* dg, uint16_t* du, int64_t ldd, float* db_part,
                                                      int64_t pitch, int parts) {
  const int64_t c = ((int64_t)blockIdx.x * DT + threadIdx.x) * W;
  if (c >= a.N) return;
  const uint16_t* in[3] = {static_cast<const uint16_t*>(a.dy) + c, static_cast<const uint16_t*>(a.z[0]) + c,
                           static_cast<const uint16_t*>(a.z[1]) + c};
  const int64_t ld[3] = {a.lddy, a.ldz[0], a.ldz[1]};
  const bool whole = W == 1 || c + W <= a.N;
  constexpr int H = (W + 1) / 2;
  float2 sum_g[H], sum_u[H];
#pragma unroll
  for (int j = 0; j < H; ++j) sum_g[j] = sum_u[j] = make_float2(0.f, 0.f);
  for (int64_t m0 = blockIdx.y; m0 < a.M; m0 += (int64_t)parts * DZ_ROWS) {
    uint32_t w[3][DZ_ROWS][H];
#pragma unroll
    for (int k = 0; k < DZ_ROWS; ++k) {
      const int64_t m = m0 + (int64_t)k * parts;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int j = 0; j < H; ++j) w[i][k][j] = 0u;
        if (m >= a.M) continue;
        const uint16_t* p = in[i] + m * ld[i];
        if (W == 8 && whole) {
          const uint4 q = *reinterpret_cast<const uint4*>(p);
          w[i][k][0] = q.x; w[i][k][H / 4] = q.y; w[i][k][H / 2] = q.z; w[i][k][H - 1] = q.w;
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j)
            if (c + j < a.N) w[i][k][j / 2] |= (uint32_t)p[j] << (16 * (j % 2));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < DZ_ROWS; ++k) {
      const int64_t m = m0 + (int64_t)k * parts;
      if (m >= a.M) continue;
      float g[2 * H], u[2 * H];
#pragma unroll
      for (int j = 0; j < H; ++j) {   // (W = 1: the pair's second is not used)
        float2 value, slope;
        act_and_slope<ACT>(bf16x2_to_f2(w[1][k][j]), value, slope);
        const float2 dy = bf16x2_to_f2(w[0][k][j]);
        const float2 x = mul2(mul2(dy, bf16x2_to_f2(w[2][k][j])), slope), y = mul2(dy, value);
        sum_g[j] = add2(sum_g[j], x);
        sum_u[j] = add2(sum_u[j], y);
        g[2 * j] = x.x;
        g[2 * j + 1] = x.y;
        u[2 * j] = y.x;
        u[2 * j + 1] = y.y;
      }
      if (!dg) continue;
      if constexpr (W == 8) {
        store8(dg + m * ldd + c, g, whole ? 8 : (int)(a.N - c));
        store8(du + m * ldd + c, u, whole ? 8 : (int)(a.N - c));
      } else {
        dg[m * ldd + c] = (uint16_t)pack_bf16(g[0], 0.f);
        du[m * ldd + c] = (uint16_t)pack_bf16(u[0], 0.f);
      }
    }
  }
  if (!db_part) return;
  float* to = db_part + (int64_t)blockIdx.y * 2 * pitch + c;   // a part: pitch of dg, pitch of du
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (c + j < a.N) {
      to[j] = j % 2 ? sum_g[j / 2].y : sum_g[j / 2].x;
      to[pitch + j] = j % 2 ? sum_u[j / 2].y : sum_u[j / 2].x;
    }
}

constexpr int kParts = 304;   // most row parts of the bias gradients
int64_t parts_most(int64_t M) {
  const int64_t p = (M + DZ_ROWS - 1) / DZ_ROWS;
  return p < kParts ? p : kParts;
}
size_t parts_bytes(int64_t M, int64_t N) { return pad256((size_t)parts_most(M) * 2 * pad8(N) * sizeof(float)); }

// Operands whose rows TMA cannot read are replaced by copies at *ws (advanced).
struct Copied {
  Operand* o;
  int64_t rows, cols;
};
cudaError_t aligned_operands(const Copied (&c)[3], char*& ws, cudaStream_t stream) {
  Repack r[3] = {};
  int n = 0;
  for (const Copied& i : c) {
    if (!i.o || tma_rows(i.o->p, i.o->ld)) continue;
    uint16_t* dst = reinterpret_cast<uint16_t*>(ws);
    ws += copy_bytes(i.rows, i.cols);
    r[n++] = Repack{static_cast<const uint16_t*>(i.o->p), i.o->ld, i.rows, i.cols, dst, pad8(i.cols)};
    *i.o = Operand{dst, pad8(i.cols)};
  }
  cudaError_t e = n > 0 ? launch_repack(r[0], r[1], stream) : cudaSuccess;
  if (e == cudaSuccess && n > 2) e = launch_repack(r[2], Repack{}, stream);
  return e;
}

}  // namespace

size_t gated_workspace_bytes(int64_t M, int64_t N, int64_t K) { return copy_bytes(M, K) + 2 * copy_bytes(N, K); }

size_t gated_workspace_needed(const GatedArgs& a) {
  if (a.M <= FEW_ROWS) return 0;
  size_t n = tma_rows(a.x, a.ldx) ? 0 : copy_bytes(a.M, a.K);
  for (int i = 0; i < 2; ++i) n += tma_rows(a.w[i], a.ldw[i]) ? 0 : copy_bytes(a.N, a.K);
  return n;
}

cudaError_t launch_gated_fwd(const GatedArgs& a, cudaStream_t stream) {
  GatedOut out{};
  for (int i = 0; i < 2; ++i) {
    out.bias[i] = a.bias[i];
    out.z[i] = static_cast<uint16_t*>(a.z[i]);
  }
  out.bias_dtype = a.bias_dtype;
  out.act = a.act;
  out.y = a.y;
  out.y_dtype = a.y_dtype;
  out.ldy = a.ldy;
  out.ldz = a.ldz;
  switch (a.M) {
    case 1: return few_rows<1>(a, out, stream);
    case 2: return few_rows<2>(a, out, stream);
    case 3: return few_rows<3>(a, out, stream);
    case FEW_ROWS: return few_rows<FEW_ROWS>(a, out, stream);
    default: break;
  }
  char* ws = static_cast<char*>(a.workspace);
  Operand x{a.x, a.ldx}, wg{a.w[0], a.ldw[0]}, wu{a.w[1], a.ldw[1]};
  if (cudaError_t e = aligned_operands({{&x, a.M, a.K}, {&wg, a.N, a.K}, {&wu, a.N, a.K}}, ws, stream); e != cudaSuccess) return e;
  const bool few = few_tiles(a.M, a.N, 1, 64);
  Maps maps{};
  const int a_rows = few && a.M < 128 ? (int)pad8(a.M) : 128;
  if (!gemm::make_map(&maps.a[0], false, x, false, a.M, a.K, a_rows) ||
      !gemm::make_map(&maps.b[0], false, wg, false, a.N, a.K, few ? 64 : 128) ||
      !gemm::make_map(&maps.b[1], false, wu, false, a.N, a.K, few ? 64 : 128))
    return cudaErrorInvalidValue;
  maps.a[1] = maps.a[0];
  ForwardOp::Params p{};
  p.M = a.M;
  p.N = a.N;
  p.loop.k_steps = (int)((a.K + gemm::BK - 1) / gemm::BK);
  p.loop.a_rows = a_rows;
  p.vec = rows16(a.y, a.y_dtype, a.ldy) && (!a.z[0] || (rows16(a.z[0], 0, a.ldz) && rows16(a.z[1], 0, a.ldz)));
  p.out = out;
  return run_tiles<ForwardOp>(maps, p, 1, 64, few, stream);
}

size_t gated_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return 2 * copy_bytes(M, N) + copy_bytes(M, K) + 2 * copy_bytes(N, K) + parts_bytes(M, N);
}

size_t gated_bwd_workspace_needed(const GatedBwdArgs& a) {
  size_t n = a.db[0] ? parts_bytes(a.M, a.N) : 0;
  if (a.dx || a.dw[0]) n += 2 * copy_bytes(a.M, a.N);
  for (int i = 0; i < 2; ++i)
    if (a.dx && !tma_rows(a.w[i], a.ldw[i])) n += copy_bytes(a.N, a.K);
  if (a.dw[0] && (a.ck.codes || !tma_rows(a.x, a.ldx))) n += copy_bytes(a.M, a.K);
  return n;
}

cudaError_t launch_gated_bwd(const GatedBwdArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.M == 0) {   // sums over no rows
    if (a.accumulate) return e;
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
      if (a.dw[i]) e = launch_zero(a.dw[i], a.dw_dtype, a.lddw[i], a.N, a.K, stream);
      if (e == cudaSuccess && a.db[i]) e = launch_zero(a.db[i], 1, a.N, 1, a.N, stream);
    }
    return e;
  }
  char* ws = static_cast<char*>(a.workspace);
  const bool products = a.dx || a.dw[0];
  const int64_t ldd = pad8(a.N);
  uint16_t* dz[2] = {nullptr, nullptr};
  for (int i = 0; i < 2 && products; ++i) {
    dz[i] = reinterpret_cast<uint16_t*>(ws);
    ws += copy_bytes(a.M, a.N);
  }
  float* part = nullptr;
  if (a.db[0]) {
    part = reinterpret_cast<float*>(ws);
    ws += parts_bytes(a.M, a.N);
  }
  {
    const bool vec = tma_rows(a.dy, a.lddy) && tma_rows(a.z[0], a.ldz[0]) && tma_rows(a.z[1], a.ldz[1]);
    const int64_t per = DT * (vec ? 8 : 1), cols = (a.N + per - 1) / per;
    int64_t parts = ((int64_t)sm_count() * 8 + cols - 1) / cols;   // about 8 CTAs an SM
    const int64_t most = parts_most(a.M);
    if (parts > most) parts = most;
    auto kernel = vec ? (a.act == RLK_ACT_GELU   ? gated_dz_kernel<8, RLK_ACT_GELU>
                         : a.act == RLK_ACT_SILU ? gated_dz_kernel<8, RLK_ACT_SILU>
                         : a.act == RLK_ACT_RELU ? gated_dz_kernel<8, RLK_ACT_RELU>
                                                 : gated_dz_kernel<8, RLK_ACT_NONE>)
                      : (a.act == RLK_ACT_GELU   ? gated_dz_kernel<1, RLK_ACT_GELU>
                         : a.act == RLK_ACT_SILU ? gated_dz_kernel<1, RLK_ACT_SILU>
                         : a.act == RLK_ACT_RELU ? gated_dz_kernel<1, RLK_ACT_RELU>
                                                 : gated_dz_kernel<1, RLK_ACT_NONE>);
    kernel<<<dim3((unsigned)cols, (unsigned)parts), DT, 0, stream>>>(a, dz[0], dz[1], ldd, part, ldd, (int)parts);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    for (int i = 0; i < 2 && a.db[0]; ++i)
      if ((e = launch_add_parts(part + i * ldd, 2 * ldd, (int)parts, a.N, a.db[i], a.accumulate, stream)) != cudaSuccess) return e;
  }
  if (!products) return e;
  Operand g{dz[0], ldd}, u{dz[1], ldd}, wg{a.w[0], a.ldw[0]}, wu{a.w[1], a.ldw[1]}, x{a.x, a.ldx};
  if ((e = aligned_operands({{a.dx ? &wg : nullptr, a.N, a.K}, {a.dx ? &wu : nullptr, a.N, a.K}, {a.dw[0] && a.x ? &x : nullptr, a.M, a.K}},
                            ws, stream)) != cudaSuccess)
    return e;
  Maps maps{};
  if (a.dx) {   // K runs over N twice; the weights [N][K] hold its columns contiguously
    using Op = StoreOp<false, true>;
    const bool few = few_tiles(a.M, a.K, 1, 128);
    const int a_rows = few && a.M < 128 ? (int)pad8(a.M) : 128;
    if (!gemm::make_map(&maps.a[0], false, g, false, a.M, a.N, a_rows) || !gemm::make_map(&maps.a[1], false, u, false, a.M, a.N, a_rows) ||
        !gemm::make_map(&maps.b[0], false, wg, true, a.K, a.N) || !gemm::make_map(&maps.b[1], false, wu, true, a.K, a.N))
      return cudaErrorInvalidValue;
    Op::Params p{};
    p.M = a.M;
    p.N = a.K;
    p.loop.part_steps = (int)((a.N + gemm::BK - 1) / gemm::BK);
    p.loop.k_steps = 2 * p.loop.part_steps;
    p.loop.a_rows = a_rows;
    p.vec = rows16(a.dx, a.dx_dtype, a.lddx);
    p.y_dtype = a.dx_dtype;
    p.out[0] = StoreOut{a.dx, a.lddx};
    if ((e = run_tiles<Op>(maps, p, 1, 128, few, stream)) != cudaSuccess) return e;
  }
  if (a.dw[0]) {   // K is M; every operand holds its rows' index contiguously
    if (!a.x) {    // the checkpoint's values are exact in bf16
      CheckpointArgs c{};
      c.x = ws;
      c.T = a.M;
      c.H = a.K;
      c.ldx = pad8(a.K);
      c.ck = a.ck;
      if ((e = launch_checkpoint_unpack(c, stream)) != cudaSuccess) return e;
      x = Operand{ws, pad8(a.K)};
    }
    using Op = StoreOp<true, false>;
    if (!gemm::make_map(&maps.a[0], false, g, true, a.N, a.M) || !gemm::make_map(&maps.a[1], false, u, true, a.N, a.M) ||
        !gemm::make_map(&maps.b[0], false, x, true, a.K, a.M))
      return cudaErrorInvalidValue;
    maps.b[1] = maps.b[0];
    Op::Params p{};
    p.M = a.N;
    p.N = a.K;
    p.loop.k_steps = (int)((a.M + gemm::BK - 1) / gemm::BK);
    p.vec = rows16(a.dw[0], a.dw_dtype, a.lddw[0]) && rows16(a.dw[1], a.dw_dtype, a.lddw[1]);
    p.y_dtype = a.dw_dtype;
    p.accumulate = a.accumulate;
    for (int i = 0; i < 2; ++i) p.out[i] = StoreOut{a.dw[i], a.lddw[i]};
    e = run_tiles<Op>(maps, p, 2, 128, few_tiles(p.M, p.N, 2, 128), stream);
  }
  return e;
}

}  // namespace rlk
