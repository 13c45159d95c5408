// rlk_linear_fwd / rlk_linear_bwd: matrix products with a fused epilogue.
//
//   forward   z = x w^T + bias,  y = act(z) + residual
//   backward  dz = dy act'(z),  dx = dz w,  dw = dz^T x,  db = sum_m dz
//
// All three products are one kernel, D[M, N] = sum_k A[m, k] B[n, k], whose
// operands may each be stored with K or with M / N contiguous, so neither w nor
// x nor dz is transposed in memory.  bf16 operands arrive by TMA (128-byte
// swizzle) in a ring of 64-deep stages, one thread issues the tcgen05 MMAs
// (fp32 accumulators in TMEM), the other warps run the epilogue on registers read
// with tcgen05.ld.
//  * Many tiles: persistent pairs of CTAs (cta_group::2), a tile of 256 x 256 a
//    pair: each SM stages half of A's and half of B's rows, half the shared-memory
//    traffic of two separate tiles.  Two TMEM accumulators, so a tile's
//    epilogue runs under the next tile's products.  Tiles are walked in groups
//    of 8 row tiles, so the pairs at work share 8 A tiles and about 10 B tiles
//    in L2.
//  * Few tiles (a call of few rows is bound by the weight's bytes, and needs
//    every SM to fetch them): tiles of 128 x 128, and a cluster of 2 or 4 CTAs
//    splits K, leaves its partial tiles in shared memory, and each CTA adds the
//    cluster's partials in rank order for its share of the columns.
// TMA needs rows that start on 16-byte boundaries; an operand whose rows do not
// is first copied into the workspace.
//
// The epilogue's arithmetic is fp32 and y, z, dx, dw are rounded once.  dz is
// rounded to bf16 before its two products, since the tensor cores take no wider
// operand beside a bf16 one (two bf16 halves of dz would double the products' time):
// up to a relative 2^-8 of each term, as much as a bf16 dw's own rounding and far above an
// fp32 one's, but of either sign, so a sum of many terms keeps less of it.  Against 64
// bits dx and dw of 8192 x 4096 x 4096 in bf16 are off by 0.0024 (root mean square), where
// products of an unrounded dz give 0.0017.  db sums dz unrounded.
// Every wait is bounded; when one runs out the CTA's unfinished tiles are NaN.
//
// Measured: 16384 x 4096 x 4096 with bias, GELU, residual and z 337 us, 1630 TFLOP/s
// (tensor pipe 79 % of its cycles); backward of 8192 x 4096 x 4096:
// dx 154 us (87 %), dw 171 us (84 %: 256 tiles on 76
// pairs are 3.4 rounds, and 4 are taken), dz and db 30 and 7 us.

#include <math.h>

#include <atomic>

#include "checkpoint.cuh"
#include "internal.h"
#include "rlk.h"
#include "tensor_core.cuh"

namespace rlk {
namespace {

constexpr int BM = 128, BK = 64;
constexpr uint32_t MN_BLOCK = 64 * BK * 2;     // a 64-element block of an MN-contiguous operand
constexpr uint32_t STAGING = 32 * 32 * 4;      // an epilogue warp's 32 x 32 piece of a tile
constexpr int GROUP_M = 8;
constexpr int MAX_SPLIT = 4;                   // CTAs that share a tile's K, at most
// The two shapes.  A pair of CTAs (one tile of 256 x 256, 128 rows of A and of B
// each; five stages, one CTA an SM), or one CTA (a tile of 128 x 128, its K perhaps split
// over a cluster; a single accumulator; six stages, or three where there are more
// CTAs than SMs, so that two share an SM and one's epilogue runs beside the other's
// products).  The pair's 16 epilogue warps take the sixth stage's room: with eight,
// and six stages, products of a short K waited on the epilogue (16384 x 4096 x 512
// with GELU 138 us against 98, 102 with the GELU of now; K 4096 the same within its noise).
constexpr int BROWS = 128;
constexpr uint32_t A_BYTES = BM * BK * 2, STAGE_BYTES = A_BYTES + BROWS * BK * 2;
template <bool SPLIT>
struct Shape {
  static constexpr int G = SPLIT ? 1 : 2;      // CTAs of a tile
  static constexpr int EPI_WARPS = SPLIT ? 8 : 16, THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int STAGES = SPLIT ? 6 : 5; // at most
  static constexpr int TM = BM * G, BN = BROWS * G;
  static constexpr uint32_t TMEM_COLS = SPLIT ? BN : 2 * BN;
  static constexpr int PLD = BN + 4;           // row pitch (floats) of a partial tile: conflict-free float4 rows
  static constexpr uint32_t STAGED = SPLIT ? 0 : EPI_WARPS * STAGING;
  static constexpr size_t smem(int stages) { return stages * STAGE_BYTES + STAGED + 1024 + 256; }
};
constexpr int MAX_STAGES = 6, FEW_STAGES = 3;
static_assert(BM * Shape<true>::PLD * 4 <= FEW_STAGES * STAGE_BYTES, "a partial tile fits into the ring");

struct Epilogue {
  const void* bias;
  int bias_dtype;
  const uint16_t* residual;
  int64_t ldr;
  int act;
  void* y;
  int y_dtype;         // 0 bf16, 1 fp32
  int64_t ldy;
  uint16_t* z;
  int64_t ldz;
  int accumulate;      // y (fp32) is added to
  int vec;             // rows of y, z and residual start on 16-byte boundaries
  int even;            // they start on 4-byte boundaries, and N is even
};
struct GemmParams {
  int64_t M, N;
  int n_mt, n_nt, k_steps;
  int n_tiles;               // n_mt x n_nt
  int stages;
  long long wait_limit;
  int withhold;              // debug: the stage of the first CTA whose barrier waits for an arrival that never comes (-1: none)
  Epilogue e;
};

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

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The epilogue of 8 columns of one row whose y, z and residual start on 16-byte
// boundaries there; n of the columns exist.
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
__device__ __forceinline__ float bias_at(const Epilogue& e, int64_t col) {
  return e.bias_dtype ? static_cast<const float*>(e.bias)[col] : bf16_val(static_cast<const uint16_t*>(e.bias)[col]);
}
__device__ __forceinline__ uint4 residual8(const Epilogue& e, int64_t row, int64_t col, int n) {
  const uint16_t* r = e.residual + row * e.ldr + col;
  if (n == 8) return *reinterpret_cast<const uint4*>(r);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j / 2] |= (uint32_t)r[j] << (16 * (j % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void finish8(const Epilogue& e, int64_t row, int64_t col, int n, float (&v)[8],
                                        const float (&bias)[8], uint4 res) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 o = add2(make_float2(v[j], v[j + 1]), make_float2(bias[j], bias[j + 1]));
    v[j] = o.x;
    v[j + 1] = o.y;
  }
  if (e.z) store8(e.z + row * e.ldz + col, v, n);
  activate(v, e.act);
  if (e.residual) {
    const uint32_t w[4] = {res.x, res.y, res.z, res.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 o = add2(make_float2(v[2 * k], v[2 * k + 1]), bf16x2_to_f2(w[k]));
      v[2 * k] = o.x;
      v[2 * k + 1] = o.y;
    }
  }
  if (e.y_dtype == 0) {
    store8(static_cast<uint16_t*>(e.y) + row * e.ldy + col, v, n);
    return;
  }
  float* y = static_cast<float*>(e.y) + row * e.ldy + col;
  if (n == 8) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float4 o = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      if (e.accumulate) {
        const float4 old = reinterpret_cast<const float4*>(y)[k];
        o = make_float4(__fadd_rn(old.x, o.x), __fadd_rn(old.y, o.y), __fadd_rn(old.z, o.z), __fadd_rn(old.w, o.w));
      }
      reinterpret_cast<float4*>(y)[k] = o;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) y[j] = e.accumulate ? __fadd_rn(y[j], v[j]) : v[j];
  }
}
// W columns (1, or 2 at an even place of rows that start on 4-byte boundaries) of R
// rows, `step` apart from `row` on; those up to n rows from `row` exist.
template <int R, int W>
__device__ __forceinline__ void finish_rows(const Epilogue& e, int64_t row, int step, int n, int64_t col, float (&v)[R * W],
                                            const float (&bias)[W], const uint32_t (&res)[R]) {
#pragma unroll
  for (int k = 0; k < R * W; ++k) v[k] = __fadd_rn(v[k], bias[k % W]);
  auto store = [&](uint16_t* p, int64_t ld) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (k * step >= n) continue;
      if (W == 2) *reinterpret_cast<uint32_t*>(p + k * step * ld) = pack_bf16(v[k * W], v[k * W + W - 1]);
      else p[k * step * ld] = (uint16_t)pack_bf16(v[k * W], 0.f);
    }
  };
  if (e.z) store(e.z + row * e.ldz + col, e.ldz);
  activate(v, e.act);
  if (e.residual) {
#pragma unroll
    for (int k = 0; k < R * W; ++k) v[k] = __fadd_rn(v[k], k % W ? bf16_hi(res[k / W]) : bf16_lo(res[k / W]));
  }
  if (e.y_dtype == 0) {
    store(static_cast<uint16_t*>(e.y) + row * e.ldy + col, e.ldy);
  } else {
    float* y = static_cast<float*>(e.y) + row * e.ldy + col;
#pragma unroll
    for (int k = 0; k < R * W; ++k) {
      float* q = y + (k / W) * step * e.ldy + k % W;
      if ((k / W) * step < n) *q = e.accumulate ? __fadd_rn(*q, v[k]) : v[k];
    }
  }
}
template <int R, int W>
__device__ __forceinline__ void residual_rows(const Epilogue& e, int64_t row, int step, int n, int64_t col,
                                              uint32_t (&res)[R]) {
  const uint16_t* p = e.residual + row * e.ldr + col;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    res[k] = 0u;
    if (e.residual && k * step < n)
      res[k] = W == 2 ? *reinterpret_cast<const uint32_t*>(p + k * step * e.ldr) : p[k * step * e.ldr];
  }
}
// The epilogue warp's 32 x 32 piece in `st`, W columns a lane (32 / W lanes share a
// row): consecutive lanes share lines whatever the rows' alignment.
template <int W>
__device__ __forceinline__ void finish_piece(const Epilogue& e, const float* st, int64_t row0, int rows, int64_t col0,
                                             int64_t N) {
  constexpr int R = 8;
  const int lane = threadIdx.x & 31, c = lane % (32 / W) * W, sub = lane / (32 / W);
  if (col0 + c >= N) return;
  float bias[W];
#pragma unroll
  for (int k = 0; k < W; ++k) bias[k] = e.bias ? bias_at(e, col0 + c + k) : 0.f;
  uint32_t next[R], res[R];   // the residual of the next rows is on its way
  residual_rows<R, W>(e, row0 + sub, W, rows - sub, col0 + c, next);
#pragma unroll 1
  for (int r0 = sub; r0 < rows; r0 += R * W) {
    float o[R * W];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      res[k] = next[k];
      const int r = r0 + k * W;
      const float* q = st + r * 32 + (((c >> 2) ^ (r & 7)) << 2) + (c & 3);
#pragma unroll
      for (int u = 0; u < W; ++u) o[k * W + u] = q[u];
    }
    residual_rows<R, W>(e, row0 + r0 + R * W, W, rows - r0 - R * W, col0 + c, next);
    finish_rows<R, W>(e, row0 + r0, W, rows - r0, col0 + c, o, bias, res);
  }
}

// Tile t -> (row tile, column tile): groups of GROUP_M row tiles, row tiles
// fastest inside a group.
__device__ __forceinline__ void tile_coords(const GemmParams& p, int t, int& mt, int& nt) {
  const int group = t / (GROUP_M * p.n_nt), r = t - group * GROUP_M * p.n_nt;
  const int g0 = group * GROUP_M, gm = p.n_mt - g0 < GROUP_M ? p.n_mt - g0 : GROUP_M;
  mt = g0 + r % gm;
  nt = r / gm;
}

// SPLIT: a cluster of CTAs works on one tile of 128 x 128, each on its share of
// K; else pair b works on tiles b, + the number of pairs, ... of 256 x 256.
template <bool A_MN, bool B_MN, bool SPLIT>
__global__ void __launch_bounds__(Shape<SPLIT>::THREADS, SPLIT ? 2 : 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const GemmParams p, int cluster) {
  using S = Shape<SPLIT>;
  constexpr int G = S::G, TM = S::TM, BN = S::BN, PLD = S::PLD, EPI_WARPS = S::EPI_WARPS;
  const int stages = SPLIT ? p.stages : S::STAGES;
  const uint32_t ring = stages * STAGE_BYTES;
  constexpr uint32_t TMEM_COLS = S::TMEM_COLS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  float* staging = reinterpret_cast<float*>(base_ptr + ring);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base_ptr + ring + S::STAGED);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * MAX_STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * MAX_STAGES + 5);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * MAX_STAGES;
  const uint32_t accf0 = empty0 + 8 * MAX_STAGES, acce0 = accf0 + 16;
  const uint32_t drain_bar = smem_u32(bars + 2 * MAX_STAGES + 6);
  constexpr uint32_t idesc = tc::idesc_bf16(A_MN, B_MN, TM, BN);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, 1 + (s == p.withhold && blockIdx.x == 0));
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf0 + 8 * a, 1);
      mbar_init(acce0 + 8 * a, EPI_WARPS * G);   // one arrive per epilogue warp of the tile's CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tc::prefetch_map(&map_a);
    tc::prefetch_map(&map_b);
  }
  if (warp == 1) tc::alloc<G>(smem_u32(tmem_slot), TMEM_COLS);
  tc::fence_before();
  pdl_wait();   // the operands may come from the kernel before
  __syncthreads();
  if (G == 2) tc::cluster_sync();   // the other CTA's barriers are there
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  // SPLIT: which share of K; else: which half of the tile
  const uint32_t rank = tc::cluster_rank();
  const int per = SPLIT ? cluster : G;   // CTAs that work on one tile
  const int tile0 = (int)(blockIdx.x / (unsigned)per);
  const int tile_step = SPLIT ? p.n_tiles : (int)(gridDim.x / G);
  const int k0 = SPLIT ? (int)((int64_t)rank * p.k_steps / cluster) : 0;
  const int k1 = SPLIT ? (int)((int64_t)(rank + 1) * p.k_steps / cluster) : p.k_steps;
  const int a_off = SPLIT ? 0 : (int)rank * BM, b_off = SPLIT ? 0 : (int)rank * BROWS;
  const bool leader = SPLIT || rank == 0;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, used = 0u, last_parity = 0u;   // per stage: issued at all, parity of the last issue
      bool ok = true;
      for (int t = tile0; t < p.n_tiles && ok; t += tile_step) {
        int mt, nt;
        tile_coords(p, t, mt, nt);
        for (int k = k0; k < k1; ++k) {
          if (!tc::wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.wait_limit) || *abort_flag) {
            ok = false;
            break;
          }
          const uint32_t fb = full0 + 8 * stage;
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES;
          // a pair's copies all report to the even CTA, whose barrier expects them all
          if (leader) mbar_expect_tx(fb, G * STAGE_BYTES);
          const uint32_t to = G == 2 ? tc::peer_addr(fb, 0u) : fb;
          auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
            if (G == 2) tc::load_2d_pair(dst, map, to, x, y);
            else tc::load_2d(dst, map, to, x, y);
          };
          const int am = mt * TM + a_off, bn = nt * BN + b_off;
          if (A_MN) {
#pragma unroll
            for (int j = 0; j < BM / 64; ++j) load(sa + j * MN_BLOCK, &map_a, am + j * 64, k * BK);
          } else {
            load(sa, &map_a, k * BK, am);
          }
          if (B_MN) {
#pragma unroll
            for (int j = 0; j < BROWS / 64; ++j) load(sb + j * MN_BLOCK, &map_b, bn + j * 64, k * BK);
          } else {
            load(sb, &map_b, k * BK, bn);
          }
          used |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
      }
      // Every copy lands before the CTAs exit (bounded), also when another role's wait runs
      // out only after the last copy was asked for.  (A pair's odd CTA may have asked for
      // stages that the even one no longer did; after that its own roles wait out the limit.)
      if (leader)
        for (int s = 0; s < stages; ++s)
          if (used & (1u << s)) tc::drain(full0 + 8 * s, (last_parity >> s) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0, tile = 0;
      bool ok = true;
      for (int t = tile0; t < p.n_tiles && ok; t += tile_step, ++tile) {
        const uint32_t acc = tile & 1u, accph = (tile >> 1) & 1u;
        if (!tc::wait<G == 2>(acce0 + 8 * acc, accph ^ 1u, abort_flag, p.wait_limit)) { ok = false; break; }
        tc::fence_after();
        const uint32_t d_tmem = tmem + acc * BN;
        for (int k = k0; k < k1; ++k) {
          if (!tc::wait(full0 + 8 * stage, phase, abort_flag, p.wait_limit)) { ok = false; break; }
          tc::fence_after();
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            // 16 K elements: 32 bytes inside a K-contiguous row, 16 rows of an MN-contiguous block
            const uint64_t da = A_MN ? tc::desc_mn(sa + kk * 2048, MN_BLOCK) : tc::desc_k(sa) + (uint64_t)(kk * 2);
            const uint64_t db = B_MN ? tc::desc_mn(sb + kk * 2048, MN_BLOCK) : tc::desc_k(sb) + (uint64_t)(kk * 2);
            tc::mma<G>(d_tmem, da, db, idesc, (k > k0 || kk > 0) ? 1u : 0u);
          }
          tc::commit<G>(empty0 + 8 * stage);
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (ok) tc::commit<G>(accf0 + 8 * acc);
      }
      if (!ok) {   // every MMA already issued finishes before TMEM is freed
        tc::commit<G>(drain_bar);
        tc::drain(drain_bar, 0u);
      }
    }
  } else {
    // ------------------------------------------------------ epilogue
    // Two warps (a pair's tile: four) a TMEM quadrant (32 rows), each with its share of
    // the columns, 32 at a time: tcgen05.ld gives a thread 32 columns of one row; a turn through the
    // warp's staging (16-byte units, swizzled: no bank conflicts) gives it 8
    // columns of 4 rows, so that a warp reads and writes whole 64-byte pieces of 8 rows.
    constexpr int PARTS = EPI_WARPS / 4, WIDTH = BN / PARTS;
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    float* st = staging + (warp - 2) * (STAGING / 4);
    uint32_t tile = 0;
    bool ok = true;
    for (int t = tile0; t < p.n_tiles; t += tile_step, ++tile) {
      int mt, nt;
      tile_coords(p, t, mt, nt);
      const uint32_t acc = tile & 1u, accph = (tile >> 1) & 1u;
      if (p.e.residual) {   // on its way to L2 while the products run: the lines of a row that hold this warp's columns
        const int64_t r = (int64_t)mt * TM + a_off + q * 32 + lane, c = (int64_t)nt * BN + part * WIDTH;
        if (r < p.M) {
#pragma unroll
          for (int k = 0; k <= WIDTH / 64; ++k) {
            const int64_t at = c + (k < WIDTH / 64 ? k * 64 : WIDTH - 1);
            if (at < p.N) prefetch_l2(p.e.residual + r * p.e.ldr + at);
          }
        }
      }
      // after a wait has run out, this tile and the CTA's later ones are NaN
      ok = __all_sync(0xFFFFFFFFu, ok && tc::wait(accf0 + 8 * acc, accph, abort_flag, p.wait_limit));
      tc::fence_after();
      const int64_t row0 = (int64_t)mt * TM + a_off + q * 32;
#pragma unroll 1
      for (int ch = 0; ch < WIDTH / 32; ++ch) {
        const int c0 = part * WIDTH + ch * 32;
        const int64_t col0 = (int64_t)nt * BN + c0;
        const int sub = lane & 3, r8 = lane >> 2;           // 8 columns, one of 8 rows
        const int64_t col = col0 + sub * 8;
        const int n = (int)(p.N - col < 8 ? (p.N - col > 0 ? p.N - col : 0) : 8);
        uint4 res[4];
        float bias[8];
        if (!SPLIT && p.e.vec) {                             // these loads run under the wait below
#pragma unroll
          for (int it = 0; it < 4; ++it)
            if (p.e.residual && n > 0 && row0 + it * 8 + r8 < p.M)
              res[it] = residual8(p.e, row0 + it * 8 + r8, col, n);
#pragma unroll
          for (int j = 0; j < 8; ++j) bias[j] = p.e.bias && j < n ? bias_at(p.e, col + j) : 0.f;
        }
        float v[32];
        if (ok) {
          tc::ld32(tmem + lane_base + acc * BN + c0, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = NAN;
        }
        if (ch == WIDTH / 32 - 1) {   // the accumulator is in registers: its next tile may begin
          tc::fence_before();
          __syncwarp();
          if (lane == 0 && ok) {
            if (G == 2) tc::arrive_peer(tc::peer_addr(acce0 + 8 * acc, 0u));
            else mbar_arrive(acce0 + 8 * acc);
          }
        }
        if (SPLIT) {
          if (row0 + lane < p.M && col0 < p.N) {
            float* own = reinterpret_cast<float*>(base_ptr) + (q * 32 + lane) * PLD + c0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              reinterpret_cast<float4*>(own)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
          continue;
        }
        if (col0 >= p.N) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          reinterpret_cast<float4*>(st + lane * 32)[j ^ (lane & 7)] =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        __syncwarp();
        if (p.e.vec) {
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int r = it * 8 + r8;
            const float4* src = reinterpret_cast<const float4*>(st + r * 32);
            const float4 a = src[(2 * sub) ^ (r & 7)], b = src[(2 * sub + 1) ^ (r & 7)];
            float o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            if (row0 + r < p.M && n > 0) finish8(p.e, row0 + r, col, n, o, bias, res[it]);
          }
        } else {
          const int rows = (int)(p.M - row0 < 32 ? p.M - row0 : 32);
          if (p.e.even) finish_piece<2>(p.e, st, row0, rows, col0, p.N);
          else finish_piece<1>(p.e, st, row0, rows, col0, p.N);
        }
        __syncwarp();
      }
    }
  }
  if (SPLIT) {
    __syncwarp();
    tc::cluster_sync();   // every partial tile is in its CTA's shared memory
    bool dead = false;    // a wait of some CTA of the cluster ran out
    const uint32_t abort_at = smem_u32(bars + 2 * MAX_STAGES + 4);
    for (int k = 0; k < cluster; ++k) dead = tc::ld_peer_u32(tc::peer_addr(abort_at, (uint32_t)k)) != 0u || dead;
    // this CTA's share of the columns, all rows
    int mt, nt;
    tile_coords(p, tile0, mt, nt);
    const int width = BN / cluster, c0 = (int)rank * width;
    const int64_t row0 = (int64_t)mt * BM, col0 = (int64_t)nt * BN + c0;
    const int rows = (int)(p.M - row0 < BM ? p.M - row0 : BM);
    if (p.e.vec) {
      const int octs = width / 8;
      for (int i = threadIdx.x; i < rows * octs; i += Shape<SPLIT>::THREADS) {
        const int r = i / octs, c = (i - r * octs) * 8;
        const int64_t col = col0 + c;
        if (col >= p.N) continue;
        const int n = (int)(p.N - col < 8 ? p.N - col : 8);
        uint4 res = make_uint4(0u, 0u, 0u, 0u);
        if (p.e.residual) res = residual8(p.e, row0 + r, col, n);
        float bias[8], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          bias[j] = p.e.bias && j < n ? bias_at(p.e, col + j) : 0.f;
          v[j] = 0.f;
        }
        const uint32_t at = base + (uint32_t)(r * PLD + c0 + c) * 4u;
        float4 part[2 * MAX_SPLIT];   // all in flight together
#pragma unroll
        for (int k = 0; k < MAX_SPLIT; ++k)
          if (k < cluster) {
            const uint32_t peer = tc::peer_addr(at, (uint32_t)k);
            part[2 * k] = tc::ld_peer4(peer);
            part[2 * k + 1] = tc::ld_peer4(peer + 16u);
          }
#pragma unroll
        for (int k = 0; k < MAX_SPLIT; ++k)
          if (k < cluster) {
            const float4 a = part[2 * k], b = part[2 * k + 1];
            const float o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], o[j]);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = dead ? NAN : v[j];
        finish8(p.e, row0 + r, col, n, v, bias, res);
      }
    } else {
      // a column a thread, 8 rows at a time
      constexpr int T = 256, R = 8;
      const int c = (int)threadIdx.x & (width - 1), step = T / width;
      const int64_t col = col0 + c;
      if (threadIdx.x < T && col < p.N) {
        const float bias[1] = {p.e.bias ? bias_at(p.e, col) : 0.f};
        for (int r0 = (int)threadIdx.x / width; r0 < rows; r0 += step * R) {
          uint32_t res[R];
          residual_rows<R, 1>(p.e, row0 + r0, step, rows - r0, col, res);
          float v[R];
#pragma unroll
          for (int k = 0; k < R; ++k) v[k] = 0.f;
          for (int q = 0; q < cluster; ++q) {
            const uint32_t peer = tc::peer_addr(base + (uint32_t)(r0 * PLD + c0 + c) * 4u, (uint32_t)q);
            float part[R];   // in flight together
#pragma unroll
            for (int k = 0; k < R; ++k)
              part[k] = r0 + k * step < rows ? tc::ld_peer_f32(peer + (uint32_t)(k * step * PLD) * 4u) : 0.f;
#pragma unroll
            for (int k = 0; k < R; ++k) v[k] = __fadd_rn(v[k], part[k]);
          }
#pragma unroll
          for (int k = 0; k < R; ++k) v[k] = dead ? NAN : v[k];
          finish_rows<R, 1>(p.e, row0 + r0, step, rows - r0, col, v, bias, res);
        }
      }
    }
    tc::cluster_sync();   // no CTA leaves while its shared memory is read
  }
  tc::fence_before();
  __syncthreads();
  if (G == 2) tc::cluster_sync();   // the pair's products, copies and arrivals are all done
  tc::fence_after();
  if (warp == 1) tc::dealloc<G>(tmem, TMEM_COLS);
}

// ------------------------------------------------------------ a few rows
// Up to GEMV_ROWS rows: the weight's bytes bound the call and a tile of 128
// rows would be almost empty, so each output feature is a dot product of its
// own (4 rows of 4096 x 4096: 12.7 us; 5 by tiles 14.4.  On 2-byte rows, where tiles
// need a copy first, 22 and 35).  `wpf` warps share a feature (each takes a run of
// K), as many as it takes to give every SM 32 warps (40: 11.1 us for one row of
// 2560 x 7488, 32: 9.3).  Their sums are joined in a fixed order.
// A load takes W columns: 8 where the rows of x and w start on 16-byte boundaries,
// 2 where they do on 4-byte ones, else 1; up to 16 of them are in flight a lane, at
// distances known when this is compiled (computed ones, and bounds tested at each load:
// 9.1 us for one row of 4096 x 4096, now 7.6; 75 us for 4 rows of 2560 x 7490, now 23).
constexpr int GEMV_ROWS = 4, GEMV_T = 256;

// W bf16 columns as they lie in memory, and as floats.
template <int W>
struct Cols;
template <>
struct Cols<8> {
  using type = uint4;
  static __device__ __forceinline__ void floats(uint4 q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(u[j]);
      v[2 * j + 1] = bf16_hi(u[j]);
    }
  }
};
template <>
struct Cols<2> {
  using type = uint32_t;
  static __device__ __forceinline__ void floats(uint32_t q, float (&v)[2]) {
    v[0] = bf16_lo(q);
    v[1] = bf16_hi(q);
  }
};
template <>
struct Cols<1> {
  using type = uint16_t;
  static __device__ __forceinline__ void floats(uint16_t q, float (&v)[1]) { v[0] = bf16_val(q); }
};

template <int R, int W>
__global__ void __launch_bounds__(GEMV_T, 4) linear_gemv_kernel(const uint16_t* x, int64_t ldx, const uint16_t* w,
                                                             int64_t ldw, int64_t N, int K, int wpf, Epilogue e) {
  pdl_wait();
  __shared__ float s_part[GEMV_T / 32][R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & (wpf - 1);
  const int64_t f = (int64_t)blockIdx.x * (GEMV_T / 32 / wpf) + warp / wpf;
  float acc[R];
#pragma unroll
  for (int m = 0; m < R; ++m) acc[m] = 0.f;
  if (f < N) {
    const uint16_t* wf = w + f * ldw;
    using T = typename Cols<W>::type;
    constexpr int U = W == 8 ? (R == 1 ? 8 : 4) : 16, STEP = 32 * W;
    const int share = (K + wpf * STEP - 1) / (wpf * STEP) * STEP, k1 = K / W * W;   // a warp's columns: whole loads
    const int end = min(k1, (part + 1) * share);
    constexpr int B = W == 8 ? 1 : 8;   // loads of a row of x together
    auto add = [&](const T* a, const uint16_t* xk) {
#pragma unroll
      for (int m = 0; m < R; ++m) {
        T b[B];
#pragma unroll
        for (int u = 0; u < B; ++u) b[u] = *reinterpret_cast<const T*>(xk + m * ldx + u * STEP);
#pragma unroll
        for (int u = 0; u < B; ++u) {
          float av[W], bv[W];
          Cols<W>::floats(a[u], av);
          Cols<W>::floats(b[u], bv);
#pragma unroll
          for (int j = 0; j < W; ++j) acc[m] = __fmaf_rn(av[j], bv[j], acc[m]);
        }
      }
    };
    int k0 = part * share + lane * W;
    for (; k0 - lane * W + STEP * U <= end; k0 += STEP * U) {   // U loads of every lane's, at fixed distances
      T a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) a[u] = __ldcs(reinterpret_cast<const T*>(wf + k0 + u * STEP));
#pragma unroll
      for (int u = 0; u < U; u += B) add(a + u, x + k0 + u * STEP);
    }
    T a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) a[u] = k0 + u * STEP < end ? __ldcs(reinterpret_cast<const T*>(wf + k0 + u * STEP)) : T{};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * STEP >= end) continue;
      float av[W], bv[W];
      Cols<W>::floats(a[u], av);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        Cols<W>::floats(*reinterpret_cast<const T*>(x + m * ldx + k0 + u * STEP), bv);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[m] = __fmaf_rn(av[j], bv[j], acc[m]);
      }
    }
    const int k = K / W * W + lane;   // the last K % W columns
    if (part == 0 && k < K) {
#pragma unroll
      for (int m = 0; m < R; ++m) acc[m] = __fmaf_rn(bf16_val(wf[k]), bf16_val(x[m * ldx + k]), acc[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < R; ++m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[m] = __fadd_rn(acc[m], __shfl_xor_sync(0xFFFFFFFFu, acc[m], o));
    if (lane == 0) s_part[warp][m] = acc[m];
  }
  __syncthreads();
  if (part != 0 || f >= N || lane >= R) return;
  float v[1] = {0.f};
  for (int k = 0; k < wpf; ++k) v[0] = __fadd_rn(v[0], s_part[warp + k][lane]);
  uint32_t res[1];
  residual_rows<1, 1>(e, lane, 1, 1, f, res);
  const float bias[1] = {e.bias ? bias_at(e, f) : 0.f};
  finish_rows<1, 1>(e, lane, 1, 1, f, v, bias, res);
}

// ------------------------------------------------------------ around the products
constexpr int ET = 256;

// bf16 matrices copied to rows that start on 16-byte boundaries: a warp a row, 8
// columns a lane.
struct Repack {
  const uint16_t* src;
  int64_t ld, rows, cols;
  uint16_t* dst;
  int64_t ldd;
};
__global__ void __launch_bounds__(ET) repack_kernel(Repack a, Repack b) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  for (int64_t r = (int64_t)blockIdx.x * (ET / 32) + (threadIdx.x >> 5); r < a.rows + b.rows;
       r += (int64_t)gridDim.x * (ET / 32)) {
    const bool first = r < a.rows;
    const int64_t row = first ? r : r - a.rows, cols = first ? a.cols : b.cols;
    const uint16_t* src = first ? a.src + row * a.ld : b.src + row * b.ld;
    uint16_t* dst = first ? a.dst + row * a.ldd : b.dst + row * b.ldd;
#pragma unroll 2
    for (int64_t c = lane * 8; c < cols; c += 256) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};   // columns past the end are filled with zeros
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) w[j / 2] |= (uint32_t)src[c + j] << (16 * (j % 2));
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// dz = dy act'(z) as bf16 and the partial column sums of the unrounded dz: part
// blockIdx.y takes rows blockIdx.y, + parts, ...  W = 8 columns a thread where
// the rows of dy and z start on 16-byte boundaries (dz's do), else 1; DZ_ROWS rows in
// flight.  Bound by memory (6 bytes an element): 30 us on 8192 x 4096 with SiLU.
constexpr int DT = 128, DZ_ROWS = 4;

template <int W, int ACT>
__global__ void __launch_bounds__(DT) linear_dz_kernel(LinearBwdArgs a, uint16_t* dz, int64_t ldd, float* db_part,
                                                       int64_t pitch, int parts) {
  const int64_t c = ((int64_t)blockIdx.x * DT + threadIdx.x) * W;
  if (c >= a.N) return;
  const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + c;
  const uint16_t* z = static_cast<const uint16_t*>(a.z) + c;
  const bool whole = W == 1 || c + W <= a.N;
  constexpr bool act = ACT != RLK_ACT_NONE;
  float sum[W];
#pragma unroll
  for (int j = 0; j < W; ++j) sum[j] = 0.f;
  for (int64_t m0 = blockIdx.y; m0 < a.M; m0 += (int64_t)parts * DZ_ROWS) {
    uint32_t g[DZ_ROWS][(W + 1) / 2], zz[DZ_ROWS][(W + 1) / 2];
#pragma unroll
    for (int k = 0; k < DZ_ROWS; ++k) {
      const int64_t m = m0 + (int64_t)k * parts;
#pragma unroll
      for (int j = 0; j < (W + 1) / 2; ++j) g[k][j] = zz[k][j] = 0u;
      if (m >= a.M) continue;
      if (W == 8 && whole) {
        const uint4 u = *reinterpret_cast<const uint4*>(dy + m * a.lddy);
        g[k][0] = u.x; g[k][W / 8] = u.y; g[k][W / 4] = u.z; g[k][W / 2 - W / 8] = u.w;
        if (act) {
          const uint4 v = *reinterpret_cast<const uint4*>(z + m * a.ldz);
          zz[k][0] = v.x; zz[k][W / 8] = v.y; zz[k][W / 4] = v.z; zz[k][W / 2 - W / 8] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (c + j < a.N) {
            g[k][j / 2] |= (uint32_t)dy[m * a.lddy + j] << (16 * (j % 2));
            if (act) zz[k][j / 2] |= (uint32_t)z[m * a.ldz + j] << (16 * (j % 2));
          }
      }
    }
#pragma unroll
    for (int k = 0; k < DZ_ROWS; ++k) {
      const int64_t m = m0 + (int64_t)k * parts;
      if (m >= a.M) continue;
      float v[W];
#pragma unroll
      for (int j = 0; j < W; j += 2) {   // (W = 1: the pair's second is not used)
        float2 d = bf16x2_to_f2(g[k][j / 2]);
        if (act) d = mul2(d, activation_slope<ACT>(bf16x2_to_f2(zz[k][j / 2])));
        v[j] = d.x;
        sum[j] = __fadd_rn(sum[j], d.x);
        if (j + 1 < W) {
          v[j + 1] = d.y;
          sum[j + 1] = __fadd_rn(sum[j + 1], d.y);
        }
      }
      if (!dz) continue;
      uint16_t* d = dz + m * ldd + c;
      if constexpr (W == 8) {
        store8(d, v, whole ? 8 : (int)(a.N - c));
      } else {
        *d = (uint16_t)pack_bf16(v[0], 0.f);
      }
    }
  }
  if (!db_part) return;
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (c + j < a.N) db_part[(int64_t)blockIdx.y * pitch + c + j] = sum[j];
}

// Adds the parts in order: 32 columns a CTA, warp w takes parts w, w + 8, ...,
// 20 of them on their way together.
__global__ void __launch_bounds__(256) linear_db_kernel(const float* part, int64_t pitch, int parts, int64_t N, float* db,
                                                        int accumulate) {
  pdl_wait();
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  for (int k0 = warp; k0 < parts; k0 += 160) {
    float x[20];
#pragma unroll
    for (int u = 0; u < 20; ++u) x[u] = c < N && k0 + 8 * u < parts ? part[(int64_t)(k0 + 8 * u) * pitch + c] : 0.f;
#pragma unroll
    for (int u = 0; u < 20; ++u) v = __fadd_rn(v, x[u]);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < N) {
    for (int k = 1; k < 8; ++k) v = __fadd_rn(v, s[k][lane]);
    db[c] = accumulate ? __fadd_rn(db[c], v) : v;
  }
}

__global__ void __launch_bounds__(ET) linear_zero_kernel(void* p, int dtype, int64_t ld, int64_t rows, int64_t cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += ET) {
      if (dtype) static_cast<float*>(p)[r * ld + c] = 0.f;
      else static_cast<uint16_t*>(p)[r * ld + c] = 0u;
    }
}

// ------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load();
  if (f) return f;
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiledFn>(ptr);
  fn.store(f);
  return f;
}

// A bf16 operand: K-contiguous ([mn][k], boxes of 64 K x box_mn rows) or
// MN-contiguous ([k][mn], boxes of 64 columns x 64 K rows).
struct Operand {
  const void* p;
  int64_t ld;
};
bool make_map(CUtensorMap* map, const Operand& o, bool mn_major, int64_t mn, int64_t k, uint32_t box_mn) {
  EncodeTiledFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(mn_major ? mn : k), (cuuint64_t)(mn_major ? k : mn)};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
  const cuuint32_t box[2] = {64u, mn_major ? 64u : box_mn};
  const cuuint32_t estr[2] = {1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(o.p), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rows16(const void* p, int dtype, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % (dtype ? 4 : 8) == 0;
}
bool tma_rows(const void* p, int64_t ld) { return rows16(p, 0, ld); }
// rows of bf16 that start on 4-byte boundaries
bool rows4(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0; }
int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

template <bool A_MN, bool B_MN, bool SPLIT>
cudaError_t set_smem() {
  static std::atomic<int> done[64];
  const int ds = device_slot();
  if (ds >= 0 && done[ds].load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(linear_gemm_kernel<A_MN, B_MN, SPLIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<SPLIT>::smem(Shape<SPLIT>::STAGES));
  if (e == cudaSuccess && ds >= 0) done[ds].store(1);
  return e;
}

// CTAs that share a tile's K when there are `tiles` tiles of 128 x 128: 2 or 4
// while all have an SM and at least four stages of K each, or half an SM and at
// least eight.  Measured (us): 64 tiles of K 1000, by 2 13.7, by 4 18.0; 128 tiles
// of K 4096, whole 35.3, by 2 26.3.
int split_for(int tiles, int k_steps) {
  int s = 1;
  while (s < MAX_SPLIT && k_steps >= 8 * s && tiles * 2 * s <= (k_steps >= 16 * s ? 2 : 1) * sm_count()) s *= 2;
  return s;
}

// One launch over the tiles, as a programmatic dependent of the kernel before it.
template <bool A_MN, bool B_MN, bool SPLIT>
cudaError_t launch_gemm(const CUtensorMap& ma, const CUtensorMap& mb, GemmParams p, int split,
                        cudaStream_t stream) {
  if (cudaError_t e = set_smem<A_MN, B_MN, SPLIT>(); e != cudaSuccess) return e;
  const int tiles = p.n_tiles;
  cudaLaunchConfig_t cfg{};
  const int pairs = sm_count() / 2;
  cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * split : 2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(Shape<SPLIT>::THREADS);
  p.stages = SPLIT && tiles * split > sm_count() ? FEW_STAGES : Shape<SPLIT>::STAGES;
  cfg.dynamicSmemBytes = Shape<SPLIT>::smem(p.stages);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)(SPLIT ? split : 2);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_gemm_kernel<A_MN, B_MN, SPLIT>, ma, mb, p, split);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool A_MN, bool B_MN>
cudaError_t gemm(const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, const Epilogue& epi,
                 cudaStream_t stream) {
  GemmParams p{};
  p.M = M;
  p.N = N;
  p.k_steps = (int)((K + BK - 1) / BK);
  p.wait_limit = debug_wait_limit();
  p.withhold = (int)debug_take_withheld();
  p.e = epi;
  p.e.vec = rows16(epi.y, epi.y_dtype, epi.ldy) && (!epi.z || rows16(epi.z, 0, epi.ldz)) &&
            (!epi.residual || rows16(epi.residual, 0, epi.ldr));
  p.e.even = N % 2 == 0 && (epi.y_dtype != 0 || rows4(epi.y, epi.ldy)) && (!epi.z || rows4(epi.z, epi.ldz)) &&
             (!epi.residual || rows4(epi.residual, epi.ldr));
  const int64_t small = ((M + 127) / 128) * ((N + 127) / 128);
  if (small > (1 << 30)) return cudaErrorInvalidValue;
  // Tiles of 128 x 128, K split over a cluster while SMs are left, when there is
  // an SM for each (or there are no rows for a pair); else pairs' tiles of 256 x 256.
  // Measured with 256 tiles of K 4096: 43 us as small ones, two an SM, 36 us as pairs'.
  const bool few = small <= sm_count() || M <= BM;
  CUtensorMap ma, mb;
  if (!make_map(&ma, a, A_MN, M, K, BM) || !make_map(&mb, b, B_MN, N, K, BROWS)) return cudaErrorInvalidValue;
  const int tm = few ? 128 : 256;
  p.n_mt = (int)((M + tm - 1) / tm);
  p.n_nt = (int)((N + tm - 1) / tm);
  p.n_tiles = p.n_mt * p.n_nt;
  return few ? launch_gemm<A_MN, B_MN, true>(ma, mb, p, split_for(p.n_tiles, p.k_steps), stream)
             : launch_gemm<A_MN, B_MN, false>(ma, mb, p, 1, stream);
}

size_t copy_bytes(int64_t rows, int64_t cols) { return pad256((size_t)rows * pad8(cols) * 2); }

template <int R>
cudaError_t gemv_rows(const LinearArgs& a, const Epilogue& e, cudaStream_t stream) {
  const bool vec = tma_rows(a.x, a.ldx) && tma_rows(a.w, a.ldw), even = rows4(a.x, a.ldx) && rows4(a.w, a.ldw);
  const int64_t warps = (int64_t)sm_count() * 32, least = vec ? 512 : (even ? 128 : 64);   // columns of K that are worth a warp
  int wpf = 1;
  while (wpf < GEMV_T / 32 && a.N * wpf * 2 <= warps && a.K >= least * wpf * 2) wpf *= 2;
  const dim3 grid((unsigned)((a.N * wpf + GEMV_T / 32 - 1) / (GEMV_T / 32)));
  const auto kernel = vec ? linear_gemv_kernel<R, 8> : (even ? linear_gemv_kernel<R, 2> : linear_gemv_kernel<R, 1>);
  const cudaError_t err = launch_after(kernel, grid, dim3(GEMV_T), 0, stream, static_cast<const uint16_t*>(a.x), a.ldx,
                                       static_cast<const uint16_t*>(a.w), a.ldw, a.N, (int)a.K, wpf, e);
  return err != cudaSuccess ? err : cudaGetLastError();
}

// Up to two operands whose rows TMA cannot read are replaced by copies at *ws
// (advanced), made in one launch.
struct Copied {
  Operand* o;
  int64_t rows, cols;
};
cudaError_t aligned_operands(Copied x, Copied w, char*& ws, cudaStream_t stream) {
  Repack r[2] = {};
  int n = 0;
  for (const Copied& c : {x, w}) {
    if (!c.o || tma_rows(c.o->p, c.o->ld)) continue;
    uint16_t* dst = reinterpret_cast<uint16_t*>(ws);
    ws += copy_bytes(c.rows, c.cols);
    r[n++] = Repack{static_cast<const uint16_t*>(c.o->p), c.o->ld, c.rows, c.cols, dst, pad8(c.cols)};
    *c.o = Operand{dst, pad8(c.cols)};
  }
  if (n == 0) return cudaSuccess;
  const int64_t want = (r[0].rows + r[1].rows + ET / 32 - 1) / (ET / 32), cap = (int64_t)sm_count() * 16;
  const cudaError_t e = launch_after(repack_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(ET), 0, stream, r[0], r[1]);
  return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kDbParts = 304;   // most row parts of the bias gradient
// A part has DZ_ROWS rows or more.
int64_t db_parts_most(int64_t M) {
  const int64_t p = (M + DZ_ROWS - 1) / DZ_ROWS;
  return p < kDbParts ? p : kDbParts;
}
size_t db_bytes(int64_t M, int64_t N) { return pad256((size_t)db_parts_most(M) * pad8(N) * sizeof(float)); }

}  // namespace

size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K) { return copy_bytes(M, K) + copy_bytes(N, K); }

size_t linear_workspace_needed(const LinearArgs& a) {
  if (a.M <= GEMV_ROWS) return 0;
  return (tma_rows(a.x, a.ldx) ? 0 : copy_bytes(a.M, a.K)) + (tma_rows(a.w, a.ldw) ? 0 : copy_bytes(a.N, a.K));
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  Operand x{a.x, a.ldx}, w{a.w, a.ldw};
  Epilogue e{};
  e.bias = a.bias;
  e.bias_dtype = a.bias_dtype;
  e.residual = static_cast<const uint16_t*>(a.residual);
  e.ldr = a.ldr;
  e.act = a.act;
  e.y = a.y;
  e.y_dtype = a.y_dtype;
  e.ldy = a.ldy;
  e.z = static_cast<uint16_t*>(a.z);
  e.ldz = a.ldz;
  switch (a.M) {
    case 1: return gemv_rows<1>(a, e, stream);
    case 2: return gemv_rows<2>(a, e, stream);
    case 3: return gemv_rows<3>(a, e, stream);
    case GEMV_ROWS: return gemv_rows<GEMV_ROWS>(a, e, stream);
    default: break;
  }
  if (cudaError_t err = aligned_operands({&x, a.M, a.K}, {&w, a.N, a.K}, ws, stream); err != cudaSuccess) return err;
  return gemm<false, false>(x, w, a.M, a.N, a.K, e, stream);
}

size_t linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return copy_bytes(M, N) + copy_bytes(M, K) + copy_bytes(N, K) + db_bytes(M, N);
}

size_t linear_bwd_workspace_needed(const LinearBwdArgs& a) {
  const bool products = a.dx || a.dw;
  size_t n = a.db ? db_bytes(a.M, a.N) : 0;
  if (products && (a.act != RLK_ACT_NONE || !tma_rows(a.dy, a.lddy))) n += copy_bytes(a.M, a.N);
  if (a.dx && !tma_rows(a.w, a.ldw)) n += copy_bytes(a.N, a.K);
  if (a.dw && (a.ck.codes || !tma_rows(a.x, a.ldx))) n += copy_bytes(a.M, a.K);
  return n;
}

cudaError_t launch_linear_bwd(const LinearBwdArgs& a, cudaStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  if (a.M == 0) {   // sums over no rows
    const int64_t cap = (int64_t)sm_count() * 8;
    if (a.dw && !a.accumulate)
      linear_zero_kernel<<<(unsigned)(a.N < cap ? a.N : cap), ET, 0, stream>>>(a.dw, a.dw_dtype, a.lddw, a.N, a.K);
    if (a.db && !a.accumulate) linear_zero_kernel<<<1, ET, 0, stream>>>(a.db, 1, a.N, 1, a.N);
    return cudaGetLastError();
  }
  // dz, and the bias gradient with it
  Operand dz{a.dy, a.lddy};
  const bool products = a.dx || a.dw;
  const bool make_dz = products && (a.act != RLK_ACT_NONE || !tma_rows(a.dy, a.lddy));
  if (make_dz || a.db) {
    uint16_t* dst = nullptr;
    const int64_t ld = pad8(a.N);
    if (make_dz) {
      dst = reinterpret_cast<uint16_t*>(ws);
      ws += copy_bytes(a.M, a.N);
      dz = Operand{dst, ld};
    }
    float* part = nullptr;
    if (a.db) {
      part = reinterpret_cast<float*>(ws);
      ws += db_bytes(a.M, a.N);
    }
    const int64_t pitch = pad8(a.N);
    const bool vec = tma_rows(a.dy, a.lddy) && (a.act == RLK_ACT_NONE || tma_rows(a.z, a.ldz));
    const unsigned cols = (unsigned)((a.N + DT * (vec ? 8 : 1) - 1) / (DT * (vec ? 8 : 1)));
    // about 8 CTAs an SM
    int64_t parts = ((int64_t)sm_count() * 8 + cols - 1) / cols, most = db_parts_most(a.M);
    if (parts > most) parts = most;
    const dim3 grid(cols, (unsigned)parts);
    auto kernel = vec ? (a.act == RLK_ACT_GELU   ? linear_dz_kernel<8, RLK_ACT_GELU>
                         : a.act == RLK_ACT_SILU ? linear_dz_kernel<8, RLK_ACT_SILU>
                         : a.act == RLK_ACT_RELU ? linear_dz_kernel<8, RLK_ACT_RELU>
                                                 : linear_dz_kernel<8, RLK_ACT_NONE>)
                      : (a.act == RLK_ACT_GELU   ? linear_dz_kernel<1, RLK_ACT_GELU>
                         : a.act == RLK_ACT_SILU ? linear_dz_kernel<1, RLK_ACT_SILU>
                         : a.act == RLK_ACT_RELU ? linear_dz_kernel<1, RLK_ACT_RELU>
                                                 : linear_dz_kernel<1, RLK_ACT_NONE>);
    kernel<<<grid, DT, 0, stream>>>(a, dst, ld, part, pitch, (int)parts);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (a.db) {
      const cudaError_t e = launch_after(linear_db_kernel, dim3((unsigned)((a.N + 31) / 32)), dim3(256), 0, stream,
                                         (const float*)part, pitch, (int)parts, a.N, a.db, a.accumulate);
      if (e != cudaSuccess) return e;
    }
  }
  Operand w{a.w, a.ldw}, x{a.x, a.ldx};
  if (cudaError_t e = aligned_operands({a.dx ? &w : nullptr, a.N, a.K}, {a.dw && a.x ? &x : nullptr, a.M, a.K}, ws, stream);
      e != cudaSuccess)
    return e;
  if (a.dx) {   // dx = dz w: K is N, w [N][K] holds its columns contiguously
    Epilogue e{};
    e.y = a.dx;
    e.y_dtype = a.dx_dtype;
    e.ldy = a.lddx;
    if (cudaError_t er = gemm<false, true>(dz, w, a.M, a.K, a.N, e, stream); er != cudaSuccess) return er;
  }
  if (a.dw) {   // dw = dz^T x: K is M, both operands hold M / N contiguously
    if (!a.x) {   // the checkpoint's values are exact in bf16
      const int64_t ld = pad8(a.K);
      CheckpointArgs c{};
      c.x = ws;
      c.T = a.M;
      c.H = a.K;
      c.ldx = ld;
      c.ck = a.ck;
      if (cudaError_t e = launch_checkpoint_unpack(c, stream); e != cudaSuccess) return e;
      x = Operand{ws, ld};
      ws += copy_bytes(a.M, a.K);
    }
    Epilogue e{};
    e.y = a.dw;
    e.y_dtype = a.dw_dtype;
    e.ldy = a.lddw;
    e.accumulate = a.accumulate;
    return gemm<true, true>(dz, x, a.N, a.K, a.M, e, stream);
  }
  return cudaSuccess;
}

}  // namespace rlk
