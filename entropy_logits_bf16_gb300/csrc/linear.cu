// rlk_linear_fwd / rlk_linear_bwd: matrix products with a fused epilogue.
//
//   forward   z = x w^T + bias,  y = act(z) + residual
//   backward  dz = dy act'(z),  dx = dz w,  dw = dz^T x,  db = sum_m dz
//
// All three products are one kernel, D[M, N] = sum_k A[m, k] B[n, k], whose
// operands may each be stored with K or with M / N contiguous, so neither w nor
// x nor dz is transposed in memory.  bf16 operands arrive by TMA (128-byte
// swizzle) in a ring of 64-deep stages, one thread issues the tcgen05 MMAs
// (128 x 256 x 16, fp32 accumulators in TMEM), four warps run the epilogue on
// registers read with tcgen05.ld, one row a thread.
//  * Many tiles: persistent CTAs, one an SM; two TMEM accumulators, so a tile's
//    epilogue runs under the next tile's products.  Tiles are walked in groups
//    of 16 row tiles, so the CTAs at work share 16 A tiles and about 10 B tiles
//    in L2.
//  * Few tiles (a call of few rows is bound by the weight's bytes, and needs
//    every SM to fetch them): a cluster of 2, 4 or 8 CTAs splits K, leaves its
//    partial tiles in shared memory, and each CTA adds the cluster's partials
//    in rank order for its share of the columns.
// TMA needs rows that start on 16-byte boundaries; an operand whose rows do not
// is first copied into the workspace.
//
// The epilogue's arithmetic is fp32 and y, z, dx, dw are rounded once.  dz is
// rounded to bf16 before its two products (the tensor cores' operand type; a
// relative 2^-9 of each term, below the rounding of a bf16 dw); db sums it
// unrounded.
// Every wait is bounded; when one runs out the CTA's unfinished tiles are NaN.

#include <math.h>

#include <atomic>

#include "checkpoint.cuh"
#include "internal.h"
#include "rlk.h"
#include "tensor_core.cuh"

namespace rlk {
namespace {

constexpr int BM = 128, BN = 256, BK = 64, STAGES = 4, THREADS = 192;
constexpr uint32_t A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t MN_BLOCK = 64 * BK * 2;   // a 64-element block of an MN-contiguous operand
constexpr uint32_t TMEM_COLS = 512;
constexpr size_t SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;
constexpr int GROUP_M = 16;
constexpr int PLD = BN + 4;   // row pitch (floats) of a partial tile: conflict-free float4 rows
static_assert(BM * PLD * 4 <= STAGES * STAGE_BYTES, "a partial tile fits into the ring");

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
};
struct GemmParams {
  int64_t M, N;
  int n_mt, n_nt, n_tiles, k_steps;
  long long wait_limit;
  Epilogue e;
};

__device__ __forceinline__ float activate(float z, int act) {
  if (act == RLK_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  if (act == RLK_ACT_SILU) return __fdiv_rn(z, 1.f + expf(-z));
  if (act == RLK_ACT_RELU) return z < 0.f ? 0.f : z;
  return z;
}
__device__ __forceinline__ float activation_slope(float z, int act) {
  if (act == RLK_ACT_GELU)
    return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
           z * expf(-0.5f * z * z) * 0.39894228040143268f;
  if (act == RLK_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  return z > 0.f ? 1.f : (z != z ? z : 0.f);   // ReLU
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The epilogue of W columns of one row (columns [col, col + n) valid).
template <int W>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t row, int64_t col, int n, float (&v)[W]) {
  if (e.bias) {
    if (e.bias_dtype == 0) {
      const uint16_t* b = static_cast<const uint16_t*>(e.bias) + col;
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < n) v[j] = __fadd_rn(v[j], bf16_val(b[j]));
    } else {
      const float* b = static_cast<const float*>(e.bias) + col;
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < n) v[j] = __fadd_rn(v[j], b[j]);
    }
  }
  if (e.z) {
    uint16_t* z = e.z + row * e.ldz + col;
    if (W % 8 == 0 && n == W && aligned16(z)) {
#pragma unroll
      for (int j = 0; j < W / 8; ++j)
        reinterpret_cast<uint4*>(z)[j] =
            make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                       pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < n) z[j] = (uint16_t)pack_bf16(v[j], 0.f);
    }
  }
  if (e.act != RLK_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = activate(v[j], e.act);
  }
  if (e.residual) {
    const uint16_t* r = e.residual + row * e.ldr + col;
    if (W % 8 == 0 && n == W && aligned16(r)) {
#pragma unroll
      for (int j = 0; j < W / 8; ++j) {
        const uint4 q = reinterpret_cast<const uint4*>(r)[j];
        const uint32_t w4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[8 * j + 2 * k] = __fadd_rn(v[8 * j + 2 * k], bf16_lo(w4[k]));
          v[8 * j + 2 * k + 1] = __fadd_rn(v[8 * j + 2 * k + 1], bf16_hi(w4[k]));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < n) v[j] = __fadd_rn(v[j], bf16_val(r[j]));
    }
  }
  if (e.y_dtype == 0) {
    uint16_t* y = static_cast<uint16_t*>(e.y) + row * e.ldy + col;
    if (W % 8 == 0 && n == W && aligned16(y)) {
#pragma unroll
      for (int j = 0; j < W / 8; ++j)
        reinterpret_cast<uint4*>(y)[j] =
            make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                       pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < n) y[j] = (uint16_t)pack_bf16(v[j], 0.f);
    }
  } else {
    float* y = static_cast<float*>(e.y) + row * e.ldy + col;
    if (W % 4 == 0 && n == W && aligned16(y)) {
#pragma unroll
      for (int j = 0; j < W / 4; ++j) {
        float4 o = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        if (e.accumulate) {
          const float4 old = reinterpret_cast<const float4*>(y)[j];
          o = make_float4(__fadd_rn(old.x, o.x), __fadd_rn(old.y, o.y), __fadd_rn(old.z, o.z),
                          __fadd_rn(old.w, o.w));
        }
        reinterpret_cast<float4*>(y)[j] = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < n) y[j] = e.accumulate ? __fadd_rn(y[j], v[j]) : v[j];
    }
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

// SPLIT: a cluster of CTAs works on one tile, each on its share of K; else a
// CTA works on whole tiles blockIdx.x, + gridDim.x, ...
template <bool A_MN, bool B_MN, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const GemmParams p, int cluster) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base_ptr + STAGES * STAGE_BYTES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
  const uint32_t accf0 = empty0 + 8 * STAGES, acce0 = accf0 + 16;
  const uint32_t drain_bar = smem_u32(bars + 2 * STAGES + 6);
  constexpr uint32_t idesc = tc::idesc_bf16(A_MN, B_MN, BM, BN);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf0 + 8 * a, 1);
      mbar_init(acce0 + 8 * a, 4);   // one arrive per epilogue warp
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) tc::alloc(smem_u32(tmem_slot), TMEM_COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  const uint32_t rank = SPLIT ? tc::cluster_rank() : 0u;
  const int tile0 = SPLIT ? (int)(blockIdx.x / (unsigned)cluster) : (int)blockIdx.x;
  const int tile_step = SPLIT ? p.n_tiles : (int)gridDim.x;
  const int k0 = SPLIT ? (int)((int64_t)rank * p.k_steps / cluster) : 0;
  const int k1 = SPLIT ? (int)((int64_t)(rank + 1) * p.k_steps / cluster) : p.k_steps;

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
          mbar_expect_tx(fb, STAGE_BYTES);
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES;
          if (A_MN) {
#pragma unroll
            for (int j = 0; j < BM / 64; ++j) tc::load_2d(sa + j * MN_BLOCK, &map_a, fb, mt * BM + j * 64, k * BK);
          } else {
            tc::load_2d(sa, &map_a, fb, k * BK, mt * BM);
          }
          if (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 64; ++j) tc::load_2d(sb + j * MN_BLOCK, &map_b, fb, nt * BN + j * 64, k * BK);
          } else {
            tc::load_2d(sb, &map_b, fb, k * BK, nt * BN);
          }
          used |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok || *abort_flag) {   // let every issued copy land before the CTA exits
        for (int s = 0; s < STAGES; ++s)
          if (used & (1u << s)) tc::drain(full0 + 8 * s, (last_parity >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, tile = 0;
      bool ok = true;
      for (int t = tile0; t < p.n_tiles && ok; t += tile_step, ++tile) {
        const uint32_t acc = tile & 1u, accph = (tile >> 1) & 1u;
        if (!tc::wait(acce0 + 8 * acc, accph ^ 1u, abort_flag, p.wait_limit)) { ok = false; break; }
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
            tc::mma(d_tmem, da, db, idesc, (k > k0 || kk > 0) ? 1u : 0u);
          }
          tc::commit(empty0 + 8 * stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok) tc::commit(accf0 + 8 * acc);
      }
      if (!ok) {   // every MMA already issued finishes before TMEM is freed
        tc::commit(drain_bar);
        tc::drain(drain_bar, 0u);
      }
    }
  } else {
    // ------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    uint32_t tile = 0;
    bool ok = true;
    for (int t = tile0; t < p.n_tiles; t += tile_step, ++tile) {
      int mt, nt;
      tile_coords(p, t, mt, nt);
      const uint32_t acc = tile & 1u, accph = (tile >> 1) & 1u;
      // after a wait has run out, this tile and the CTA's later ones are NaN
      ok = ok && tc::wait(accf0 + 8 * acc, accph, abort_flag, p.wait_limit);
      tc::fence_after();
      const int r = q * 32 + lane;
      const int64_t row = (int64_t)mt * BM + r;
#pragma unroll 1
      for (int ch = 0; ch < BN / 32; ++ch) {
        float v[32];
        if (ok) {
          tc::ld32(tmem + lane_base + acc * BN + ch * 32, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = NAN;
        }
        const int64_t col = (int64_t)nt * BN + ch * 32;
        if (row >= p.M || col >= p.N) continue;
        if (SPLIT) {
          float* part = reinterpret_cast<float*>(base_ptr) + r * PLD + ch * 32;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            reinterpret_cast<float4*>(part)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          finish<32>(p.e, row, col, (int)(p.N - col < 32 ? p.N - col : 32), v);
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(acce0 + 8 * acc);
    }
  }
  if (SPLIT) {
    __syncwarp();
    tc::cluster_sync();   // every partial tile is in its CTA's shared memory
    bool dead = false;    // a wait of some CTA of the cluster ran out
    const uint32_t abort_at = smem_u32(bars + 2 * STAGES + 4);
    for (int k = 0; k < cluster; ++k) dead = tc::ld_peer_u32(tc::peer_addr(abort_at, (uint32_t)k)) != 0u || dead;
    // this CTA's share of the columns, all rows: groups of 4 columns
    int mt, nt;
    tile_coords(p, tile0, mt, nt);
    const int width = BN / cluster, quads = width / 4;
    const int64_t row0 = (int64_t)mt * BM;
    const int rows = (int)(p.M - row0 < BM ? p.M - row0 : BM);
    for (int i = threadIdx.x; i < rows * quads; i += THREADS) {
      const int r = i / quads, c = (int)rank * width + (i - r * quads) * 4;
      const int64_t col = (int64_t)nt * BN + c;
      if (col >= p.N) continue;
      const uint32_t at = base + (uint32_t)(r * PLD + c) * 4u;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < cluster; ++k) {
        const float4 o = tc::ld_peer4(tc::peer_addr(at, (uint32_t)k));
        v[0] = __fadd_rn(v[0], o.x);
        v[1] = __fadd_rn(v[1], o.y);
        v[2] = __fadd_rn(v[2], o.z);
        v[3] = __fadd_rn(v[3], o.w);
      }
      if (dead) v[0] = v[1] = v[2] = v[3] = NAN;
      finish<4>(p.e, row0 + r, col, (int)(p.N - col < 4 ? p.N - col : 4), v);
    }
    tc::cluster_sync();   // no CTA leaves while its shared memory is read
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::dealloc(tmem, TMEM_COLS);
}

// ------------------------------------------------------------ around the products
constexpr int ET = 256;

// A bf16 matrix copied to rows that start on 16-byte boundaries.
__global__ void __launch_bounds__(ET) repack_kernel(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols,
                                                    uint16_t* dst, int64_t ldd) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += ET) dst[r * ldd + c] = src[r * ld + c];
}

// dz = dy act'(z) as bf16 and the partial column sums of the unrounded dz: part
// blockIdx.y takes rows blockIdx.y, + parts, ...
__global__ void __launch_bounds__(ET) linear_dz_kernel(LinearBwdArgs a, uint16_t* dz, int64_t ldd, float* db_part,
                                                       int parts) {
  const int64_t c = (int64_t)blockIdx.x * ET + threadIdx.x;
  if (c >= a.N) return;
  const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
  const uint16_t* z = static_cast<const uint16_t*>(a.z);
  float sum = 0.f;
  for (int64_t m = blockIdx.y; m < a.M; m += parts) {
    float g = bf16_val(dy[m * a.lddy + c]);
    if (a.act != RLK_ACT_NONE) g = __fmul_rn(g, activation_slope(bf16_val(z[m * a.ldz + c]), a.act));
    sum = __fadd_rn(sum, g);
    if (dz) dz[m * ldd + c] = (uint16_t)pack_bf16(g, 0.f);
  }
  if (db_part) db_part[(int64_t)blockIdx.y * a.N + c] = sum;
}

__global__ void __launch_bounds__(ET) linear_db_kernel(const float* part, int parts, int64_t N, float* db,
                                                       int accumulate) {
  const int64_t c = (int64_t)blockIdx.x * ET + threadIdx.x;
  if (c >= N) return;
  float v = 0.f;
  for (int p = 0; p < parts; ++p) v = __fadd_rn(v, part[(int64_t)p * N + c]);
  db[c] = accumulate ? __fadd_rn(db[c], v) : v;
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

bool tma_rows(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }
int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

// CTAs that share a tile's K: as many (2, 4, 8) as keep the grid within the
// SMs and leave each at least four stages.
int split_for(int tiles, int k_steps) {
  int s = 1;
  while (s < 8 && tiles * 2 * s <= sm_count() && k_steps >= 8 * s) s *= 2;
  return s;
}

template <bool A_MN, bool B_MN, bool SPLIT>
cudaError_t set_smem() {
  static std::atomic<int> done[64];
  const int ds = device_slot();
  if (ds >= 0 && done[ds].load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(linear_gemm_kernel<A_MN, B_MN, SPLIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e == cudaSuccess && ds >= 0) done[ds].store(1);
  return e;
}

template <bool A_MN, bool B_MN>
cudaError_t gemm(const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, const Epilogue& epi,
                 cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!make_map(&ma, a, A_MN, M, K, BM) || !make_map(&mb, b, B_MN, N, K, BN)) return cudaErrorInvalidValue;
  GemmParams p{};
  p.M = M;
  p.N = N;
  p.n_mt = (int)((M + BM - 1) / BM);
  p.n_nt = (int)((N + BN - 1) / BN);
  const int64_t tiles = (int64_t)p.n_mt * p.n_nt;
  if (tiles > (1 << 30)) return cudaErrorInvalidValue;
  p.n_tiles = (int)tiles;
  p.k_steps = (int)((K + BK - 1) / BK);
  p.wait_limit = debug_wait_limit();
  p.e = epi;
  const int split = split_for(p.n_tiles, p.k_steps);
  if (split == 1) {
    if (cudaError_t e = set_smem<A_MN, B_MN, false>(); e != cudaSuccess) return e;
    const int grid = p.n_tiles < sm_count() ? p.n_tiles : sm_count();
    linear_gemm_kernel<A_MN, B_MN, false><<<grid, THREADS, SMEM_BYTES, stream>>>(ma, mb, p, 1);
    return cudaGetLastError();
  }
  if (cudaError_t e = set_smem<A_MN, B_MN, true>(); e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.n_tiles * split));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_gemm_kernel<A_MN, B_MN, true>, ma, mb, p, split);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The operand itself when TMA can read it, else its copy at *ws (advanced).
cudaError_t aligned_operand(Operand& o, int64_t rows, int64_t cols, char*& ws, cudaStream_t stream) {
  if (tma_rows(o.p, o.ld)) return cudaSuccess;
  uint16_t* dst = reinterpret_cast<uint16_t*>(ws);
  const int64_t ld = pad8(cols);
  ws += pad256((size_t)rows * ld * 2);
  const int64_t cap = (int64_t)sm_count() * 8;
  repack_kernel<<<(unsigned)(rows < cap ? rows : cap), ET, 0, stream>>>(static_cast<const uint16_t*>(o.p), o.ld, rows,
                                                                       cols, dst, ld);
  o = Operand{dst, ld};
  return cudaGetLastError();
}

size_t copy_bytes(int64_t rows, int64_t cols) { return pad256((size_t)rows * pad8(cols) * 2); }

constexpr int kDbParts = 64;
size_t db_bytes(int64_t N) { return pad256((size_t)kDbParts * N * sizeof(float)); }

}  // namespace

size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K) { return copy_bytes(M, K) + copy_bytes(N, K); }

size_t linear_workspace_needed(const LinearArgs& a) {
  return (tma_rows(a.x, a.ldx) ? 0 : copy_bytes(a.M, a.K)) + (tma_rows(a.w, a.ldw) ? 0 : copy_bytes(a.N, a.K));
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  Operand x{a.x, a.ldx}, w{a.w, a.ldw};
  if (cudaError_t e = aligned_operand(x, a.M, a.K, ws, stream); e != cudaSuccess) return e;
  if (cudaError_t e = aligned_operand(w, a.N, a.K, ws, stream); e != cudaSuccess) return e;
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
  return gemm<false, false>(x, w, a.M, a.N, a.K, e, stream);
}

size_t linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return copy_bytes(M, N) + copy_bytes(M, K) + copy_bytes(N, K) + db_bytes(N);
}

size_t linear_bwd_workspace_needed(const LinearBwdArgs& a) {
  const bool products = a.dx || a.dw;
  size_t n = a.db ? db_bytes(a.N) : 0;
  if (products && (a.act != RLK_ACT_NONE || !tma_rows(a.dy, a.lddy))) n += copy_bytes(a.M, a.N);
  if (a.dx && !tma_rows(a.w, a.ldw)) n += copy_bytes(a.N, a.K);
  if (a.dw && (a.ck.codes || !tma_rows(a.x, a.ldx))) n += copy_bytes(a.M, a.K);
  return n;
}

cudaError_t launch_linear_bwd(const LinearBwdArgs& a, cudaStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  const unsigned ncols = (unsigned)((a.N + ET - 1) / ET);
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
      ws += db_bytes(a.N);
    }
    const int parts = (int)(a.M < kDbParts ? a.M : kDbParts);
    linear_dz_kernel<<<dim3(ncols, parts), ET, 0, stream>>>(a, dst, ld, part, parts);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (a.db) {
      linear_db_kernel<<<ncols, ET, 0, stream>>>(part, parts, a.N, a.db, a.accumulate);
      if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
  }
  if (a.dx) {   // dx = dz w: K is N, w [N][K] holds its columns contiguously
    Operand w{a.w, a.ldw};
    if (cudaError_t e = aligned_operand(w, a.N, a.K, ws, stream); e != cudaSuccess) return e;
    Epilogue e{};
    e.y = a.dx;
    e.y_dtype = a.dx_dtype;
    e.ldy = a.lddx;
    if (cudaError_t er = gemm<false, true>(dz, w, a.M, a.K, a.N, e, stream); er != cudaSuccess) return er;
  }
  if (a.dw) {   // dw = dz^T x: K is M, both operands hold M / N contiguously
    Operand x{a.x, a.ldx};
    if (a.ck.codes) {   // the checkpoint's values are exact in bf16
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
    } else {
      if (cudaError_t e = aligned_operand(x, a.M, a.K, ws, stream); e != cudaSuccess) return e;
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
