// The tcgen05 matrix product that the gated layer and the orthogonalisation share:
// D[m, n] = sum_k A[m, k] B[n, k] over many tiles, 16-bit operands, fp32 accumulators, with
// what is done to D left to an `Op`.
//
// Operands may be K- or MN-contiguous and arrive by TMA (128-byte swizzle) in a ring of 64-deep
// stages; one thread issues the MMAs; the other warps run the epilogue.
//  * Many tiles: persistent pairs of CTAs (cta_group::2), 256 x 256 a pair, two TMEM
//    accumulators, so that a tile's epilogue runs under the next tile's products.
//  * Few tiles: 128 x 128 a CTA, K split over a cluster of up to 4 CTAs whose partial tiles are
//    added in rank order through distributed shared memory.
// Every wait is bounded; when one runs out the CTA's unfinished tiles are NaN and the status
// word, where the call has one, gets RLK_STATUS_TIMEOUT.
//
// An Op has
//   A_MN, B_MN   whether an operand holds its rows' index contiguously
//   F16          operands fp16, else bf16
//   DUAL         B's tile is one half of rows of b[0] and one of b[1]: two products that
//                share A, joined column by column in the epilogue
//   TRI_A, TRI_B  the operand is a symmetric matrix (K-contiguous) of which the blocks of loop.tri x
//                loop.tri above the diagonal are not in memory (0: all are): such a step takes the block's
//                mirror image, MN-contiguous
//   STACKED      maps are of stacks of matrices, of which a tile takes number `which`
//   Params       with `Loop loop`
//   tile(p, t, tm, bn)   the place of tile t
//   source(tl, part, ia, ib)   which maps the steps of a part of K take (loop.part_steps each)
//   Aux, aux8    what finish8 needs from memory for its row (asked for before the accumulator is
//                waited for); Cols, cols8: what it needs for its columns
//   finish8, column8   D's 8 columns of a row / one column of 8 rows `step` apart (of which those
//                up to n rows on exist), to memory
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "rlk.h"
#include "tensor_core.cuh"

namespace rlk {
namespace gemm {

constexpr int BM = 128, BK = 64, BROWS = 128;
constexpr uint32_t MN_BLOCK = 64 * BK * 2;     // a 64-element block of an MN-contiguous operand
constexpr uint32_t STAGING = 32 * 32 * 4;      // an epilogue warp's 32 x 32 piece of a tile
constexpr uint32_t A_BYTES = BM * BK * 2, STAGE_BYTES = A_BYTES + BROWS * BK * 2;
constexpr int MAX_SPLIT = 4, MAX_STAGES = 6, FEW_STAGES = 3;

template <bool SPLIT>
struct Shape {
  static constexpr int G = SPLIT ? 1 : 2;      // CTAs of a tile
  static constexpr int EPI_WARPS = SPLIT ? 8 : 16, THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int STAGES = SPLIT ? 6 : 5; // at most
  static constexpr int TM = BM * G, BN = BROWS * G;
  static constexpr uint32_t TMEM_COLS = SPLIT ? BN : 2 * BN;
  static constexpr int PLD = BN + 4;           // row pitch (floats) of a partial tile
  static constexpr uint32_t STAGED = SPLIT ? 0 : EPI_WARPS * STAGING;
  static constexpr size_t smem(int stages) { return stages * STAGE_BYTES + STAGED + 1024 + 256; }
};
static_assert(BM * Shape<true>::PLD * 4 <= FEW_STAGES * STAGE_BYTES, "a partial tile fits into the ring");

struct Maps {
  CUtensorMap a[2], b[2];
};
struct TriMaps : Maps {
  CUtensorMap ta[2], tb[2];   // the mirror images of TRI operands
};
template <class Op>
using MapsOf = std::conditional_t<Op::TRI_A || Op::TRI_B, TriMaps, Maps>;
struct Tile {
  int a_row, b_row;      // first index of the operands' rows (M, N); MN-contiguous: column
  int64_t row, col;      // first row and column of D
  int64_t rows, cols;    // D's extents
  int which;             // of several products or matrices
};
struct Loop {
  int n_tiles, k_steps, stages;
  int part_steps;        // K's steps fall into parts of so many, each from maps of its own (0: one part)
  int tri;               // side of a TRI operand's blocks (a multiple of a tile's rows), or 0
  int a_rows;            // rows of A's boxes (K-contiguous, tiles of 128 x 128; else 128)
  long long wait_limit;
  uint32_t* status;      // RLK_STATUS_TIMEOUT goes here when a wait runs out (NULL: the call has no such word)
  int withhold;          // debug: the stage of the first CTA whose barrier waits for an arrival that never comes (-1: none)
};

// Adds a bit to the caller's status word; many threads may, so each looks first.
__device__ __forceinline__ void report(uint32_t* status, uint32_t bit) {
  if (status && !(*static_cast<volatile uint32_t*>(status) & bit)) atomicOr(status, bit);
}
// Tile t of n_mt x n_nt: groups of 8 row tiles, row tiles fastest inside a group, so that the
// CTAs at work share tiles of both operands in L2.
__device__ __forceinline__ void grouped(int t, int n_mt, int n_nt, int& mt, int& nt) {
  constexpr int GROUP = 8;
  const int group = t / (GROUP * n_nt), r = t - group * GROUP * n_nt;
  const int g0 = group * GROUP, gm = n_mt - g0 < GROUP ? n_mt - g0 : GROUP;
  mt = g0 + r % gm;
  nt = r / gm;
}

// Calls steps(A's layout, B's layout, from, to) for the runs of [k0, k1) in which neither
// changes (true: MN-contiguous); `first`: the step of K's start.
template <class Op, class F>
__device__ __forceinline__ void by_layout(const Loop& l, int a_row, int b_row, int first, int k0, int k1, F& steps) {
  using A = std::bool_constant<Op::A_MN>;
  using B = std::bool_constant<Op::B_MN>;
  using Mirror = std::true_type;
  if constexpr (Op::TRI_A || Op::TRI_B) {
    auto from = [&](int row) {
      const int k = l.tri ? first + (row / l.tri + 1) * (l.tri / BK) : k1;   // the first step whose columns lie above the diagonal's blocks
      return k < k0 ? k0 : (k < k1 ? k : k1);
    };
    const int a = Op::TRI_A ? from(a_row) : k1, b = Op::TRI_B ? from(b_row) : k1, one = a < b ? a : b, two = a < b ? b : a;
    steps(A{}, B{}, k0, one);
    if (Op::TRI_A && a < b) steps(Mirror{}, B{}, one, two);
    if (Op::TRI_B && b < a) steps(A{}, Mirror{}, one, two);
    if (Op::TRI_A && Op::TRI_B) steps(Mirror{}, Mirror{}, two, k1);
  } else {
    steps(A{}, B{}, k0, k1);
  }
}

template <class Op, bool SPLIT>
__global__ void __launch_bounds__(Shape<SPLIT>::THREADS, SPLIT ? 2 : 1)
    gemm_tiles_kernel(const __grid_constant__ MapsOf<Op> maps, const __grid_constant__ typename Op::Params p, int cluster) {
  using S = Shape<SPLIT>;
  constexpr int G = S::G, TM = S::TM, BN = S::BN, PLD = S::PLD, EPI_WARPS = S::EPI_WARPS;
  constexpr int OUT = Op::DUAL ? BN / 2 : BN;   // D's columns of a tile
  const int stages = SPLIT ? p.loop.stages : S::STAGES;
  const long long limit = p.loop.wait_limit;
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, 1 + (s == p.loop.withhold && blockIdx.x == 0));
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
    tc::prefetch_map(&maps.a[0]);
    tc::prefetch_map(&maps.b[0]);
    if (Op::DUAL) tc::prefetch_map(&maps.b[1]);
  }
  if (warp == 1) tc::alloc<G>(smem_u32(tmem_slot), TMEM_COLS);
  tc::fence_before();
  __syncthreads();
  // The next kernel gets ready where there is room, and waits for this one's end: only now that
  // this CTA has its TMEM, which the other's would else hold while they wait for this grid.
  pdl_trigger();
  pdl_wait();      // the operands may come from the kernel before
  if (G == 2) tc::cluster_sync();   // the other CTA's barriers are there
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  // SPLIT: which share of K; else: which half of the tile
  const uint32_t rank = tc::cluster_rank();
  const int per = SPLIT ? cluster : G;   // CTAs that work on one tile
  const int tile0 = (int)(blockIdx.x / (unsigned)per);
  const int tile_step = SPLIT ? p.loop.n_tiles : (int)(gridDim.x / G);
  const int k0 = SPLIT ? (int)((int64_t)rank * p.loop.k_steps / cluster) : 0;
  const int k1 = SPLIT ? (int)((int64_t)(rank + 1) * p.loop.k_steps / cluster) : p.loop.k_steps;
  const int a_off = SPLIT ? 0 : (int)rank * BM;
  const bool leader = SPLIT || rank == 0;
  // a tile of fewer rows is fetched without the rest (whose accumulators nobody looks at)
  const uint32_t bytes = G * STAGE_BYTES - (SPLIT && !Op::A_MN ? (uint32_t)(BM - p.loop.a_rows) * BK * 2 : 0u);

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    // One thread, whose instructions bound the products unless its loop is short (800 cycles a
    // step of the pairs' tiles with the layouts chosen in it, 512 are the tensor cores').
    if (lane == 0) {
      int stage = 0, issued = 0;   // issued: turns of the ring begun
      uint32_t phase = 0;
      bool ok = true;
      // a pair's copies all report to the even CTA, whose barrier expects them all
      const uint32_t report = G == 2 ? tc::peer_addr(full0, 0u) : full0;
      for (int t = tile0; t < p.loop.n_tiles && ok; t += tile_step) {
        const Tile tl = Op::tile(p, t, TM, OUT);
        const int am = tl.a_row + a_off, bn = tl.b_row + (SPLIT ? 0 : (int)rank * BROWS);
        for (int k = k0, part = k0 / p.loop.part_steps; k < k1 && ok; ++part) {
          const int first = part * p.loop.part_steps, last = first + p.loop.part_steps < k1 ? first + p.loop.part_steps : k1;
          int ia = 0, ib = 0;
          Op::source(tl, part, ia, ib);
          const CUtensorMap *ma = &maps.a[ia], *mb = &maps.b[ib], *mta = ma, *mtb = mb;
          if constexpr (Op::TRI_A) mta = &maps.ta[ia];
          if constexpr (Op::TRI_B) mtb = &maps.tb[ib];
          // steps [from, to) with these layouts
          auto steps = [&](auto a_layout, auto b_layout, int from, int to) {
            constexpr bool a_mn = decltype(a_layout)::value, b_mn = decltype(b_layout)::value;
            const CUtensorMap *xa = a_mn ? mta : ma, *xb = b_mn ? mtb : mb;
            int x = (from - first) * BK;   // the K coordinate
#pragma unroll 1
            for (int i = from; i < to; ++i, x += BK) {
              if (!tc::wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, limit) || ((i & 3) == 0 && *abort_flag)) {
                ok = false;
                return;
              }
              const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES, to_bar = report + 8 * stage;
              if (leader) mbar_expect_tx(full0 + 8 * stage, bytes);
              auto load = [&](uint32_t dst, const CUtensorMap* map, int cx, int cy) {
                if constexpr (Op::STACKED) {
                  if (G == 2) tc::load_3d_pair(dst, map, to_bar, cx, cy, tl.which);
                  else tc::load_3d(dst, map, to_bar, cx, cy, tl.which);
                } else {
                  if (G == 2) tc::load_2d_pair(dst, map, to_bar, cx, cy);
                  else tc::load_2d(dst, map, to_bar, cx, cy);
                }
              };
              if (a_mn) {
#pragma unroll
                for (int j = 0; j < BM / 64; ++j) load(sa + j * MN_BLOCK, xa, am + j * 64, x);
              } else {
                load(sa, xa, x, am);
              }
              if (Op::DUAL && SPLIT) {   // 64 rows of each
                load(sb, &maps.b[0], x, tl.b_row);
                load(sb + 64 * BK * 2, &maps.b[1], x, tl.b_row);
              } else if (Op::DUAL) {     // 128 rows of one in each CTA
                load(sb, &maps.b[rank], x, tl.b_row);
              } else if (b_mn) {
#pragma unroll
                for (int j = 0; j < BROWS / 64; ++j) load(sb + j * MN_BLOCK, xb, bn + j * 64, x);
              } else {
                load(sb, xb, x, bn);
              }
              if (++stage == stages) { stage = 0; phase ^= 1u; ++issued; }
            }
          };
          by_layout<Op>(p.loop, am, bn, first, k, last, steps);
          k = last;
        }
      }
      // Every copy lands before the CTAs exit (bounded), also when another role's wait runs
      // out only after the last copy was asked for.  (A pair's odd CTA may have asked for
      // stages that the even one no longer did; after that its own roles wait out the limit.)
      if (leader)
        for (int s = 0; s < stages; ++s)   // a stage's last turn: this one, or the one before
          if (s < stage || issued > 0) tc::drain(full0 + 8 * s, (uint32_t)(s < stage ? issued : issued - 1) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0, tile = 0;
      bool ok = true;
      for (int t = tile0; t < p.loop.n_tiles && ok; t += tile_step, ++tile) {
        const uint32_t acc = tile & 1u, accph = (tile >> 1) & 1u;
        if (!tc::wait<G == 2>(acce0 + 8 * acc, accph ^ 1u, abort_flag, limit)) { ok = false; break; }
        tc::fence_after();
        const uint32_t d_tmem = tmem + acc * BN;
        // steps [from, to), with the operands' layouts known when this is compiled
        auto steps = [&](auto a_layout, auto b_layout, int from, int to) {
          constexpr bool a_mn = decltype(a_layout)::value, b_mn = decltype(b_layout)::value;
          constexpr uint32_t id = tc::idesc_16(Op::F16, a_mn, b_mn, TM, BN);
#pragma unroll 1
          for (int k = from; k < to && ok; ++k) {
            if (!tc::wait(full0 + 8 * stage, phase, abort_flag, limit)) { ok = false; break; }
            tc::fence_after();
            const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              // 16 K elements: 32 bytes inside a K-contiguous row, 16 rows of an MN-contiguous block
              const uint64_t da = a_mn ? tc::desc_mn(sa + kk * 2048, MN_BLOCK) : tc::desc_k(sa) + (uint64_t)(kk * 2);
              const uint64_t db = b_mn ? tc::desc_mn(sb + kk * 2048, MN_BLOCK) : tc::desc_k(sb) + (uint64_t)(kk * 2);
              tc::mma<G>(d_tmem, da, db, id, (k > k0 || kk > 0) ? 1u : 0u);
            }
            tc::commit<G>(empty0 + 8 * stage);
            if (++stage == stages) { stage = 0; phase ^= 1u; }
          }
        };
        int a_row = 0, b_row = 0;
        if constexpr (Op::TRI_A || Op::TRI_B) {
          const Tile tl = Op::tile(p, t, TM, OUT);
          a_row = tl.a_row;
          b_row = tl.b_row;
        }
        by_layout<Op>(p.loop, a_row, b_row, 0, k0, k1, steps);   // (mirrored operands have one part)
        if (ok) tc::commit<G>(accf0 + 8 * acc);
      }
      if (!ok) {   // every MMA already issued finishes before TMEM is freed
        tc::commit<G>(drain_bar);
        tc::drain(drain_bar, 0u);
      }
    }
  } else {
    // ------------------------------------------------------ epilogue
    // Two warps (a pair's tile: four) a TMEM quadrant (32 rows), each with its share of the
    // columns, 32 at a time.  tcgen05.ld gives a thread 32 columns of one row; a turn through
    // the warp's staging (16-byte units, swizzled) gives it 8 columns of 4 rows.
    constexpr int PARTS = EPI_WARPS / 4, WIDTH = (SPLIT ? BN : OUT) / PARTS;
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    float* st = staging + (warp - 2) * (STAGING / 4);
    uint32_t tile = 0;
    bool ok = true;
    for (int t = tile0; t < p.loop.n_tiles; t += tile_step, ++tile) {
      const Tile tl = Op::tile(p, t, TM, OUT);
      const uint32_t acc = tile & 1u, accph = (tile >> 1) & 1u;
      const int64_t row0 = tl.row + a_off + q * 32;
      const int sub = lane & 3, r8 = lane >> 2;   // 8 columns, one of 8 rows
      typename Op::Aux aux[4] = {};
      auto ask = [&](int64_t col0) {
        const int64_t col = col0 + sub * 8;
        const int n = (int)(tl.cols - col < 8 ? (tl.cols - col > 0 ? tl.cols - col : 0) : 8);
#pragma unroll
        for (int it = 0; it < 4; ++it)
          if (n > 0 && row0 + it * 8 + r8 < tl.rows) Op::aux8(p, tl, row0 + it * 8 + r8, col, n, aux[it]);
      };
      if (!SPLIT && Op::vec(p)) ask(tl.col + part * WIDTH);   // on its way while the products run
      // after a wait has run out, this tile and the CTA's later ones are NaN
      ok = __all_sync(0xFFFFFFFFu, ok && tc::wait(accf0 + 8 * acc, accph, abort_flag, limit));
      if (!ok && lane == 0) report(p.loop.status, RLK_STATUS_TIMEOUT);
      tc::fence_after();
#pragma unroll 1
      for (int ch = 0; ch < WIDTH / 32; ++ch) {
        const int c0 = part * WIDTH + ch * 32;
        const int64_t col0 = tl.col + c0;
        auto read32 = [&](float (&x)[32], int at) {
          if (ok) {
            tc::ld32(tmem + lane_base + acc * BN + at, x);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = NAN;
          }
        };
        auto release = [&] {   // when the last columns are in registers, the accumulator's next tile may begin
          if (ch != WIDTH / 32 - 1) return;
          tc::fence_before();
          __syncwarp();
          if (lane == 0 && ok) {
            if (G == 2) tc::arrive_peer(tc::peer_addr(acce0 + 8 * acc, 0u));
            else mbar_arrive(acce0 + 8 * acc);
          }
        };
        constexpr bool TWICE = Op::DUAL && !SPLIT;   // columns c and c + OUT belong together
        float v[32];
        read32(v, c0);
        if (!TWICE) release();
        if constexpr (SPLIT) {
          float* own = reinterpret_cast<float*>(base_ptr) + (q * 32 + lane) * PLD + c0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            reinterpret_cast<float4*>(own)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          if (col0 >= tl.cols) {
            if (TWICE) release();
            continue;
          }
          auto stage_in = [&](const float (&x)[32]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              reinterpret_cast<float4*>(st + lane * 32)[j ^ (lane & 7)] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            __syncwarp();
          };
          auto get8 = [&](int r, float (&x)[8]) {
            const float4* src = reinterpret_cast<const float4*>(st + r * 32);
            const float4 a = src[(2 * sub) ^ (r & 7)], b = src[(2 * sub + 1) ^ (r & 7)];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
          };
          auto get1 = [&](int r) { return st[r * 32 + ((((lane >> 2) ^ (r & 7)) << 2) | (lane & 3))]; };   // this lane's column
          const int64_t col = col0 + sub * 8;
          const int n = (int)(tl.cols - col < 8 ? (tl.cols - col > 0 ? tl.cols - col : 0) : 8);
          stage_in(v);
          if (Op::vec(p)) {
            float o[TWICE ? 4 : 1][8];
            if constexpr (TWICE) {
#pragma unroll
              for (int it = 0; it < 4; ++it) get8(it * 8 + r8, o[it]);
              __syncwarp();
              read32(v, OUT + c0);
              release();
              stage_in(v);
            }
            typename Op::Cols cols{};
            Op::cols8(p, tl, col, n, cols);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
              const int r = it * 8 + r8;
              float w[8];
              get8(r, TWICE ? w : o[0]);
              if (row0 + r < tl.rows && n > 0) Op::finish8(p, tl, row0 + r, col, n, o[TWICE ? it : 0], w, aux[it], cols);
            }
            if (ch + 1 < WIDTH / 32) ask(col0 + 32);
            __syncwarp();
          } else {
            // a lane: one column, 8 rows at a time, so that a warp stores 32 consecutive columns
            const int rows = (int)(tl.rows - row0 < 32 ? tl.rows - row0 : 32);
            float o[TWICE ? 32 : 1];
            if constexpr (TWICE) {
#pragma unroll
              for (int r = 0; r < 32; ++r) o[r] = get1(r);
              __syncwarp();
              read32(v, OUT + c0);
              release();
              stage_in(v);
            }
            if (col0 + lane < tl.cols) {
#pragma unroll
              for (int r = 0; r < 32; r += 8) {
                if (r >= rows) continue;
                float x[8], w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  w[j] = get1(r + j);
                  x[j] = TWICE ? o[TWICE ? r + j : 0] : w[j];
                }
                Op::column8(p, tl, row0 + r, 1, rows - r, col0 + lane, x, w);
              }
            }
            __syncwarp();
          }
        }
      }
    }
  }
  if constexpr (SPLIT) {
    const Tile tl = Op::tile(p, tile0, TM, OUT);
    const int width = OUT / cluster, c0 = (int)rank * width;   // this CTA's share of the columns, all rows
    const int rows = (int)(tl.rows - tl.row < BM ? tl.rows - tl.row : BM);
    // 8 columns of a row at a time, consecutive threads along a row.  What an item needs from
    // memory is asked for an item ahead.
    const int octs = width / 8, items = rows * octs;
    auto place = [&](int i, int& r, int& c, int& n) {
      r = i / octs;
      c = c0 + (i - r * octs) * 8;
      const int64_t left = tl.cols - tl.col - c;
      n = i < items ? (int)(left < 8 ? (left > 0 ? left : 0) : 8) : 0;
    };
    const bool vec = Op::vec(p);
    typename Op::Aux next{};
    if (vec) {
      int r, c, n;
      place((int)threadIdx.x, r, c, n);
      if (n > 0) Op::aux8(p, tl, tl.row + r, tl.col + c, n, next);
    }
    __syncwarp();
    tc::cluster_sync();   // every partial tile is in its CTA's shared memory
    bool dead = false;    // a wait of some CTA of the cluster ran out
    const uint32_t abort_at = smem_u32(bars + 2 * MAX_STAGES + 4);
    for (int k = 0; k < cluster; ++k) dead = tc::ld_peer_u32(tc::peer_addr(abort_at, (uint32_t)k)) != 0u || dead;
    if (dead && threadIdx.x == 0) report(p.loop.status, RLK_STATUS_TIMEOUT);
    if (vec) {
      for (int i = threadIdx.x; i < items; i += S::THREADS) {
        int r, c, n, r2, c2, n2;
        place(i, r, c, n);
        place(i + S::THREADS, r2, c2, n2);
        const typename Op::Aux aux = next;
        if (n2 > 0) Op::aux8(p, tl, tl.row + r2, tl.col + c2, n2, next);
        if (n == 0) continue;
        const int64_t col = tl.col + c;
        float v[8], u[8];
        auto add8 = [&](float (&x)[8], int at_col) {
          const uint32_t at = base + (uint32_t)(r * PLD + at_col) * 4u;
          float4 part[2 * MAX_SPLIT];   // all in flight together
#pragma unroll
          for (int k = 0; k < MAX_SPLIT; ++k)
            if (k < cluster) {
              const uint32_t peer = tc::peer_addr(at, (uint32_t)k);
              part[2 * k] = tc::ld_peer4(peer);
              part[2 * k + 1] = tc::ld_peer4(peer + 16u);
            }
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = dead ? NAN : 0.f;
#pragma unroll
          for (int k = 0; k < MAX_SPLIT; ++k)
            if (k < cluster) {
              const float4 a = part[2 * k], b = part[2 * k + 1];
              const float o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(x[j], o[j]);
            }
        };
        add8(v, c);
        if constexpr (Op::DUAL) add8(u, OUT + c);
        typename Op::Cols cols{};
        Op::cols8(p, tl, col, n, cols);
        Op::finish8(p, tl, tl.row + r, col, n, v, u, aux, cols);
      }
    } else {
      // a column a thread, 8 rows at a time
      constexpr int T = 256;
      const int c = c0 + ((int)threadIdx.x & (width - 1)), step = T / width;
      if (threadIdx.x < T && tl.col + c < tl.cols) {
        for (int r0 = (int)threadIdx.x / width; r0 < rows; r0 += step * 8) {
          float v[8], u[8];
          auto add1 = [&](float (&x)[8], int at_col) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = dead ? NAN : 0.f;
            for (int q = 0; q < cluster; ++q) {
              const uint32_t peer = tc::peer_addr(base + (uint32_t)(r0 * PLD + at_col) * 4u, (uint32_t)q);
              float part[8];   // in flight together
#pragma unroll
              for (int k = 0; k < 8; ++k) part[k] = r0 + k * step < rows ? tc::ld_peer_f32(peer + (uint32_t)(k * step * PLD) * 4u) : 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = __fadd_rn(x[k], part[k]);
            }
          };
          add1(v, c);
          if constexpr (Op::DUAL) add1(u, OUT + c);
          Op::column8(p, tl, tl.row + r0, step, rows - r0, tl.col + c, v, u);
        }
      }
    }
    tc::cluster_leave();   // no CTA leaves while its shared memory is read
  }
  tc::fence_before();
  __syncthreads();
  if (G == 2) tc::cluster_sync();   // the pair's products, copies and arrivals are all done
  tc::fence_after();
  if (warp == 1) tc::dealloc<G>(tmem, TMEM_COLS);
}

// ------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
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

// A 16-bit operand: K-contiguous ([mn][k], boxes of 64 K x box_mn rows) or MN-contiguous
// ([k][mn], boxes of 64 columns x 64 K rows); what lies past its extents reads as 0.
struct Operand {
  const void* p;
  int64_t ld;
};
inline bool make_map(CUtensorMap* map, bool f16, const Operand& o, bool mn_major, int64_t mn, int64_t k, uint32_t box_mn = BROWS) {
  EncodeTiledFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(mn_major ? mn : k), (cuuint64_t)(mn_major ? k : mn)};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
  const cuuint32_t box[2] = {64u, mn_major ? 64u : box_mn};
  const cuuint32_t estr[2] = {1, 1};
  return f(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(o.p), dims, strides,
           box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Op, bool SPLIT>
cudaError_t set_smem() {
  static std::atomic<int> done[64];
  const int ds = device_slot();
  if (ds >= 0 && done[ds].load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(gemm_tiles_kernel<Op, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Shape<SPLIT>::smem(Shape<SPLIT>::STAGES));
  if (e == cudaSuccess && ds >= 0) done[ds].store(1);
  return e;
}

// CTAs that share a tile's K when there are `tiles` tiles of 128 x 128: 2 or 4 while all have
// an SM and two stages of K each, or half an SM and at least eight.  (40 tiles of 16 stages by
// 4 on 152 SMs, eight of which then have two CTAs: 1.8 us slower than by 2.)
inline int split_for(int tiles, int k_steps) {
  int s = 1;
  while (s < MAX_SPLIT && ((k_steps >= 4 * s && tiles * 2 * s <= sm_count()) || (k_steps >= 16 * s && tiles * 2 * s <= 2 * sm_count()))) s *= 2;
  return s;
}

// One launch over p.loop.n_tiles tiles, as a programmatic dependent of the kernel before it.
template <class Op, bool SPLIT>
cudaError_t launch(const MapsOf<Op>& maps, typename Op::Params p, cudaStream_t stream) {
  if (cudaError_t e = set_smem<Op, SPLIT>(); e != cudaSuccess) return e;
  const int tiles = p.loop.n_tiles, split = SPLIT ? split_for(tiles, p.loop.k_steps) : 1;
  if (!SPLIT || p.loop.a_rows == 0) p.loop.a_rows = BM;
  if (p.loop.part_steps == 0) p.loop.part_steps = p.loop.k_steps;
  p.loop.wait_limit = debug_wait_limit();
  p.loop.withhold = (int)debug_take_withheld();
  p.loop.stages = SPLIT && tiles * split > sm_count() ? FEW_STAGES : Shape<SPLIT>::STAGES;
  cudaLaunchConfig_t cfg{};
  const int pairs = sm_count() / 2;
  cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * split : 2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(Shape<SPLIT>::THREADS);
  cfg.dynamicSmemBytes = Shape<SPLIT>::smem(p.loop.stages);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_tiles_kernel<Op, SPLIT>, maps, p, split);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gemm
}  // namespace rlk
