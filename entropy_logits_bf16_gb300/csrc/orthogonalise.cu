// rlk_orthogonalise: the polar factor of an update, nearly, by Newton-Schulz products.
//
//   X_0 = G / (|G|_F + eps);   A = X X^T,  P = b A + c A^2,  X <- a X + P X,  `steps` times
// (rows <= columns; else A = X^T X and X <- a X + X P).  Each step maps the singular values by
// s -> a s + b s^3 + c s^5 and leaves the singular vectors.
//
// Up to 128 x 1024 one kernel for all steps (below).  Else three products a step on the tcgen05
// kernel of gemm.cuh.  A and P are symmetric: only their
// blocks of 256 x 256 (or 128 x 128) on and below the diagonal are computed and stored, and a product takes a
// missing block as the mirror image of the one that is there, with the other index contiguous
// (storing each twice took a third of these products' epilogues).  Nothing is transposed in
// memory: X too is taken with its rows' or its columns' index contiguous.  A stack of matrices
// is one launch a product, by three-dimensional tensor maps.
//
// Numbers.  The products' operands are fp16 (11 bits where bf16 has 8, at the same rate), held
// times 2^10: the iterates' entries lie between about 1 / (longer side) and 1.2, so that a matrix
// of up to 2^14 on a side keeps its typical entries among fp16's normal numbers, and the entries
// of A and P may grow to 63.9 (A's diagonal are the squared norms of X's rows, so those to 7.99 and
// X's entries no further).  What passes that is infinite, and the result is then NaN or infinite
// (b times an infinite A is NaN even for b = 0), which the last product reports.  X is held in two fp16 (value and rest, 22 bits), since a X carries the small
// singular values on unrounded: with one, each step's rounding noise is multiplied by a like
// they are (an update of rank 64 over noise 1 / 50 of it: 0.013 of the result off, with two
// 0.0004; bf16 0.11).
// The rounding of A, P and X moves each singular value by up to 0.05 of it in five steps (the
// polynomial's slope adds up: first-order sum over the steps with u = 2^-11), about 0.0015 on
// the average of many.  Where the shorter side is kPrecise or less there may be few to average
// over, and the call is bound by its chain: A and P are held in two fp16 as well, and each
// product is three (values, value times rest both ways), one sum in the accumulator (as launches,
// replayed: 64 x 64 109 us, 98 with one product each; 256 x 256 144 and 123).  The errors add up less well
// where few directions or many steps count (2-norm, the bf16 rounding's 0.0017 included: noise 0.0021 to 0.0024,
// 300 x 700 with one row of numbers 0.0040, ten steps on 300 x 700 0.0045).
//
// Measured (replayed graphs, the start included): 4096 x 14336 2.84 to 3.0 ms (1.32 to 1.39 PFLOP/s with halves of
// A and P counted; A 86 % of the tensor pipe, X 61 to 70 %: operands at the 64 bytes a cycle that an SM takes
// from L2, and 16 bytes an element in its epilogue), 4096 x 4096 1.0 to 1.09 ms, 24 x 512 x 1024 311 to 338 us,
// 2731 x 1003 228 to 237 us, 256 x 256 122 to 126 us: the last three by what a launch costs besides its products
// (8 to 15 us each, 17 launches).
#include <cuda_fp16.h>
#include <math.h>

#include "activation.cuh"
#include "gemm.cuh"

namespace rlk {
namespace {

using gemm::Loop;
using gemm::Tile;
using gemm::report;

constexpr float kDown = 1.f / 1024.f;   // the operands' scale is 2^10
constexpr int kPrecise = 128;

// Whether one of the first n is infinite or NaN (0 times it is NaN).
__device__ __forceinline__ bool not_finite(const float (&v)[8], int n) {
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) z = __fmaf_rn(v[j], 0.f, z);
  return z != 0.f;
}

int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// Eight numbers as four pairs.
__device__ __forceinline__ void halves(const uint4& q, float2 (&v)[4]) {
  v[0] = unpack_half(q.x);
  v[1] = unpack_half(q.y);
  v[2] = unpack_half(q.z);
  v[3] = unpack_half(q.w);
}
__device__ __forceinline__ uint4 to_halves(const float2 (&v)[4]) {
  return make_uint4(pack_half(v[0].x, v[0].y), pack_half(v[1].x, v[1].y), pack_half(v[2].x, v[2].y), pack_half(v[3].x, v[3].y));
}

// A stack of B matrices of the iteration, each number in two fp16 (rest may be NULL: one); rows
// of pad8(columns), columns past the end hold anything.
struct Buffer {
  uint16_t *value, *rest;
  int64_t ld, matrix;   // strides in elements
  __device__ __forceinline__ int64_t at(int b, int64_t row, int64_t col) const { return b * matrix + row * ld + col; }
  __device__ __forceinline__ void store8(int64_t i, const float2 (&v)[4]) const {
    const uint4 h = to_halves(v);
    *reinterpret_cast<uint4*>(value + i) = h;
    if (!rest) return;
    float2 x[4];
    halves(h, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = fma2(x[j], both(-1.f), v[j]);
    *reinterpret_cast<uint4*>(rest + i) = to_halves(x);
  }
};
// 8 numbers of one, asked for ahead.
struct Eight {
  uint4 value, rest;
  __device__ __forceinline__ void ask(const Buffer& b, int64_t i) {
    value = *reinterpret_cast<const uint4*>(b.value + i);
    if (b.rest) rest = *reinterpret_cast<const uint4*>(b.rest + i);
  }
  // their product with f, plus v
  __device__ __forceinline__ void add_to(const Buffer& b, float f, float2 (&v)[4]) const {
    float2 x[4];
    halves(value, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fma2(x[j], both(f), v[j]);
    if (!b.rest) return;
    halves(rest, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fma2(x[j], both(f), v[j]);
  }
};
// A product is one or three sums (parts): values, values times rest, rest times values.
__device__ __forceinline__ void of_three(int part, int& ia, int& ib) {
  ia = part == 2;
  ib = part == 1;
}

// Tile t of stacked matrices, `per` tiles each; tri: of the blocks of tri x tri on and below the
// diagonal, row by row (a block is a tile, or four).
__device__ __forceinline__ Tile stacked(int t, int per, int n_mt, int n_nt, int tm, int tn, int64_t rows, int64_t cols, int tri) {
  const int b = t / per, r = t - b * per;
  int mt, nt;
  if (tri) {
    const int in = tri / tm, q = r / (in * in), u = r - q * in * in;   // in: 1 or 2
    mt = (int)((sqrtf(8.f * (float)q + 1.f) - 1.f) * 0.5f);                   // row mt starts at mt (mt + 1) / 2
    while ((mt + 1) * (mt + 2) / 2 <= q) ++mt;
    while (mt * (mt + 1) / 2 > q) --mt;
    nt = (q - mt * (mt + 1) / 2) * in + u % in;
    mt = mt * in + u / in;
  } else {
    gemm::grouped(r, n_mt, n_nt, mt, nt);
  }
  return Tile{mt * tm, nt * tn, (int64_t)mt * tm, (int64_t)nt * tn, rows, cols, b};
}

// A = X X^T (MN: X^T X), and P = b A + c A A (POLY).
template <bool MN, bool POLY>
struct SquareOp {
  static constexpr bool A_MN = MN, B_MN = MN, F16 = true, DUAL = false, STACKED = true, TRI_A = POLY, TRI_B = POLY;
  struct Params {
    Loop loop;
    int per, side;
    int whole;         // tiles a side where all are computed, 0: the blocks on and below the diagonal
    float scale, b;    // of the accumulators; of A (POLY)
    Buffer a, out;
  };
  static __device__ __forceinline__ Tile tile(const Params& p, int t, int tm, int tn) {
    return stacked(t, p.per, p.whole, p.whole, tm, tn, p.side, p.side, p.loop.tri);
  }
  static __device__ __forceinline__ void source(const Tile&, int part, int& ia, int& ib) { of_three(part, ia, ib); }
  static __device__ __forceinline__ bool vec(const Params&) { return true; }
  struct Aux {
    Eight a;
  };
  static __device__ __forceinline__ void aux8(const Params& p, const Tile& tl, int64_t row, int64_t col, int, Aux& x) {
    if (POLY) x.a.ask(p.a, p.a.at(tl.which, row, col));
  }
  struct Cols {};
  static __device__ __forceinline__ void cols8(const Params&, const Tile&, int64_t, int, Cols&) {}
  static __device__ __forceinline__ void finish8(const Params& p, const Tile& tl, int64_t row, int64_t col, int, float (&v)[8],
                                                 float (&)[8], const Aux& x, const Cols&) {
    float2 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = mul2(make_float2(v[2 * j], v[2 * j + 1]), both(p.scale));
    if (POLY) x.a.add_to(p.a, p.b, o);
    p.out.store8(p.out.at(tl.which, row, col), o);   // rows are padded to 8 columns
  }
  static __device__ __forceinline__ void column8(const Params&, const Tile&, int64_t, int, int, int64_t, float (&)[8], float (&)[8]) {}
};

// X <- a X + P X (TALL: a X + X P), to two fp16 or, the last time, to the caller's bf16.
template <bool TALL>
struct ApplyOp {
  static constexpr bool A_MN = false, B_MN = !TALL, F16 = true, DUAL = false, STACKED = true, TRI_A = !TALL, TRI_B = TALL;
  struct Params {
    Loop loop;
    int per, n_mt, n_nt;
    int64_t m, n;
    float a;
    Buffer x, to;
    uint16_t* out;          // bf16, or NULL
    int64_t ldo, out_matrix;
    int out_vec;            // its rows start on 16-byte boundaries
  };
  static __device__ __forceinline__ Tile tile(const Params& p, int t, int tm, int tn) {
    return stacked(t, p.per, p.n_mt, p.n_nt, tm, tn, p.m, p.n, 0);
  }
  static __device__ __forceinline__ void source(const Tile&, int part, int& ia, int& ib) { of_three(part, ia, ib); }
  static __device__ __forceinline__ bool vec(const Params& p) { return !p.out || p.out_vec; }
  struct Aux {
    Eight x;
  };
  static __device__ __forceinline__ void aux8(const Params& p, const Tile& tl, int64_t row, int64_t col, int, Aux& x) {
    x.x.ask(p.x, p.x.at(tl.which, row, col));
  }
  struct Cols {};
  static __device__ __forceinline__ void cols8(const Params&, const Tile&, int64_t, int, Cols&) {}
  static __device__ __forceinline__ void finish8(const Params& p, const Tile& tl, int64_t row, int64_t col, int n, float (&v)[8],
                                                 float (&)[8], const Aux& x, const Cols&) {
    float2 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = mul2(make_float2(v[2 * j], v[2 * j + 1]), both(kDown));
    x.x.add_to(p.x, p.a, o);
    if (p.out) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __fmul_rn(o[j].x, kDown);
        v[2 * j + 1] = __fmul_rn(o[j].y, kDown);
      }
      store8(p.out + tl.which * p.out_matrix + row * p.ldo + col, v, n);
      if (not_finite(v, n)) report(p.loop.status, RLK_STATUS_NONFINITE);
      return;
    }
    p.to.store8(p.to.at(tl.which, row, col), o);
  }
  // the caller's rows that do not start on 16-byte boundaries
  static __device__ __forceinline__ void column8(const Params& p, const Tile& tl, int64_t row, int step, int n, int64_t col,
                                                 float (&v)[8], float (&)[8]) {
    uint16_t h[8], r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t at = p.x.at(tl.which, row + k * step, col);
      h[k] = k * step < n ? p.x.value[at] : 0u;
      r[k] = k * step < n ? p.x.rest[at] : 0u;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = __fadd_rn(unpack_half(h[k]).x, unpack_half(r[k]).x);
      const float y = __fmul_rn(__fmaf_rn(v[k], kDown, __fmul_rn(p.a, x)), kDown);
      if (k * step < n) {
        p.out[tl.which * p.out_matrix + (row + k * step) * p.ldo + col] = (uint16_t)pack_bf16(y, 0.f);
        if (!isfinite(y)) report(p.loop.status, RLK_STATUS_NONFINITE);
      }
    }
  }
};

// ------------------------------------------------------------ the start
constexpr int OT = 256;
constexpr int kNormParts = 512;   // most parts of a matrix's sum

// 8 columns of a row as floats, 0 past the end; vec: rows start on 16-byte boundaries.
template <int DT>
__device__ __forceinline__ void load8(const void* g, int64_t at, int n, bool vec, float (&v)[8]) {
  if (DT == 0) {
    const uint16_t* p = static_cast<const uint16_t*>(g) + at;
    if (vec && n == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(w[j]);
        v[2 * j + 1] = bf16_hi(w[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? bf16_val(p[j]) : 0.f;
    }
  } else {
    const float* p = static_cast<const float*>(g) + at;
    if (vec && n == 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.f;
    }
  }
}

// Sums of squares in three ranges, so that none over- or underflows: of numbers of 2^40 and
// more (times 2^-96), of less than 2^-40 (times 2^80: the sum of 2^32 squares stays under 2^112,
// and the least number's square is 2^-138), of the others; a group of 8 goes by its largest.
struct Squares {
  float small, mid, big;
};
constexpr float kBig = 0x1p40f, kSmall = 0x1p-40f;
__device__ __forceinline__ void add_squares(Squares& s, const float (&v)[8]) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
  const float f = top >= kBig ? 0x1p-96f : (top < kSmall ? 0x1p80f : 1.f);
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = __fmul_rn(v[j], f);
    sum = __fmaf_rn(x, x, sum);
  }
  if (top >= kBig) s.big = __fadd_rn(s.big, sum);
  else if (top < kSmall) s.small = __fadd_rn(s.small, sum);
  else s.mid = __fadd_rn(s.mid, sum);
}

struct Start {
  const void* g;
  int64_t ldg, g_matrix;
  int64_t m, n;
  int vec;
  float eps;
  int parts;             // of a matrix's sum
  Squares* sums;         // [B][parts]
  Buffer x;
  uint32_t* status;
};

template <int DT>
__global__ void __launch_bounds__(OT) orth_norm_kernel(const Start a) {
  pdl_trigger();
  const int b = blockIdx.y;
  const int64_t base = b * a.g_matrix;
  const unsigned octs = (unsigned)(a.n + 7) / 8, all = (unsigned)a.m * octs, step = (unsigned)a.parts * OT;
  Squares s{0.f, 0.f, 0.f};
#pragma unroll 2
  for (unsigned i = blockIdx.x * OT + threadIdx.x; i < all; i += step) {
    const unsigned r = i / octs, c = (i - r * octs) * 8;
    float v[8];
    load8<DT>(a.g, base + r * a.ldg + c, a.n - c < 8 ? (int)(a.n - c) : 8, a.vec, v);
    add_squares(s, v);
  }
  __shared__ Squares sh[OT / 32];
  float w[3] = {s.small, s.mid, s.big};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) w[k] = __fadd_rn(w[k], __shfl_xor_sync(0xFFFFFFFFu, w[k], o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = Squares{w[0], w[1], w[2]};
  __syncthreads();
  if (threadIdx.x == 0) {
    Squares t = sh[0];
    for (int k = 1; k < OT / 32; ++k) {
      t.small = __fadd_rn(t.small, sh[k].small);
      t.mid = __fadd_rn(t.mid, sh[k].mid);
      t.big = __fadd_rn(t.big, sh[k].big);
    }
    a.sums[b * a.parts + blockIdx.x] = t;
  }
}

// X_0 = G times one factor, as two powers of two and a number in [1, 2) (the factor itself may
// be outside fp32's range).
template <int DT>
__global__ void __launch_bounds__(OT) orth_start_kernel(const Start a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float s_f[3];
  const int b = blockIdx.y;
  if (threadIdx.x < 32) {
    float s[3] = {0.f, 0.f, 0.f};
    Squares q[kNormParts / 32];   // all in flight together
#pragma unroll
    for (int k = 0; k < kNormParts / 32; ++k)
      q[k] = (int)threadIdx.x + 32 * k < a.parts ? a.sums[b * a.parts + threadIdx.x + 32 * k] : Squares{0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kNormParts / 32; ++k) {
      s[0] = __fadd_rn(s[0], q[k].small);
      s[1] = __fadd_rn(s[1], q[k].mid);
      s[2] = __fadd_rn(s[2], q[k].big);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < 3; ++k) s[k] = __fadd_rn(s[k], __shfl_xor_sync(0xFFFFFFFFu, s[k], o));
    if (threadIdx.x == 0) {
      // the norm plus eps as n 2^e, in fp32 (in fp64, which runs at 1/64 of its rate here, this kernel took 8 us)
      float n;
      int e;
      if (s[2] > 0.f) {          // n from 2^-56 to 2^48
        e = 96;
        n = __fadd_rn(sqrtf(__fadd_rn(s[2], __fmul_rn(__fmul_rn(s[1], 0x1p-96f), 0x1p-96f))), __fmul_rn(a.eps, 0x1p-96f));
      } else if (s[1] > 0.f || a.eps >= kSmall) {
        e = 0;
        n = __fadd_rn(sqrtf(__fadd_rn(s[1], __fmul_rn(__fmul_rn(s[0], 0x1p-80f), 0x1p-80f))), a.eps);
      } else {                   // up to 2^56
        e = -80;
        n = __fadd_rn(sqrtf(s[0]), __fmul_rn(a.eps, 0x1p80f));
      }
      const bool finite = isfinite(s[0]) && isfinite(s[1]) && isfinite(s[2]) && isfinite(n);
      if (!finite) {
        s_f[0] = NAN;
        s_f[1] = s_f[2] = 1.f;
        if (blockIdx.x == 0) report(a.status, RLK_STATUS_NONFINITE);
      } else if (n == 0.f) {   // eps is 0 and so is G
        s_f[0] = 0.f;
        s_f[1] = s_f[2] = 1.f;
      } else {
        int of_n;
        s_f[0] = __frcp_rn(frexpf(n, &of_n));   // in (1, 2]
        e += of_n;
        s_f[1] = ldexpf(1.f, -(e / 2) + 5);     // and times 2^10
        s_f[2] = ldexpf(1.f, -(e - e / 2) + 5);
      }
    }
  }
  __syncthreads();
  const float f0 = s_f[0], f1 = s_f[1], f2 = s_f[2];
  const int64_t base = b * a.g_matrix;
  const unsigned octs = (unsigned)(a.n + 7) / 8, all = (unsigned)a.m * octs, step = gridDim.x * OT;
#pragma unroll 2
  for (unsigned i = blockIdx.x * OT + threadIdx.x; i < all; i += step) {
    const unsigned r = i / octs, c = (i - r * octs) * 8;
    float v[8];
    load8<DT>(a.g, base + r * a.ldg + c, a.n - c < 8 ? (int)(a.n - c) : 8, a.vec, v);
    float2 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(mul2(make_float2(v[2 * j], v[2 * j + 1]), both(f1)), both(f2)), both(f0));
    a.x.store8(a.x.at(b, r, c), x);
  }
}

// ------------------------------------------------------------ small matrices, in one kernel
// Up to 128 x 1024 (either way) the whole iteration stays in the shared memory of a cluster: a
// CTA holds 128 of the longer side's columns (TALL: rows) of X, both halves of each number, and
// all of A, then P, in the 128-byte swizzle that TMA brought X in.  The same bytes are a K-contiguous
// operand where X's columns are summed over and an MN-contiguous one where its rows are.  A step:
// each CTA's share of A in TMEM; the shares joined through distributed shared memory, each CTA
// its part of A for all (in rank order: the same bits in all); A A, P and X's product locally.
// Bound by the chain of a step's products and epilogues, about 6 us where there is one CTA, 14
// with eight (replayed, the start included: one 64 x 64 37 us where 17 launches take 109, 128 x 512
// 64 and 138, 128 x 1024 78 and 146): a chain of latencies, the tensor pipe 37 % busy and the issue slots 25 % (twice the threads change nothing;
// fences of all memory instead of this CTA's shared memory cost 3 us).
constexpr int RT = 256, RES_MOST = 8;   // threads; CTAs of a cluster, 128 of the longer side each
constexpr uint32_t RES_HALF = 128 * 128 * 2, RES_PITCH = 132;   // bytes of 128 x 128 fp16; floats of a row of shares
constexpr size_t RES_SMEM = 4 * RES_HALF + 128 * RES_PITCH * 4 + 1024 + 64;

struct Resident {
  int64_t m, n;
  int steps, cluster;
  float a, b, c;
  uint16_t* out;          // bf16
  int64_t ldo, out_matrix;
  int out_vec;
  uint32_t* status;
  long long limit;
  int withhold;           // debug: the first CTA's load waits for an arrival that never comes
};
struct Halves {
  CUtensorMap value, rest;
};

__device__ __forceinline__ void store_peer16(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <bool TALL>
__global__ void __launch_bounds__(RT, 1) orth_resident_kernel(const __grid_constant__ Halves maps, const Resident p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* mem = smem_raw + (base - raw);
  constexpr uint32_t XH = 0, XL = RES_HALF, AH = 2 * RES_HALF, AL = 3 * RES_HALF, F = 4 * RES_HALF;
  uint64_t* bars = reinterpret_cast<uint64_t*>(mem + F + 128 * RES_PITCH * 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 3);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4);
  const uint32_t loaded = smem_u32(bars), done = loaded + 8, drain_bar = loaded + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = p.cluster;
  const int rank = (int)tc::cluster_rank(), matrix = (int)(blockIdx.x / (unsigned)C);
  const int row = (warp & 3) * 32 + lane, half = warp >> 2;   // this thread's row of a 128 x 128 tile, and 64 of its columns
  if (threadIdx.x == 0) {
    mbar_init(loaded, 1 + (p.withhold >= 0 && blockIdx.x == 0));
    mbar_init(done, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tc::prefetch_map(&maps.value);
    tc::prefetch_map(&maps.rest);
  }
  if (warp == 0) tc::alloc<1>(smem_u32(tmem_slot), 128);
  tc::fence_before();
  __syncthreads();
  pdl_trigger();   // the next kernel's CTAs may come: this one has its TMEM
  pdl_wait();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) {
    mbar_expect_tx(loaded, 2 * RES_HALF);
#pragma unroll
    for (int b = 0; b < 2; ++b) {   // 64 columns a block of 128 rows
      const int x = TALL ? b * 64 : rank * 128 + b * 64, y = TALL ? rank * 128 : 0;
      tc::load_3d(base + XH + b * (RES_HALF / 2), &maps.value, loaded, x, y, matrix);
      tc::load_3d(base + XL + b * (RES_HALF / 2), &maps.rest, loaded, x, y, matrix);
    }
  }
  bool ok = tc::wait(loaded, 0u, abort_flag, p.limit);
  uint32_t phase = 0u;

  // where 8 numbers of a row lie (unit: 8 columns)
  auto at = [](int r, int unit) { return (uint32_t)((unit >> 3) * (int)(RES_HALF / 2) + r * 128 + (((unit & 7) ^ (r & 7)) << 4)); };
  // D = A B^T of three terms, K 128; then every thread waits for it
  auto product = [&](auto a_layout, auto b_layout, uint32_t a_value, uint32_t a_rest, uint32_t b_value, uint32_t b_rest) {
    constexpr bool a_mn = decltype(a_layout)::value, b_mn = decltype(b_layout)::value;
    constexpr uint32_t id = tc::idesc_16(true, a_mn, b_mn, 128, 128);
    if (threadIdx.x == 0 && !*abort_flag) {
      fence_proxy_async_smem();
      tc::fence_after();
#pragma unroll 1
      for (int term = 0; term < 3; ++term) {
        const uint32_t a = base + (term == 2 ? a_rest : a_value), b = base + (term == 1 ? b_rest : b_value);
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // 16 of K: 32 bytes of a K-contiguous row, 16 rows of MN-contiguous blocks
          const uint64_t da = a_mn ? tc::desc_mn(a + i * 2048, RES_HALF / 2) : tc::desc_k(a + (i >> 2) * (RES_HALF / 2)) + (uint64_t)((i & 3) * 2);
          const uint64_t db = b_mn ? tc::desc_mn(b + i * 2048, RES_HALF / 2) : tc::desc_k(b + (i >> 2) * (RES_HALF / 2)) + (uint64_t)((i & 3) * 2);
          tc::mma<1>(tmem, da, db, id, (term > 0 || i > 0) ? 1u : 0u);
        }
      }
      tc::commit<1>(done);
    }
    ok = ok && tc::wait(done, phase, abort_flag, p.limit);
    phase ^= 1u;
    tc::fence_after();
  };
  float v[2][32];
  auto read = [&] {   // this thread's 64 numbers of D
    const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 64;
    const bool good = __all_sync(0xFFFFFFFFu, ok);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (good) {
        tc::ld32(from + h * 32, v[h]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[h][j] = NAN;
      }
    }
    tc::fence_before();
  };
  auto eight = [&](int j, float f, float2 (&o)[4]) {   // group j of the 64, times f
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul2(make_float2(v[j >> 2][(j & 3) * 8 + 2 * i], v[j >> 2][(j & 3) * 8 + 2 * i + 1]), both(f));
  };
  auto add_kept = [&](uint32_t value, uint32_t rest, uint32_t off, float f, float2 (&o)[4]) {
    float2 x[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      halves(*reinterpret_cast<const uint4*>(mem + (k ? rest : value) + off), x);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fma2(x[i], both(f), o[i]);
    }
  };
  auto split = [&](const float2 (&o)[4], uint4& value, uint4& rest) {
    float2 x[4];
    value = to_halves(o);
    halves(value, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fma2(x[i], both(-1.f), o[i]);
    rest = to_halves(x);
  };
  auto keep = [&](uint32_t value, uint32_t rest, uint32_t off, const float2 (&o)[4]) {
    uint4 h, l;
    split(o, h, l);
    *reinterpret_cast<uint4*>(mem + value + off) = h;
    *reinterpret_cast<uint4*>(mem + rest + off) = l;
  };
  using K = std::false_type;    // K-contiguous
  using MN = std::true_type;    // MN-contiguous

  for (int step = 0; step < p.steps; ++step) {
    // A = X X^T (TALL: X^T X)
    product(std::bool_constant<TALL>{}, std::bool_constant<TALL>{}, XH, XL, XH, XL);
    read();
    if (C == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float2 o[4];
        eight(j, kDown, o);
        keep(AH, AL, at(row, half * 8 + j), o);
      }
      fence_proxy_async_smem();
      __syncthreads();
    } else {
      float4* share = reinterpret_cast<float4*>(mem + F + (row * RES_PITCH + half * 64) * 4);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        share[j] = make_float4(v[j >> 3][(j & 7) * 4], v[j >> 3][(j & 7) * 4 + 1], v[j >> 3][(j & 7) * 4 + 2], v[j >> 3][(j & 7) * 4 + 3]);
      tc::cluster_sync();   // all shares are there, and every CTA is through with P
      const int first = 2048 * rank / C, last = 2048 * (rank + 1) / C;   // groups of 8: 16 a row
      for (int i = first + (int)threadIdx.x; i < last; i += RT) {
        const int r = i >> 4, u = i & 15;
        const uint32_t from = base + F + (uint32_t)(r * (int)RES_PITCH + u * 8) * 4u;
        float4 q[2 * RES_MOST];   // all in flight together
#pragma unroll
        for (int k = 0; k < RES_MOST; ++k)
          if (k < C) {
            const uint32_t peer = tc::peer_addr(from, (uint32_t)k);
            q[2 * k] = tc::ld_peer4(peer);
            q[2 * k + 1] = tc::ld_peer4(peer + 16u);
          }
        float2 o[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
        for (int k = 0; k < RES_MOST; ++k)
          if (k < C) {
            o[0] = add2(o[0], make_float2(q[2 * k].x, q[2 * k].y));
            o[1] = add2(o[1], make_float2(q[2 * k].z, q[2 * k].w));
            o[2] = add2(o[2], make_float2(q[2 * k + 1].x, q[2 * k + 1].y));
            o[3] = add2(o[3], make_float2(q[2 * k + 1].z, q[2 * k + 1].w));
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = mul2(o[k], both(kDown));
        uint4 h, l;
        split(o, h, l);
        const uint32_t to = at(r, u);
#pragma unroll
        for (int k = 0; k < RES_MOST; ++k)
          if (k < C) {
            store_peer16(tc::peer_addr(base + AH + to, (uint32_t)k), h);
            store_peer16(tc::peer_addr(base + AL + to, (uint32_t)k), l);
          }
      }
      fence_proxy_async();
      __syncwarp();
      tc::cluster_sync();   // A is whole in every CTA
    }
    // P = b A + c A A, in A's place
    product(K{}, K{}, AH, AL, AH, AL);
    read();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 o[4];
      const uint32_t off = at(row, half * 8 + j);
      eight(j, p.c * kDown, o);
      add_kept(AH, AL, off, p.b, o);
      keep(AH, AL, off, o);
    }
    fence_proxy_async_smem();
    __syncthreads();
    // X <- a X + P X (TALL: a X + X P)
    if constexpr (TALL) product(K{}, K{}, XH, XL, AH, AL);
    else product(K{}, MN{}, AH, AL, XH, XL);
    read();
    if (step == p.steps - 1) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 o[4];
      const uint32_t off = at(row, half * 8 + j);
      eight(j, kDown, o);
      add_kept(XH, XL, off, p.a, o);
      keep(XH, XL, off, o);
    }
    fence_proxy_async_smem();
    __syncthreads();
  }
  // a wait that ran out in one CTA spoils the matrix
  __syncthreads();
  tc::cluster_sync();
  bool dead = false;
  for (int k = 0; k < C; ++k) dead = tc::ld_peer_u32(tc::peer_addr(smem_u32(bars + 3), (uint32_t)k)) != 0u || dead;
  if (dead && threadIdx.x == 0) report(p.status, RLK_STATUS_TIMEOUT);
  const int64_t r0 = TALL ? rank * 128 + row : row, c0 = (TALL ? 0 : rank * 128) + half * 64;
  if (r0 < p.m) {
    uint16_t* to = p.out + matrix * p.out_matrix + r0 * p.ldo + c0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int n = (int)(p.n - c0 - j * 8 < 8 ? p.n - c0 - j * 8 : 8);
      if (n <= 0) continue;
      float2 o[4];
      eight(j, kDown, o);
      add_kept(XH, XL, at(row, half * 8 + j), p.a, o);
      float w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = dead ? NAN : __fmul_rn(o[i].x, kDown);
        w[2 * i + 1] = dead ? NAN : __fmul_rn(o[i].y, kDown);
      }
      if (not_finite(w, n)) report(p.status, RLK_STATUS_NONFINITE);
      if (p.out_vec) {
        store8(to + j * 8, w, n);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) to[j * 8 + i] = (uint16_t)pack_bf16(w[i], 0.f);
      }
    }
  }
  if (threadIdx.x == 0 && *abort_flag) {   // what was asked for has landed, and been multiplied, before the CTA exits
    if (p.withhold >= 0 && blockIdx.x == 0) mbar_arrive(loaded);
    tc::drain(loaded, 0u);
    tc::commit<1>(drain_bar);
    tc::drain(drain_bar, 0u);
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_leave();   // no CTA leaves while its shared memory is read
  tc::fence_after();
  if (warp == 0) tc::dealloc<1>(tmem, 128);
}

// ------------------------------------------------------------ host side
struct Layout {
  int64_t side, x_ld, p_ld;
  int parts;
  bool precise;
  size_t x, p, sums;    // bytes of a stack of X, of A or P (one fp16 a number), of the sums
  size_t total() const { return 4 * x + (precise ? 4 : 2) * p + sums; }
};
Layout layout(int64_t B, int64_t m, int64_t n) {
  Layout l{};
  l.side = m < n ? m : n;
  l.precise = l.side <= kPrecise;
  l.x_ld = pad8(n);
  l.p_ld = pad8(l.side);
  // a part: two groups of 8 numbers a thread or more, and about 1200 parts in all
  const int64_t octs = m * ((n + 7) / 8), most = B < 3 ? kNormParts : 1216 / B + 1;
  const int64_t parts = (octs + OT * 2 - 1) / (OT * 2);
  l.parts = (int)(parts > most ? most : parts);
  l.x = pad256((size_t)B * m * l.x_ld * 2);
  l.p = pad256((size_t)B * l.side * l.p_ld * 2);
  l.sums = pad256((size_t)B * l.parts * sizeof(Squares));
  return l;
}

// Whether the rows of the caller's result start on 16-byte boundaries.
bool out_vec(const OrthArgs& a) {
  return reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && (a.m == 1 || a.ldo % 8 == 0) && (a.B == 1 || a.out_matrix % 8 == 0);
}

// Maps of a stack of [rows][cols] matrices: boxes of 64 columns and `box` rows.
bool stack_map(CUtensorMap* map, void* p, const Buffer& o, int64_t B, int64_t rows, int64_t cols, uint32_t box) {
  gemm::EncodeTiledFn f = gemm::encode_fn();
  if (!f) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)B};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.matrix * 2};
  const cuuint32_t boxes[3] = {64u, box, 1u}, estr[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tiles of the products: small ones where there is an SM for each, else pairs', as for the
// linear layer.  Of A and P all where there are SMs for all with K split by four; else the
// blocks on and below the diagonal, of 128 where X's tiles are small ones too.  A pair's tile
// needs blocks of 256, so X's are also small ones, two an SM, where those of A and P then get K
// split by four and with blocks of 256 would not.  Replayed, us, blocks of 128 with small tiles for X
// and blocks of 256: inside those limits 896 x 2560 191 and 211, 1024 x 4096 223 and 241, 1024 x 4864
// 230 and 247, 2 of 640 x 3584 207 and 264; outside 640 x 4096 203 and 198 (K split by four both ways),
// 768 x 4096 212 and 203, 3 of 512 x 2560 194 and 189, 1152 x 2560 243 and 234.  All of A where there is an SM
// for a quarter of each tile: 384 x 3200, four of them 220, blocks of 128 192, of 256 253; 3 of 512 x 1536 162 as
// all, 173.  (The limits lose at 1152 x 4096, 259 and 290, and 2 of 768 x 3200, 235 and 258.)
struct Cover {
  bool few, x_few;
  int whole, tri, per;   // tiles a side where all of A's are there, else 0; blocks' side, or 0; A's tiles of a matrix
  bool fits;
};
Cover cover(int64_t B, int64_t m, int64_t n) {
  const int64_t side = m < n ? m : n, sms = sm_count(), t = (side + 127) / 128, u = (side + 255) / 256;
  const int64_t of128 = B * t * (t + 1) / 2, of256 = B * u * (u + 1) / 2, x_small = B * ((m + 127) / 128) * ((n + 127) / 128);
  Cover c{};
  c.x_few = m <= 128 || x_small <= sms;
  if (side <= 128 || 4 * B * t * t <= sms) {
    c.few = true;
    c.whole = (int)t;
  } else if (of128 <= sms && (c.x_few || (x_small <= 2 * sms && 4 * of128 <= sms && 16 * of256 > sms))) {
    c.few = c.x_few = true;
    c.tri = 128;
  } else {
    c.few = 4 * of256 <= sms;
    c.tri = 256;
  }
  const int64_t per = c.whole ? t * t : (c.tri == 128 ? t * (t + 1) / 2 : u * (u + 1) / 2 * (c.few ? 4 : 1));
  c.per = (int)per;
  c.fits = B * per <= (1 << 30) && x_small <= (1 << 30);
  return c;
}
template <class Op>
cudaError_t run_square(const gemm::MapsOf<Op>& maps, typename Op::Params& p, int64_t B, const Cover& c, cudaStream_t stream) {
  p.whole = c.whole;
  p.per = c.per;
  p.loop.n_tiles = (int)(B * c.per);
  p.loop.tri = c.tri;
  return c.few ? gemm::launch<Op, true>(maps, p, stream) : gemm::launch<Op, false>(maps, p, stream);
}
template <class Op>
cudaError_t run_apply(const gemm::MapsOf<Op>& maps, typename Op::Params& p, int64_t B, const Cover& c, cudaStream_t stream) {
  const int tm = c.x_few ? 128 : 256;
  p.n_mt = (int)((p.m + tm - 1) / tm);
  p.n_nt = (int)((p.n + tm - 1) / tm);
  p.per = p.n_mt * p.n_nt;
  p.loop.n_tiles = (int)(B * p.per);
  p.loop.tri = c.tri;
  return c.x_few ? gemm::launch<Op, true>(maps, p, stream) : gemm::launch<Op, false>(maps, p, stream);
}

// The CTAs of a matrix's cluster, or 0 where the products are launches of their own.  The SMs hold
// 76 clusters of 2 at a time, 46, 36, 28, 23, 15 and 15 of 3 to 8, and a round of them takes as long
// as one matrix, where launches fill the SMs evenly.  The limits are two such rounds, or one where seven
// or eight CTAs share a matrix of up to 64, whose launches are shorter.  Replayed, us, one kernel and
// launches: 760 of 128 x 256 555 and 810; 90 of 128 x 384 137 and 201, 96 of 64 x 384 175 and 142; 68 of
// 128 x 512 135 and 176, 74 187 and 178; 68 of 64 x 512 131 and 135, 76 185 and 137; 44 of 128 x 768 155 and
// 211, 48 214 and 211; 24 of 128 x 1024 162 and 183, 33 231 and 184; 14 of 64 x 1024 85 and 130, 16 150 and
// 131.  (By the SMs, not by asking for the clusters that fit: that differs between cards, and with it
// the bits of a call.  The limits lose where a third round still pays: 60 of 128 x 768 225 and 260.)
int resident_cluster(int64_t B, int64_t side, int64_t longer) {
  const int64_t c = (longer + 127) / 128, sms = sm_count();
  if (side > 128 || c > RES_MOST) return 0;
  const int64_t most = c <= 6 ? sms * 9 / 5 : (side > 64 ? sms * 11 / 8 : sms * 2 / 3);
  return c <= 2 || B * c <= most ? (int)c : 0;
}

template <bool TALL>
cudaError_t launch_resident(const OrthArgs& a, const Buffer& x, int cluster, cudaStream_t stream) {
  static std::atomic<int> done[64];
  const int ds = device_slot();
  if (ds < 0 || !done[ds].load()) {
    const cudaError_t e = cudaFuncSetAttribute(orth_resident_kernel<TALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RES_SMEM);
    if (e != cudaSuccess) return e;
    if (ds >= 0) done[ds].store(1);
  }
  Halves maps;
  if (!stack_map(&maps.value, x.value, x, a.B, a.m, a.n, 128) || !stack_map(&maps.rest, x.rest, x, a.B, a.m, a.n, 128))
    return cudaErrorInvalidValue;
  Resident p{};
  p.m = a.m;
  p.n = a.n;
  p.steps = a.steps;
  p.cluster = cluster;
  p.a = a.coef[0];
  p.b = a.coef[1];
  p.c = a.coef[2];
  p.out = static_cast<uint16_t*>(a.out);
  p.ldo = a.ldo;
  p.out_matrix = a.out_matrix;
  p.out_vec = out_vec(a);
  p.status = a.status;
  p.limit = debug_wait_limit();
  p.withhold = (int)debug_take_withheld();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * cluster));
  cfg.blockDim = dim3(RT);
  cfg.dynamicSmemBytes = RES_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, orth_resident_kernel<TALL>, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool TALL>
cudaError_t iterate(const OrthArgs& a, const Layout& l, cudaStream_t stream) {
  char* ws = static_cast<char*>(a.workspace);
  auto take = [&](size_t bytes) {
    char* p = ws;
    ws += bytes;
    return reinterpret_cast<uint16_t*>(p);
  };
  Buffer x[2], gram{}, poly{};
  for (Buffer& b : x) b = Buffer{take(l.x), take(l.x), l.x_ld, l.x_ld * a.m};
  for (Buffer* b : {&gram, &poly}) *b = Buffer{take(l.p), l.precise ? take(l.p) : nullptr, l.p_ld, l.p_ld * l.side};
  Start s{};
  s.g = a.g;
  s.ldg = a.ldg;
  s.g_matrix = a.g_matrix;
  s.m = a.m;
  s.n = a.n;
  const int64_t group = a.dtype ? 4 : 8;
  s.vec = reinterpret_cast<uintptr_t>(a.g) % 16 == 0 && (a.m == 1 || a.ldg % group == 0) && (a.B == 1 || a.g_matrix % group == 0);
  s.eps = a.eps;
  s.parts = l.parts;
  s.sums = reinterpret_cast<Squares*>(ws);
  s.x = x[0];
  s.status = a.status;
  const dim3 sums((unsigned)l.parts, (unsigned)a.B);
  if (a.dtype == 0) orth_norm_kernel<0><<<sums, OT, 0, stream>>>(s);
  else orth_norm_kernel<1><<<sums, OT, 0, stream>>>(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t ctas = (a.m * ((a.n + 7) / 8) + OT - 1) / OT;   // a group of 8 a thread, up to 8 CTAs an SM
  int64_t grid = ((int64_t)sm_count() * 8 + a.B - 1) / a.B;
  grid = grid > ctas ? ctas : grid;
  e = launch_after(a.dtype == 0 ? orth_start_kernel<0> : orth_start_kernel<1>, dim3((unsigned)grid, (unsigned)a.B), dim3(OT), 0, stream, s);
  if (e != cudaSuccess) return e;

  const int64_t longer = a.m < a.n ? a.n : a.m;
  if (const int cluster = resident_cluster(a.B, l.side, longer)) return launch_resident<TALL>(a, x[0], cluster, stream);

  using Gram = SquareOp<TALL, false>;
  using Poly = SquareOp<false, true>;
  using Apply = ApplyOp<TALL>;
  // maps of both halves of X, A and P in boxes of 128 rows, and of 64 (their columns' index contiguous)
  CUtensorMap of_x[2][2][2], of_gram[2][2], of_poly[2][2];
  bool ok = true;
  for (int h = 0; h < 2; ++h) {
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j)
        ok = ok && stack_map(&of_x[i][j][h], h ? x[i].rest : x[i].value, x[i], a.B, a.m, a.n, j ? 64 : 128);
    const bool two = h && l.precise;   // else never taken
    for (int j = 0; j < 2; ++j)
      ok = ok && stack_map(&of_gram[j][h], two ? gram.rest : gram.value, gram, a.B, l.side, l.side, j ? 64 : 128) &&
           stack_map(&of_poly[j][h], two ? poly.rest : poly.value, poly, a.B, l.side, l.side, j ? 64 : 128);
  }
  const Cover cov = cover(a.B, a.m, a.n);
  ok = ok && cov.fits;
  if (!ok) return cudaErrorInvalidValue;
  auto set = [](CUtensorMap (&to)[2], const CUtensorMap (&from)[2]) {
    to[0] = from[0];
    to[1] = from[1];
  };
  const int terms = l.precise ? 3 : 1, side_steps = (int)((l.side + gemm::BK - 1) / gemm::BK);
  for (int k = 0; k < a.steps; ++k) {
    const int i = k & 1;
    gemm::TriMaps maps{};
    set(maps.a, of_x[i][TALL]);
    set(maps.b, of_x[i][TALL]);
    typename Gram::Params g{};
    g.loop.status = a.status;
    g.loop.part_steps = (int)((longer + gemm::BK - 1) / gemm::BK);
    g.loop.k_steps = terms * g.loop.part_steps;
    g.side = (int)l.side;
    g.scale = kDown;
    g.out = gram;
    if ((e = run_square<Gram>(maps, g, a.B, cov, stream)) != cudaSuccess) return e;
    set(maps.a, of_gram[0]);
    set(maps.b, of_gram[0]);
    set(maps.ta, of_gram[1]);
    set(maps.tb, of_gram[1]);
    typename Poly::Params q{};
    q.loop.status = a.status;
    q.loop.part_steps = side_steps;
    q.loop.k_steps = terms * side_steps;
    q.side = (int)l.side;
    q.scale = a.coef[2] * kDown;
    q.b = a.coef[1];
    q.a = gram;
    q.out = poly;
    if ((e = run_square<Poly>(maps, q, a.B, cov, stream)) != cudaSuccess) return e;
    if (TALL) {
      set(maps.a, of_x[i][0]);
      set(maps.b, of_poly[0]);
      set(maps.tb, of_poly[1]);
    } else {
      set(maps.a, of_poly[0]);
      set(maps.ta, of_poly[1]);
      set(maps.b, of_x[i][1]);
    }
    typename Apply::Params p{};
    p.loop.status = a.status;
    p.loop.part_steps = side_steps;
    p.loop.k_steps = terms * side_steps;
    p.m = a.m;
    p.n = a.n;
    p.a = a.coef[0];
    p.x = x[i];
    p.to = x[i ^ 1];
    if (k == a.steps - 1) {
      p.out = static_cast<uint16_t*>(a.out);
      p.ldo = a.ldo;
      p.out_matrix = a.out_matrix;
      p.out_vec = out_vec(a);
    }
    if ((e = run_apply<Apply>(maps, p, a.B, cov, stream)) != cudaSuccess) return e;
  }
  return e;
}

}  // namespace

size_t orth_workspace_bytes(int64_t B, int64_t m, int64_t n) { return layout(B, m, n).total(); }

cudaError_t launch_orthogonalise(const OrthArgs& a, cudaStream_t stream) {
  const Layout l = layout(a.B, a.m, a.n);
  return a.m > a.n ? iterate<true>(a, l, stream) : iterate<false>(a, l, stream);
}

}  // namespace rlk
