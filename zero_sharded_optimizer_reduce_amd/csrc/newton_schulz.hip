// gfx950 kernels of zero_newton_schulz: X = G/||G||_F, then per step
//   A = X X^T,  C = a I + b A + c A A,  X = C X.
//
// Shapes.  k = the smaller side, l = the larger: X is kept k x l (a tall input
// is turned on the way in and out), so A and C are k x k.  Products of the k x k
// matrices and the Gram product have both operands' summed index contiguous in
// memory, D = P Q^T: A = X X^T, and A A = A A^T since A is symmetric; C X takes X's
// columns with transposing LDS reads, so one copy of X is all that is written
// (a second, transposed one cost 6% of 32 x 512 x 1024, 2% of 2 x 14336 x 4096).
// Products of commuting polynomials of one symmetric matrix are symmetric: only
// tiles on and below the diagonal are computed, and written twice.
//
// Blocks of steps.  With C_0, C_1 polynomials of A, two steps are
//   A' = C_0 A C_0,  C_1 = a I + b A' + c A' A',  X'' = (C_1 C_0) X:
// a Gram product and a product with X (3 k k l) less and three k x k products (3 k k k,
// 4 where the last of them is not symmetric) more than step by step.
//
// Rounding X after the first two steps costs most: the later steps raise what
// the rounding adds in the directions of small singular values by up to a^3 =
// 41.  The roundings E are kept (FP16, scaled) and the next product adds their
// image C E, taken as (trace C / k) E: exact where C is nearly a multiple of I,
// as it is on the small singular values that matter here.
//
// Numbers.  Operands are FP16 (11 significant bits), held times a power of
// two that leaves room for singular values up to ZERO_NS_MAX_SIGMA and gains
// up to ZERO_NS_MAX_GAIN and keeps even 2^-25 of a typical entry a normal
// number; products accumulate in FP32.  Rounding X, A and C to 11 bits moves
// the result by about 1.2e-3 of its norm; the final rounding to BF16 alone is
// 1.7e-3.  BF16 operands would move it by 1e-2.
// An FP32 input rounded to FP16 would be noise in every direction, which the steps
// raise by up to 3.44^5 = 484 where singular values are small: matrices of rank one
// came out 1.4e-1 off.  The first product with X sums over the remainder too (6.9e-3;
// 3 of 777 x 1301 197 us instead of 191, 4096 x 4096 1486 instead of 1360); the Gram
// product need not: it loses no more than by its own rounding.
// Steps that raise roundings further (see check_ns_coefs) run one by one with X, A
// and C as pairs of FP16 values, 22 bits, in three sums per product.
#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kernels.h"

namespace zero {
namespace {

typedef _Float16 half_t;
typedef half_t h8 __attribute__((ext_vector_type(8)));
typedef half_t h4 __attribute__((ext_vector_type(4)));
typedef float f16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kPad = 64;                 // the summed index is padded to this with zeros
constexpr float kScaleX = 16384.0f;      // |X| <= 2: 32768 < 65504
constexpr float kScaleA = 8192.0f;       // |A| <= 4
constexpr float kScaleC = 2048.0f;       // |C| <= 16
constexpr float kScaleQ = 128.0f;        // |C C| <= 256
constexpr float kScaleE = 2048.0f;       // of X's rounding errors, on top of X's scale

__host__ __device__ inline int64_t pad_up(int64_t n) { return (n + kPad - 1) / kPad * kPad; }

__device__ __forceinline__ uint16_t bf16_rne(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

// ------------------------------------------------------------------ norm
constexpr int kNormThreads = 256;
constexpr int kNormParts = kNormThreads;  // partial sums per matrix, at most

struct NsInput {
  const void* in;
  int64_t row, mat;   // strides in elements
  int rows, cols;
  int f32;
  int vec;            // 16-byte loads are aligned
};

typedef float f8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

// Elements [c, c + 8) of a row that starts at element `row`; zeros past the end.
__device__ __forceinline__ f8 load8(const NsInput& g, int64_t row, int c) {
  f8 v = {};
  if (g.f32) {
    const float* p = static_cast<const float*>(g.in) + row + c;
    if (g.vec && c + 8 <= g.cols) {
      const f4 lo = reinterpret_cast<const f4*>(p)[0], hi = reinterpret_cast<const f4*>(p)[1];
      v = f8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < g.cols) v[q] = p[q];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(g.in) + row + c;
    if (g.vec && c + 8 <= g.cols) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < g.cols) v[q] = __uint_as_float(static_cast<uint32_t>(p[q]) << 16);
    }
  }
  return v;
}

__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kNormThreads / 64];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < kNormThreads / 64; ++i) t += part[i];
  return t;
}

// Partial sums of squares, in FP64 and in an order fixed by the shape: wave w of
// a matrix takes its rows w, w + waves, ..., a lane 8 elements in every 512.
__global__ __launch_bounds__(kNormThreads) void ns_norm_kernel(NsInput g, double* partials) {
  const int64_t base = static_cast<int64_t>(blockIdx.y) * g.mat;
  double acc = 0.0;
  for (int r = blockIdx.x * (kNormThreads / 64) + (threadIdx.x >> 6); r < g.rows; r += gridDim.x * (kNormThreads / 64))
    for (int c = (threadIdx.x & 63) * 8; c < g.cols; c += 512) {
      const f8 v = load8(g, base + static_cast<int64_t>(r) * g.row, c);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc += static_cast<double>(v[q]) * static_cast<double>(v[q]);
    }
  const double t = block_sum(acc);
  if (threadIdx.x == 0) partials[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = t;
}

// kScaleX / norm = f * 2^e with f in [1/2, 1) from the sum of squares.  A zero
// matrix stays zero; `add` makes everything NaN when the sum is not finite.
struct NsScale {
  float f, add;
  int e;
};

__device__ __forceinline__ NsScale scale_of(double sum) {
  NsScale s = {1.0f, 0.0f, 0};
  if (sum > 0.0 && sum < __builtin_huge_val())
    s.f = static_cast<float>(frexp(static_cast<double>(kScaleX) / sqrt(sum), &s.e));
  else if (sum != 0.0)
    s.add = __builtin_nanf("");
  return s;
}

// ------------------------------------------------------------------ X
// X * kScaleX = f * (G * 2^e): the stored G * 2^e is exact for BF16 inputs (8
// bits in 11), and of FP32 inputs the remainder is stored too (22 bits); the factor
// f joins the products' scales, so that nothing is lost before the first product.
struct NsX {
  half_t* x;         // k x l, pitch pad(l), pad(k) rows: those past k are zeros, here
  half_t* next;      // and in the X that the steps write next
  int64_t mat;
  int tall;          // X is G^T
  const double* partials;
  int parts;
  float* f;          // per matrix, for the products
  half_t* low;       // what rounding G * 2^e left (nothing of BF16 values), or NULL
  half_t* next_low;  // the next X's low half, or NULL
};

constexpr int kTurn = 64;

// One 64 x 64 tile; the padding is written as zeros.  Every workgroup adds the
// partial sums up itself, while its tile is on its way.
template <bool LOW>
__global__ __launch_bounds__(kNormThreads) void ns_prepare_kernel(NsInput g, NsX x) {
  // 33 words a row: the eight rows a lane group gathers lie in different banks
  __shared__ uint32_t tile[kTurn][kTurn / 2 + 1];
  const int mat = blockIdx.z;
  const int r0 = blockIdx.y * kTurn, c0 = blockIdx.x * kTurn;
  const int ld = static_cast<int>(pad_up(x.tall ? g.rows : g.cols));
  half_t* out = x.x + mat * x.mat;
  half_t* next = x.next + mat * x.mat;
  half_t* low = LOW ? x.low + mat * x.mat : nullptr;
  half_t* next_low = LOW && x.next_low ? x.next_low + mat * x.mat : nullptr;
  const int64_t base = static_cast<int64_t>(mat) * g.mat;
  const int line = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
  constexpr int kLines = kTurn / (kNormThreads / 8);
  f8 v[kLines];
#pragma unroll
  for (int n = 0; n < kLines; ++n) {
    const int r = r0 + line + n * (kNormThreads / 8);
    v[n] = f8{};
    if (r < g.rows) v[n] = load8(g, base + static_cast<int64_t>(r) * g.row, c0 + c);
  }
  const NsScale s = scale_of(block_sum(
      static_cast<int>(threadIdx.x) < x.parts ? x.partials[static_cast<int64_t>(mat) * x.parts + threadIdx.x] : 0.0));
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) x.f[mat] = s.f;
  h8 hi[kLines], lo[kLines];
#pragma unroll
  for (int n = 0; n < kLines; ++n)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool in = r0 + line + n * (kNormThreads / 8) < g.rows && c0 + c + q < g.cols;
      const float w = in ? ldexpf(v[n][q], s.e) + s.add : 0.0f;
      hi[n][q] = static_cast<half_t>(w);
      lo[n][q] = static_cast<half_t>(w - static_cast<float>(hi[n][q]));
    }
#pragma unroll
  for (int half = 0; half < (LOW ? 2 : 1); ++half) {
    half_t* to = half ? low : out;
    half_t* zeros = half ? next_low : next;
#pragma unroll
    for (int n = 0; n < kLines; ++n) {
      const int i = line + n * (kNormThreads / 8), r = r0 + i;
      const h8 h = half ? lo[n] : hi[n];
      if (!x.tall) {
        *reinterpret_cast<h8*>(to + static_cast<int64_t>(r) * ld + c0 + c) = h;
        if (zeros && r >= g.rows) *reinterpret_cast<h8*>(zeros + static_cast<int64_t>(r) * ld + c0 + c) = h;
      }
      const u32x4 w = __builtin_bit_cast(u32x4, h);
#pragma unroll
      for (int q = 0; q < 4; ++q) tile[i][c / 2 + q] = w[q];
    }
    if (!x.tall) continue;
    __syncthreads();
#pragma unroll
    for (int i = line; i < kTurn; i += kNormThreads / 8) {
      u32x4 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a = tile[c + 2 * q][i >> 1], b = tile[c + 2 * q + 1][i >> 1];
        w[q] = i & 1 ? (a >> 16) | (b & 0xFFFF0000u) : (a & 0xFFFFu) | (b << 16);
      }
      const int64_t at = static_cast<int64_t>(c0 + i) * ld + r0 + c;
      *reinterpret_cast<u32x4*>(to + at) = w;
      if (zeros && c0 + i >= g.cols) *reinterpret_cast<u32x4*>(zeros + at) = w;
    }
    if (LOW && !half) __syncthreads();   // the tile is read
  }
}

// ------------------------------------------------------------------ products
// D = alpha' P Q^T with P m x kk, Q n x kk (pitches p_ld, q_ld; kk a multiple of
// kPad, the padding zero).
// kSym: a symmetric result, its tiles on and below the diagonal.  kRide: P = Q, and
// the tiles on the diagonal ride: P's rows of diagonal tile i are those of tile
// (i, i - 1), whose workgroup computes both.
// kTimesX: Q^T is X itself, rows in order of the summed index.
// SUMS: 2: Q is a pair of FP16 matrices, high + low, and the sum runs over P with the
// high half, then with the low one.  3: P and the result are pairs too: high high +
// high low + low high; the result's halves are written one after the other.
enum Shape { kFull, kSym, kRide, kTimesX };
enum Epilogue { kPlain, kPoly, kCarryOut, kCarryIn, kOut };
struct Product {
  const half_t* p;
  const half_t* q;
  int64_t p_mat, q_mat;
  int p_ld, q_ld;
  int m, n, kk;
  int tiles_n, tiles;       // per matrix
  half_t* d;                // FP16 result, columns n up to d_ld written as zeros
  int64_t d_mat;
  int d_ld;
  const half_t* add;        // polynomial: beta * add + diag * I joins (symmetric, pitch d_ld)
  float alpha, beta, diag;
  const float* f;           // per-matrix factor of alpha, or NULL
  int f_pow;
  uint16_t* out;            // BF16 result instead of d
  int64_t out_row, out_mat;
  int out_vec;              // 16-byte stores are aligned
  int out_turned;           // as its transpose
  half_t* carry_out;        // the FP16 roundings of d, in the lanes' own order, or NULL
  const half_t* carry_in;   // those of the X this product reads, or NULL
  int64_t carry_mat;
  int64_t p_lo, q_lo, d_lo, add_lo;   // elements from a matrix to its low half
};

constexpr int kTile = 256;    // the largest tile
constexpr int kBk = 64;      // summed index per stage: rows of 128 bytes in LDS

// Rows [row0, row0 + R) of an operand, columns [k0, k0 + 64), into LDS as R rows
// of 128 bytes; the 16-byte piece c of row r lies at piece c ^ ((r >> 1) & 7),
// so that the pieces c of any 16 consecutive rows fall into different banks (64
// banks of 4 bytes: two rows fill them once).  Each wave moves
// 1 KiB (8 rows) per instruction, straight to LDS; a row's 128 bytes are one
// cache line (rows of 64 bytes ran at 55 instead of 95 bytes/ns per CU).  Rows
// past the matrix's end hold something else of the workspace, which ends
// kTile rows after the last matrix; their results are dropped.
// LOW: the sum that takes the operand's low half.
template <int R, int NW, int SUMS, int LOW>
struct Stager {
  static constexpr int kN = R / 8 / NW;
  static_assert(kN * 8 * NW == R && kN % 2 == 0, "every wave moves the same number of pieces, an even one");
  __amdgpu_buffer_rsrc_t rsrc, none;   // none: no bytes in range, a load through it reads nothing
  half_t* base;
  int64_t low;
  int voff[2], step, wave, end;        // voff: even and odd groups of 8 rows
  __device__ __forceinline__ Stager(const half_t* mat, int ld, int row0, int kk, int wave_, int lane, int64_t low_)
      : base(const_cast<half_t*>(mat + static_cast<int64_t>(row0) * ld)), low(low_), wave(wave_), end(kk) {
    rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, R * ld * 2, 0x00020000);
    none = __builtin_amdgcn_make_buffer_rsrc(base, 0, 0, 0x00020000);
    const int r = wave * kN * 8 + (lane >> 3);
    voff[0] = r * ld * 2 + ((lane & 7) ^ (lane >> 4)) * 16;
    voff[1] = voff[0] ^ 64;   // ld is a multiple of 64
    step = 8 * ld * 2;
  }
  // A stage past the end is loaded too, so that the loads on their way can be
  // counted, but from nowhere.
  __device__ __forceinline__ void one(half_t* lds, int k0, int i) const {
#ifdef __HIP_DEVICE_COMPILE__   // the builtin is unknown to the host pass
    const bool live = k0 < SUMS * end;
    const int sum = SUMS == 1 || k0 < end ? 0 : SUMS == 2 || k0 < 2 * end ? 1 : 2;
    k0 -= sum * end;
    // (a choice between kept descriptors would put them into memory)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        LOW >= SUMS ? (live ? rsrc : none)
                    : __builtin_amdgcn_make_buffer_rsrc(base + (sum == LOW ? low : 0), 0, live ? R / 8 * step : 0, 0x00020000),
        (lds_void*)(lds + (wave * kN + i) * 8 * kBk), 16, voff[i & 1], live ? k0 * 2 + i * step : 0, 0, 0);
#endif
  }
  __device__ __forceinline__ void all(half_t* lds, int k0) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) one(lds, k0, i);
  }
};

// Of X, rows [k0, k0 + 64) and columns [col0, col0 + C): 64 rows of 2 C bytes, from
// which transposing reads take the columns.  Those read 64 bytes of four rows
// together: the 64-byte piece c of row r lies at piece c ^ (r & 3) (C = 64, where
// two rows fill the banks: c ^ ((r >> 1) & 1)).  Columns past the end hold the
// next row; their results are dropped.
template <int C, int NW, int SUMS>
struct ColumnStager {
  static constexpr int kRows = 512 / C, kN = 64 / kRows / NW;   // rows of one instruction, instructions of a wave
  static_assert(kN * kRows * NW == 64 && (C != 256 || kN % 2 == 0), "every wave moves the same number of pieces");
  half_t* base;
  int64_t lo;
  int voff[2], ld, wave, end;   // voff: even and odd instructions
  __device__ __forceinline__ ColumnStager(const half_t* mat, int ld_, int col0, int kk, int wave_, int lane, int64_t lo_)
      : base(const_cast<half_t*>(mat + col0)), lo(lo_), ld(ld_), wave(wave_), end(kk) {
    const int row = lane / (64 / kRows), piece = lane % (64 / kRows);
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const int r = row + (C == 256 ? 2 * odd : 0), s = C == 64 ? (r >> 1) & 1 : r & 3;
      voff[odd] = (wave * kN * kRows + row) * ld * 2 + (((piece >> 2) ^ s) << 6) + (piece & 3) * 16;
    }
  }
  __device__ __forceinline__ void one(half_t* lds, int k0, int i) const {
#ifdef __HIP_DEVICE_COMPILE__
    const bool live = k0 < SUMS * end;
    const int sum = SUMS == 1 || k0 < end ? 0 : SUMS == 2 || k0 < 2 * end ? 1 : 2;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(base + (sum == 1 ? lo : 0) + static_cast<int64_t>(k0 - sum * end) * ld, 0,
                                          live ? kBk * ld * 2 : 0, 0x00020000),
        (lds_void*)(lds + (wave * kN + i) * 512), 16, voff[i & 1], live ? i * kRows * ld * 2 : 0, 0, 0);
#endif
  }
  __device__ __forceinline__ void all(half_t* lds, int k0) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) one(lds, k0, i);
  }
};
// Byte offset in a slot of what the lane points a transposing read at: row 8 *
// (lane >> 5) + ((lane >> 2) & 3), columns first + 16 * ((lane >> 4) & 1) + 4 * (lane & 3).
template <int C>
__device__ __forceinline__ int lane_at_column(int first, int lane) {
  const int s = C == 64 ? (lane >> 3) & 1 : (lane >> 2) & 3;
  return ((lane >> 5) * 8 + ((lane >> 2) & 3)) * C * 2 + (((first >> 5) ^ s) << 6) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
}

// 4 values down a column, twice: the transposing LDS read hands lane j of 16 the
// component j % 4 of the lanes j / 4 + 4 q, so each lane points at four columns of
// one row and lane j gets column j of four rows.
__device__ __forceinline__ u32x4 transpose8(const void* at, const void* at4) {
  u32x4 v = {};
#ifdef __HIP_DEVICE_COMPILE__   // the builtin is unknown to the host pass
  typedef short s4 __attribute__((ext_vector_type(4)));
  typedef short s8 __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s4 lds_s4;
  const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at);
  const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at4);
  v = __builtin_bit_cast(u32x4, s8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
#endif
  return v;
}
// A wave's operands for half a stage: two 16-wide pieces of the summed index.
// SECOND: the rows of P at the wave's columns too, for P P^T.  C: Q is C columns of
// X (see ColumnStager), else 0.
template <int TM, int TN, bool SECOND, int C>
struct Frags {
  static constexpr int kSets = TM + TN + (SECOND ? TN : 0), kReads = 2 * kSets;
  h8 a[2][TM], b[2][TN], c[2][TN];
  // Read number n of kReads; at_p, at_q, at_c: the lane's byte offsets in a slot
  // (see lane_at, lane_at_column); half 0 or 1.
  __device__ __forceinline__ void one(const half_t* p, const half_t* q, int at_p, int at_q, int at_c, int half, int n) {
    const int u = n / kSets, i = n - u * kSets, flip = half * 64 + u * 32;
    auto read = [&](const half_t* m, int at, int block) {
      return *reinterpret_cast<const h8*>(reinterpret_cast<const char*>(m) + (at ^ flip) + block * 32 * kBk * 2);
    };
    if (i < TM) {
      a[u][i] = read(p, at_p, i);
    } else if (i < TM + TN) {
      if constexpr (C > 0) {
        const char* at = reinterpret_cast<const char*>(q) + (at_q ^ ((i - TM) << 6)) + (half * 32 + u * 16) * C * 2;
        b[u][i - TM] = __builtin_bit_cast(h8, transpose8(at, at + 4 * C * 2));
      } else {
        b[u][i - TM] = read(q, at_q, i - TM);
      }
    } else {
      c[u][i - TM - TN] = read(p, at_c, i - TM - TN);
    }
  }
};

// Byte offset in a slot of the lane's first fragment piece: row first + (lane &
// 31), piece lane >> 5, moved as Stager moves it.  Pieces 2, 4 and 6 further on
// are at the offset with bits 5 and 6 flipped.
__device__ __forceinline__ int lane_at(int first, int lane) {
  return (first + (lane & 31)) * kBk * 2 + (((lane >> 5) ^ ((lane >> 1) & 7)) << 4);
}

// s_waitcnt operands: vmcnt(n) alone, and all LDS operations with it.
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
constexpr int wait_vm_lds(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// All waves' LDS traffic up to here before any of theirs after it.  The empty
// asm keeps the compiler from moving memory operations across the barrier.
__device__ __forceinline__ void wave_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Workgroups go to the 8 XCDs in turn, each with its own L2: workgroup id's
// place in an order where an XCD's workgroups are neighbours.
__device__ __forceinline__ int xcd_order(int id, int n) {
  const int each = n >> 3, more = n & 7, xcd = id & 7;
  return xcd * each + (xcd < more ? xcd : more) + (id >> 3);
}

// 8 values down a column: the lane gets rows row + 8 * (lane >> 4) + 0..7 of column
// col + (lane & 15).
__device__ __forceinline__ u32x4 column_piece(const uint16_t* m, int pitch, int row, int col, int lane) {
  const uint16_t* at = m + (row + (lane >> 4) * 8 + ((lane >> 2) & 3)) * pitch + col + (lane & 3) * 4;
  return transpose8(at, at + 4 * pitch);
}

// The first n of 8 values, the others zero.
__device__ __forceinline__ u32x4 first(u32x4 v, int n) {
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = 2 * q + 1 < n ? v[q] : 2 * q < n ? v[q] & 0xFFFFu : 0u;
  return v;
}

// The first n of 8 values to memory, which is 16-byte aligned if vec.
__device__ __forceinline__ void store8(uint16_t* dst, u32x4 v, int vec, int n) {
  if (vec && n >= 8) {
    *reinterpret_cast<u32x4*>(dst) = v;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) dst[q] = static_cast<uint16_t>(v[q >> 1] >> ((q & 1) * 16));
  }
}

template <int NW>
__device__ __forceinline__ float block_sum_f32(float x, float* part) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) t += part[i];
  return t;
}

// One tile BM x BN by WR x WC waves.  Measured at 4096 x 4096 x 4096: 256 wide 113 us
// alone (1220 TFLOP/s), 117 to 131 in a call; symmetric with 192 wide tiles 69 alone,
// 77 to 89 in a call: with the matrix units busy 81 and 68% of the time the clock
// falls to 1.7 - 2.0 GHz, and power bounds both.  Small products are bound by what a
// launch does in turn: 1 us until the first stage is there, 64 wide tiles' loads at
// 55 to 95 bytes/ns per CU, and the results' way out.
//
// The loop over the summed index keeps one to one and a half stages (DEEP: four)
// on their way to LDS and half a stage ahead in registers: while the matrix cores work
// on one half the wave reads the next one's fragments, and the loads are issued
// evenly between the products (a wave issues in order: loads in a row
// hold its products up while the CU takes them in, about 26 clocks each).
template <int BM, int BN, int WR, int WC, Shape SHAPE, Epilogue EPI, bool DEEP, int SUMS>
__global__ __launch_bounds__(WR * WC * 64, BM <= 128 ? 2 : 1) void ns_product_kernel(Product g) {
  constexpr int NW = WR * WC;
  constexpr int TM = BM / WR / 32, TN = BN / WC / 32;   // 32 x 32 blocks of a wave
  constexpr int kSlot = (BM > BN ? BM : BN) * kBk;
  // Five places for an operand's rows of one stage, ten for the smallest tile: its
  // stages are short, and four of them have to be on their way.  Separate arrays,
  // so that the compiler can tell a load on its way into one from a read of another.
  constexpr bool SYM = SHAPE == kSym || SHAPE == kRide;
  constexpr int kColumns = SHAPE == kTimesX ? BN : 0;
  static_assert(TN == 1 || TN == 2 || !kColumns, "a wave's 64-byte pieces are a power of two");
  __shared__ __align__(16) half_t slot0[kSlot];
  __shared__ __align__(16) half_t slot1[kSlot];
  __shared__ __align__(16) half_t slot2[kSlot];
  __shared__ __align__(16) half_t slot3[kSlot];
  __shared__ __align__(16) half_t slot4[kSlot];
  __shared__ __align__(16) half_t slot5[DEEP ? kSlot : 1];
  __shared__ __align__(16) half_t slot6[DEEP ? kSlot : 1];
  __shared__ __align__(16) half_t slot7[DEEP ? kSlot : 1];
  __shared__ __align__(16) half_t slot8[DEEP ? kSlot : 1];
  __shared__ __align__(16) half_t slot9[DEEP ? kSlot : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int id = xcd_order(blockIdx.x, gridDim.x);
  const int mat = id / g.tiles;
  const int t = id - mat * g.tiles;
  int ti, tj;
  bool rides = false;   // the tile of P P^T on the diagonal too
  if (SHAPE == kRide) {
    const int side = (g.m + BM - 1) / BM;
    ti = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > t) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    tj = t - ti * (ti + 1) / 2;
    rides = tj == ti++;
    if (ti >= side) {                               // the only one on the diagonal, or of two the first
      ti = tj = 0;
      rides = false;
    } else if (side > 2 && ti == side - 1 && tj == 0) {   // the first diagonal tile's place
      ti = 0;
      tj = side - 1;
      rides = true;
    }
  } else if (SYM) {
    ti = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > t) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    tj = t - ti * (ti + 1) / 2;
  } else {
    ti = t / g.tiles_n;
    tj = t - ti * g.tiles_n;
  }
  const int row0 = ti * BM, col0 = tj * BN;
  static_assert(SHAPE != kRide || SUMS == 1, "a riding tile takes both operands from P's rows in LDS");
  static_assert(SUMS != 3 || EPI == kPlain || EPI == kPoly || EPI == kOut, "pairs carry no roundings");
  using PStager = Stager<BM, NW, SUMS, 2>;
  const PStager sp(g.p + mat * g.p_mat, g.p_ld, row0, g.kk, wave, lane, g.p_lo);
  using QStager = std::conditional_t<SHAPE == kTimesX, ColumnStager<BN, NW, SUMS>, Stager<BN, NW, SUMS, 1>>;
  const QStager sq(g.q + mat * g.q_mat, g.q_ld, col0, g.kk, wave, lane, g.q_lo);
  const int wr = wave / WC, wc = wave - wr * WC;
  int at_p = lane_at(wr * (BM / WR), lane);
  int at_q = SHAPE == kTimesX ? lane_at_column<BN>(wc * (BN / WC), lane) : lane_at(wc * (BN / WC), lane);
  constexpr int kP = PStager::kN, kQ = QStager::kN;
  // The lane's values of block (i, j): row lane & 31 of the block, columns 8 * u +
  // 4 * (lane >> 5) + q (the products take Q's fragment first).
  float alpha = g.alpha;
  if (g.f) {
    const float f = g.f[mat];
    alpha *= g.f_pow == 2 ? f * f : f;
  }
  const int lm = lane & 31, ln = (lane >> 5) << 2;
  // Results pass through the wave's own part of LDS, kBand blocks of rows at a
  // time, so that they leave as rows of 16-byte pieces; the transpose is read
  // from there with transposing reads.  A wave's LDS operations are carried out
  // in order, so no barrier is needed.  (Piece by piece, each read waited for
  // before its store, and the diagonal's blocks mirrored in LDS first, a 128 tile's
  // results took 4.7 us where they take 3.2, in 10.7 us for 1024 x 1024 x 1024.)
  constexpr int kBand = TM % 2 == 0 ? 2 : TM;
  constexpr int kRows = kBand * 32, kCols = TN * 32, kPitch = kCols + 8;
  constexpr int kPart = kSlot / (NW / 4);
  static_assert(TM % kBand == 0, "whole bands");
  static_assert(kRows * kPitch <= kPart, "a band fits the wave's part");
  uint16_t* mine = reinterpret_cast<uint16_t*>((wave & 3) == 0 ? slot0 : (wave & 3) == 1 ? slot1 : (wave & 3) == 2 ? slot2 : slot3) +
                   (wave >> 2) * kPart;
  // A tile on the diagonal of a symmetric product: only what lies below the
  // diagonal of its 32 x 32 blocks is kept, as for the tiles.  low: the low half.
  auto write = [&](const f16 (&acc)[TM][TN], int row0, int col0, float gain, auto low) {
    constexpr bool LOW = decltype(low)::value;
    const int wrow = row0 + wr * (BM / WR), wcol = col0 + wc * (BN / WC);
    const bool diagonal = SYM && row0 == col0;
#pragma unroll
    for (int ib = 0; ib < TM; ib += kBand) {
      const int64_t carry = mat * g.carry_mat + static_cast<int64_t>(t) * (BM * BN) + threadIdx.x * 4;
      // what joins the products: all loads of the band before the first use
      h4 more[kBand][TN][4], more_lo[kBand][TN][4];
      if constexpr (EPI == kPoly || EPI == kCarryIn) {
#pragma unroll
        for (int i = 0; i < kBand; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if constexpr (EPI == kPoly) {
                const int r = wrow + (ib + i) * 32 + lm, c = wcol + j * 32 + u * 8 + ln;
                // past the edge: some other value, dropped below
                const half_t* at =
                    g.add + mat * g.d_mat + static_cast<int64_t>(r < g.m ? r : 0) * g.d_ld + (c < g.d_ld ? c : 0);
                more[i][j][u] = *reinterpret_cast<const h4*>(at);
                if constexpr (SUMS == 3) more_lo[i][j][u] = *reinterpret_cast<const h4*>(at + g.add_lo);
              } else {
                more[i][j][u] =
                    *reinterpret_cast<const h4*>(g.carry_in + carry + (((ib + i) * TN + j) * 4 + u) * (NW * 256));
              }
            }
      }
#pragma unroll
      for (int i = 0; i < kBand; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = acc[ib + i][j][u * 4 + q] * alpha;
            if constexpr (EPI == kPoly) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float a = static_cast<float>(more[i][j][u][q]);
                if constexpr (SUMS == 3) a += static_cast<float>(more_lo[i][j][u][q]);
                v[q] += g.beta * a;
              }
              if (i == j && diagonal && wr == wc) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  if (lm == u * 8 + ln + q) v[q] += g.diag;
              }
            }
            if constexpr (EPI == kCarryIn) {
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] += gain * static_cast<float>(more[i][j][u][q]);
            }
            u16x4 o;
            if constexpr (EPI == kOut) {
#pragma unroll
              for (int q = 0; q < 4; ++q) o[q] = bf16_rne(v[q]);
            } else {
              h4 h;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                // Rounded to FP32 here: folded into the rounding to FP16 in one of the
                // two passes, the halves would now and then be those of two values.
                if constexpr (SUMS == 3) asm volatile("" : "+v"(v[q]));
                h[q] = static_cast<half_t>(v[q]);
                if constexpr (LOW) h[q] = static_cast<half_t>(v[q] - static_cast<float>(h[q]));
              }
              o = __builtin_bit_cast(u16x4, h);
              if constexpr (EPI == kCarryOut) {
                h4 w;
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = static_cast<half_t>((v[q] - static_cast<float>(h[q])) * kScaleE);
                *reinterpret_cast<h4*>(g.carry_out + carry + (((ib + i) * TN + j) * 4 + u) * (NW * 256)) = w;
              }
            }
            *reinterpret_cast<u16x4*>(mine + (i * 32 + lm) * kPitch + j * 32 + u * 8 + ln) = o;
          }
      static_assert(!SYM || (kBand == TM && TM == TN && WR == WC), "the diagonal's blocks are (i, i)");
      // Out, kStep pieces at a time: all reads of LDS before the first store.
      constexpr int kPieces = kRows * kCols / 512, kStep = kPieces % 8 == 0 ? 8 : kPieces % 6 == 0 ? 6 : kPieces;
      const int brow = wrow + ib * 32;
      if constexpr (EPI == kOut) {
        if (g.out_turned) {
          uint16_t* out = g.out + mat * g.out_mat + static_cast<int64_t>(wcol) * g.out_row + brow;
#pragma unroll 1
          for (int k0 = 0; k0 < kPieces; k0 += kStep) {
            u32x4 piece[kStep];
#pragma unroll
            for (int k = 0; k < kStep; ++k)
              piece[k] = column_piece(mine, kPitch, (k0 + k) % kBand * 32, (k0 + k) / kBand * 16, lane);
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
              const int c = (k0 + k) / kBand * 16 + (lane & 15), r = (k0 + k) % kBand * 32 + (lane >> 4) * 8;
              if (wcol + c < g.n) store8(out + c * g.out_row + r, piece[k], g.out_vec, g.m - brow - r);
            }
          }
          continue;
        }
        uint16_t* out = g.out + mat * g.out_mat + static_cast<int64_t>(brow) * g.out_row + wcol;
#pragma unroll 1
        for (int k0 = 0; k0 < kPieces; k0 += kStep) {
          u32x4 piece[kStep];
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            const int at = (k0 + k) * 64 + lane, r = at / (kCols / 8), c = (at - r * (kCols / 8)) * 8;
            piece[k] = *reinterpret_cast<const u32x4*>(mine + r * kPitch + c);
          }
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            const int at = (k0 + k) * 64 + lane, r = at / (kCols / 8), c = (at - r * (kCols / 8)) * 8;
            if (brow + r < g.m) store8(out + r * g.out_row + c, piece[k], g.out_vec, g.n - wcol - c);
          }
        }
      } else {
        half_t* d = g.d + (LOW ? g.d_lo : 0) + mat * g.d_mat + static_cast<int64_t>(brow) * g.d_ld + wcol;
#pragma unroll 1
        for (int k0 = 0; k0 < kPieces; k0 += kStep) {
          u32x4 piece[kStep];
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            const int at = (k0 + k) * 64 + lane, r = at / (kCols / 8), c = (at - r * (kCols / 8)) * 8;
            piece[k] = *reinterpret_cast<const u32x4*>(mine + r * kPitch + c);
          }
#pragma unroll
          for (int k = 0; k < kStep; ++k) {
            const int at = (k0 + k) * 64 + lane, r = at / (kCols / 8), c = (at - r * (kCols / 8)) * 8;
            if (wcol + c + 8 > g.n) piece[k] = first(piece[k], g.n - wcol - c);
            if (brow + r < g.m && wcol + c < g.d_ld && !(diagonal && (wcol + c) >> 5 >= (brow + r) >> 5))
              *reinterpret_cast<u32x4*>(d + r * g.d_ld + c) = piece[k];
          }
        }
        if constexpr (SYM) {   // its transpose
          half_t* dt = g.d + (LOW ? g.d_lo : 0) + mat * g.d_mat + static_cast<int64_t>(wcol) * g.d_ld + brow;
#pragma unroll 1
          for (int k0 = 0; k0 < kPieces; k0 += kStep) {
            // 16 columns, 8 rows of each 8 * (lane >> 4) rows on
            u32x4 piece[kStep];
#pragma unroll
            for (int k = 0; k < kStep; ++k)
              piece[k] = column_piece(mine, kPitch, (k0 + k) % kBand * 32, (k0 + k) / kBand * 16, lane);
            if (diagonal && wr == wc) {   // in a block on the diagonal the upper half comes from the lower
#pragma unroll
              for (int k = 0; k < kStep; ++k) {
                const int c = (k0 + k) / kBand * 16 + (lane & 15), r = (k0 + k) % kBand * 32 + (lane >> 4) * 8;
                const u32x4 row = *reinterpret_cast<const u32x4*>(mine + c * kPitch + r);
                if (c >> 5 == r >> 5) {
                  const u32x4 low = first(row, c - r);
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const uint32_t keep = (r + 2 * q >= c ? 0xFFFFu : 0u) | (r + 2 * q + 1 >= c ? 0xFFFF0000u : 0u);
                    piece[k][q] = (piece[k][q] & keep) | low[q];
                  }
                }
              }
            }
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
              const int c = (k0 + k) / kBand * 16 + (lane & 15), r = (k0 + k) % kBand * 32 + (lane >> 4) * 8;
              if (brow + r + 8 > g.m) piece[k] = first(piece[k], g.m - brow - r);
              if (wcol + c < g.n && brow + r < g.d_ld && !(diagonal && (wcol + c) >> 5 > (brow + r) >> 5))
                *reinterpret_cast<u32x4*>(dt + c * g.d_ld + r) = piece[k];
            }
          }
        }
      }
    }
  };

  // The whole tile; every wave has the same loads and barriers.
  auto tile = [&](auto second) {
    constexpr bool SECOND = decltype(second)::value;
    using Set = Frags<TM, TN, SECOND, kColumns>;
    constexpr int kProducts = 2 * TM * TN, kReads = Set::kReads;
    Set f0, f1;
    f16 acc[TM][TN] = {}, acc2[TM][TN] = {};
    int at_c = at_p - wr * (BM / WR) * kBk * 2 + wc * (BN / WC) * kBk * 2;
    // Half a stage: the products of `now`, and between them, evenly, the reads of
    // `then` and the loads of one operand.  The compiler keeps the groups apart.
    auto half = [&](const auto& loads, int n_loads, const Set& now, Set& then, const half_t* p, const half_t* q,
                    int which) {
      // Addresses are formed anew: kept over the loop for every slot they would
      // not fit the registers.
      asm volatile("" : "+v"(at_p), "+v"(at_q), "+v"(at_c));
#pragma unroll
      for (int s = 0; s < n_loads; ++s) {
#pragma unroll
        for (int k = s * kProducts / n_loads; k < (s + 1) * kProducts / n_loads; ++k) {
          const int u = k / (TM * TN), i = (k - u * TM * TN) / TN, j = k % TN;
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(now.b[u][j], now.a[u][i], acc[i][j], 0, 0, 0);
          if constexpr (SECOND)
            acc2[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(now.c[u][j], now.a[u][i], acc2[i][j], 0, 0, 0);
        }
        loads(s);
#pragma unroll
        for (int k = s * kReads / n_loads; k < (s + 1) * kReads / n_loads; ++k) then.one(p, q, at_p, at_q, at_c, which, k);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int k0 = 0;
    if constexpr (DEEP) {
      // One stage: its rows in p0 and q0, the next one's in p1 and q1; Q of four
      // stages on goes where the last stage's was, P of five stages on, once every
      // wave has read this one, to p0.
      auto stage = [&](half_t* p0, half_t* q0, half_t* p1, half_t* q1, half_t* q4) {
        half([&](int s) { sq.one(q4, k0 + 4 * kBk, s); }, kQ, f0, f1, p0, q0, 1);
        __builtin_amdgcn_s_waitcnt(wait_vm_lds(3 * (kP + kQ)));   // the next stage has arrived, and this one is read
        wave_barrier();
        half([&](int s) { sp.one(p0, k0 + 5 * kBk, s); }, kP, f1, f0, p1, q1, 0);
        return (k0 += kBk) < SUMS * g.kk;
      };
      sp.all(slot0, 0);
      sq.all(slot5, 0);
      sp.all(slot1, kBk);
      sq.all(slot6, kBk);
      sp.all(slot2, 2 * kBk);
      sq.all(slot7, 2 * kBk);
      sp.all(slot3, 3 * kBk);
      sq.all(slot8, 3 * kBk);
      sp.all(slot4, 4 * kBk);
      __builtin_amdgcn_s_waitcnt(wait_vm(4 * kP + 3 * kQ));
      wave_barrier();
#pragma unroll
      for (int k = 0; k < kReads; ++k) f0.one(slot0, slot5, at_p, at_q, at_c, 0, k);
      while (stage(slot0, slot5, slot1, slot6, slot9) && stage(slot1, slot6, slot2, slot7, slot5) &&
             stage(slot2, slot7, slot3, slot8, slot6) && stage(slot3, slot8, slot4, slot9, slot7) &&
             stage(slot4, slot9, slot0, slot5, slot8)) {
      }
    } else {
      // One stage: P and Q rows in p0 and q0, the next stage's in p1 and q1; the
      // stage after that goes to p2 and, once every wave has read this one, p0.
      auto stage = [&](half_t* p0, half_t* q0, half_t* p1, half_t* q1, half_t* p2) {
        half([&](int s) { sp.one(p2, k0 + 2 * kBk, s); }, kP, f0, f1, p0, q0, 1);
        // the next stage has arrived (all but p2's loads), and this one is read
        __builtin_amdgcn_s_waitcnt(wait_vm_lds(kP));
        wave_barrier();
        half([&](int s) { sq.one(p0, k0 + 2 * kBk, s); }, kQ, f1, f0, p1, q1, 0);
        return (k0 += kBk) < SUMS * g.kk;
      };
      sp.all(slot0, 0);
      sq.all(slot1, 0);
      sp.all(slot2, kBk);
      sq.all(slot3, kBk);
      __builtin_amdgcn_s_waitcnt(wait_vm(kP + kQ));
      wave_barrier();
#pragma unroll
      for (int k = 0; k < kReads; ++k) f0.one(slot0, slot1, at_p, at_q, at_c, 0, k);
      while (stage(slot0, slot1, slot2, slot3, slot4) && stage(slot2, slot3, slot4, slot0, slot1) &&
             stage(slot4, slot0, slot1, slot2, slot3) && stage(slot1, slot2, slot3, slot4, slot0) &&
             stage(slot3, slot4, slot0, slot1, slot2)) {
      }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
    wave_barrier();   // nothing is on its way into LDS any more
    float gain = 0.0f;
    if constexpr (EPI == kCarryIn) {
      const half_t* c = g.p + mat * g.p_mat;
      float sum = 0.0f;
      for (int i = threadIdx.x; i < g.m; i += NW * 64) sum += static_cast<float>(c[static_cast<int64_t>(i) * g.p_ld + i]);
      gain = block_sum_f32<NW>(sum, reinterpret_cast<float*>(slot4)) * g.alpha / (static_cast<float>(g.m) * kScaleE);
    }
    write(acc, row0, col0, gain, std::false_type());
    if constexpr (SUMS == 3 && EPI != kOut) {
      asm volatile("" : "+v"(alpha));   // the scaled sums are formed anew: kept, they would not fit the registers
      write(acc, row0, col0, gain, std::true_type());
    }
    if constexpr (SECOND) write(acc2, row0, row0, gain, std::false_type());
  };
  const bool second = rides && wr >= wc;   // above the diagonal nothing is kept
  if constexpr (SHAPE == kRide) {
    if (second)
      tile(std::true_type());
    else
      tile(std::false_type());
  } else {
    tile(std::false_type());
  }
}

// ------------------------------------------------------------------ launches
// Workgroups per matrix.
int64_t tile_count(const Product& g, int side, Shape shape) {
  const int64_t tm = (g.m + side - 1) / side, tn = (g.n + side - 1) / side;
  if (shape == kFull || shape == kTimesX) return tm * tn;
  return shape == kSym ? tm * (tm + 1) / 2 : tm > 2 ? tm * (tm - 1) / 2 : tm;
}

template <int BM, int BN, int WR, int WC, Shape SHAPE, Epilogue EPI, bool DEEP = false, int SUMS = 1>
hipError_t product_tiles(Product g, int64_t mats, hipStream_t s) {
  g.tiles_n = (g.n + BN - 1) / BN;
  g.tiles = static_cast<int>(tile_count(g, BM, SHAPE));
  hipLaunchKernelGGL((ns_product_kernel<BM, BN, WR, WC, SHAPE, EPI, DEEP, SUMS>), dim3(static_cast<unsigned>(g.tiles * mats)),
                     dim3(WR * WC * 64), 0, s, g);
  return hipGetLastError();
}

// The tile for a product, by its modelled time: rounds of 256 tiles, one per CU,
// each with a part proportional to the summed index (us at 4096) and a fixed one,
// and the launch's own; fitted to launches at k = 256 to 4096 on MI355X.  Both
// sides of some choices, measured over whole calls with the symmetric products'
// tiles forced: 32 of 512 x 1024 take 338 us with 64, 347 with 128, 400 with 192;
// 3 of 777 x 1301, 189, 225, 321; 3000 x 3000, 1069, 847, 865; 4096 x 4096, 2240,
// 1693, 1430.  With C X's forced: 2 of 1024 x 4096, 319 with 64, 259 with 128, 269
// with 256; 4096 x 4096, 2193, 1554, 1416.
// With two sums the choice is that of one: the roundings that a product hands to the
// next lie in the order of its tiles.
template <Shape SHAPE, Epilogue EPI, int SUMS = 1>
hipError_t product(const Product& g, int64_t mats, hipStream_t s) {
  constexpr Shape kOwn = SHAPE == kRide ? kSym : SHAPE;
  constexpr bool kTri = kOwn == kSym;
  auto rounds = [&](int side, Shape shape) { return (tile_count(g, side, shape) * mats + 255) / 256; };
  const bool ride = SHAPE == kRide && rounds(64, kRide) < rounds(64, kSym);
  auto time = [&](int64_t n, double us, double fixed, double launch) {
    return static_cast<double>(n) * (us * (SUMS == 3 ? 3 : 1) * g.kk / 4096.0 + fixed) + launch;
  };
  const double large = kTri ? time(rounds(192, kOwn), 66.0, 11.0, 2.0) : time(rounds(256, kOwn), 115.0, 11.0, 2.0);
  const double t128 = time(rounds(128, kOwn), 32.0, 5.0, 3.0);
  const double t64 = time(rounds(64, ride ? kRide : kOwn), 17.0, 1.2, 1.5);
  if (t64 <= t128 && t64 <= large) {
    if constexpr (SHAPE == kRide) {
      // The tiles on the diagonal ride where that saves a round (1152 of 512 x 512 x
      // 512: 16 us without, 14 with; 300 of 1536 x 1536 x 4096, two rounds either way,
      // 27 and 28).  A long sum: more stages on their way, for fewer workgroups per
      // CU (2 of 1024 x 1024 x 4096: 29 and 23 us; of 1024 x 1024 x 1024, 8.5 and 8.7).
      if constexpr (EPI == kPlain) {
        if (g.kk > 1024)
          return ride ? product_tiles<64, 64, 2, 2, kRide, EPI, true>(g, mats, s)
                      : product_tiles<64, 64, 2, 2, kSym, EPI, true>(g, mats, s);
      }
      if (ride) return product_tiles<64, 64, 2, 2, kRide, EPI>(g, mats, s);
    }
    return product_tiles<64, 64, 2, 2, kOwn, EPI, false, SUMS>(g, mats, s);
  }
  if (t128 <= large) return product_tiles<128, 128, 2, 2, kOwn, EPI, false, SUMS>(g, mats, s);
  if constexpr (kTri)
    return product_tiles<192, 192, 2, 2, kOwn, EPI, false, SUMS>(g, mats, s);
  else
    return product_tiles<256, 256, 2, 4, kOwn, EPI, false, SUMS>(g, mats, s);
}

// The workspace: partial sums and factors, X and the next X, three k x k matrices, X's
// roundings or the low half of the next X, the low half of X, a fourth k x k matrix,
// each for all matrices.
struct Layout {
  int64_t k, l, kp, lp;
  int64_t e_mat;                                   // rounding errors of one matrix: whole tiles
  int64_t partials, f, x[2], sq[3], e, low, sq_low, bytes;  // byte offsets
  Layout(int64_t mats, int64_t rows, int64_t cols) {
    k = rows < cols ? rows : cols;
    l = rows < cols ? cols : rows;
    kp = pad_up(k);
    lp = pad_up(l);
    int64_t at = 0;
    auto take = [&](int64_t n) {
      const int64_t o = at;
      at += (n + 255) / 256 * 256;
      return o;
    };
    partials = take(mats * kNormParts * 8);
    f = take(mats * 4);
    for (int64_t& o : x) o = take(mats * kp * lp * 2);
    for (int64_t& o : sq) o = take(mats * k * kp * 2);
    e_mat = (k + kTile - 1) / kTile * kTile * ((l + kTile - 1) / kTile * kTile);
    e = take(mats * e_mat * 2);
    low = take(mats * kp * lp * 2);
    sq_low = take(mats * k * kp * 2);
    bytes = at + kTile * (lp > kp ? lp : kp) * 2;   // rows that the last tiles read past their matrix
  }
};

// ------------------------------------------------------------------ small matrices
// A matrix that fits one CU's LDS is taken through all its steps by one
// workgroup in one launch: the general path's launches, about 4 us each however
// small, would be nearly all of its time.  X (k x l, rows in order) and A, then
// C, are kept as pairs of FP16 values, v = hi + lo (22 bits), and a product is
// hi hi + hi lo + lo hi: matrix time is not what bounds these sizes, and small
// matrices gain most from the bits (2.6e-3 to 1.7e-3 off at 32 x 32, the BF16
// rounding of the result alone).  Step by step, in 16 x 16 blocks.
// Measured: 64 x 256 26.5 us (the general path 81), 96 x 96 28 (82), 16 x 16 11, 256
// of 64 x 256 32.  Of 63k clocks 64 x 256 takes 11k to load, norm and split, and per
// step 3.7k for A, 0.6k for A A, 1.1k for C and 4.9k for C X: LDS reads and the wait
// for them at every barrier.
struct SmallNs {
  NsInput in;
  uint16_t* out;
  int64_t out_row, out_mat;
  int k, l, lp, steps, tall, out_vec;
  float scale;
  float coefs[3 * ZERO_NS_MAX_STEPS];
};

typedef float acc4 __attribute__((ext_vector_type(4)));

// 8 values from `at` on.
__device__ __forceinline__ h8 row8(const half_t* p, int at) { return *reinterpret_cast<const h8*>(p + at); }

// Where element (row, col) of X lies, pitch XP a multiple of 128 values (256
// bytes, the banks once): the 16-byte piece of a row is moved by a permutation of
// row % 16, so that neither 16 rows' pieces of one column group nor the eight
// rows a transposing read takes from two pieces meet in a bank.  (A row pitch of
// 8 values more instead left half of the LDS time to conflicts: the 16 lanes
// served together are not 16 neighbours.)
__device__ __forceinline__ int fold(int row) {
  return ((row & 1) << 1) | ((row & 2) << 1) | (((row ^ (row << 1)) & 8)) | ((row >> 2) & 1);
}
template <int XP>
__device__ __forceinline__ int x_at(int row, int col) {
  return row * XP + ((((col >> 3) ^ fold(row))) << 3) + (col & 7);
}

// The same for A and C, KP values wide.
constexpr int small_pitch_s(int kp) { return kp <= 64 ? kp : 128; }
template <int KP>
__device__ __forceinline__ int s_at(int row, int col) {
  const int f = KP == 32 ? (row >> 2) & 3 : KP == 64 ? (row >> 1) & 7 : fold(row);
  return row * small_pitch_s(KP) + (((col >> 3) ^ f) << 3) + (col & 7);
}

// P Q^T of pairs, as three sums that do not wait for each other.
struct Acc3 {
  acc4 hh = {0, 0, 0, 0}, hl = {0, 0, 0, 0}, lh = {0, 0, 0, 0};
  __device__ __forceinline__ void add(const h8& ph, const h8& pl, const h8& qh, const h8& ql) {
    lh = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, qh, lh, 0, 0, 0);
    hl = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, ql, hl, 0, 0, 0);
    hh = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, qh, hh, 0, 0, 0);
  }
  __device__ __forceinline__ acc4 sum() const { return hh + (hl + lh); }
};

// 8 values down a column of X: rows k0 + 8 * (lane >> 4) + 0..7 of column c0 +
// (lane & 15).
template <int XP>
__device__ __forceinline__ h8 column8(const half_t* m, int k0, int c0, int lane) {
  const int row = k0 + (lane >> 4) * 8 + ((lane >> 2) & 3), col = c0 + (lane & 3) * 4;
  return __builtin_bit_cast(h8, transpose8(m + x_at<XP>(row, col), m + x_at<XP>(row + 4, col)));
}

__device__ __forceinline__ void split4(acc4 v, h4* hi, h4* lo) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    (*hi)[q] = static_cast<half_t>(v[q]);
    (*lo)[q] = static_cast<half_t>(v[q] - static_cast<float>((*hi)[q]));
  }
}

constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;
// For the smallest A its blocks are fewer than the waves: the summed index of A
// is then shared by `splits` waves, whose sums meet in LDS.
constexpr int small_splits(int kp) { return kp * kp / 256 >= kSmallWaves ? 1 : kSmallWaves / (kp * kp / 256); }
constexpr int small_lds(int kp, int xp) {
  return (2 * kp * xp + 2 * kp * small_pitch_s(kp)) * 2 + (small_splits(kp) > 1 ? small_splits(kp) * kp * kp * 4 : 0);
}
constexpr int kLdsBytes = 160 * 1024;

// XP, the pitch of X, is fixed so that a wave's addresses in X are few registers
// and constants.
template <int KP, int XP>
__global__ __launch_bounds__(kSmallThreads) void ns_small_kernel(SmallNs g) {
  extern __shared__ __align__(16) half_t lds[];
  const int lp = g.lp;
  constexpr int sp = small_pitch_s(KP), kSplits = small_splits(KP);
  half_t *xh = lds, *xl = xh + KP * XP, *sh = xl + KP * XP, *sl = sh + KP * sp;
  double* part = reinterpret_cast<double*>(sh);   // before A is
  float* sums = reinterpret_cast<float*>(sl + KP * sp);
  const int wave = threadIdx.x >> 6;
  int lane = threadIdx.x & 63;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * g.in.mat;

  const int per_row = (g.in.cols + 7) >> 3, groups = g.in.rows * per_row;
  constexpr int kGroups = (KP * XP / 8 + kSmallThreads - 1) / kSmallThreads;   // of 8 input values
  f8 v[kGroups];
  double sum = 0.0;
#pragma unroll
  for (int n = 0; n < kGroups; ++n) {
    const int i = threadIdx.x + n * kSmallThreads;
    v[n] = f8{};
    if (i < groups) {
      const int r = i / per_row;
      v[n] = load8(g.in, base + r * g.in.row, (i - r * per_row) * 8);
    }
  }
  for (int i = threadIdx.x; i < KP * XP / 4; i += kSmallThreads) reinterpret_cast<u32x4*>(xh)[i] = u32x4{};   // hi and lo
#pragma unroll
  for (int n = 0; n < kGroups; ++n)
#pragma unroll
    for (int q = 0; q < 8; ++q) sum += static_cast<double>(v[n][q]) * static_cast<double>(v[n][q]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kSmallWaves; ++i) sum += part[i];
  const NsScale x = scale_of(sum);
#pragma unroll
  for (int n = 0; n < kGroups; ++n) {
    const int i = threadIdx.x + n * kSmallThreads;
    if (i < groups) {
      const int r = i / per_row, c = (i - r * per_row) * 8;
      h8 h, l;   // past the end: load8's zeros
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float w = c + q < g.in.cols ? ldexpf(v[n][q], x.e) * x.f + x.add : 0.0f;
        h[q] = static_cast<half_t>(w);
        l[q] = static_cast<half_t>(w - static_cast<float>(h[q]));
      }
      if (!g.tall) {
        *reinterpret_cast<h8*>(xh + x_at<XP>(r, c)) = h;
        *reinterpret_cast<h8*>(xl + x_at<XP>(r, c)) = l;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (c + q < g.in.cols) {
            xh[x_at<XP>(c + q, r)] = h[q];
            xl[x_at<XP>(c + q, r)] = l[q];
          }
      }
    }
  }
  __syncthreads();

  // The blocks on and below the diagonal, or, where the waves share them, all.
  constexpr int kSide = KP / 16, kBlocks = kSplits > 1 ? kSide * kSide : kSide * (kSide + 1) / 2;
  constexpr int kMine = (kBlocks + kSmallWaves - 1) / kSmallWaves;
  auto block_row = [](int blk) {
    return kSplits > 1 ? blk / kSide : (blk >= 1) + (blk >= 3) + (blk >= 6) + (blk >= 10) + (blk >= 15);
  };
  auto block_col = [&](int blk) {
    const int bi = block_row(blk);
    return kSplits > 1 ? blk % kSide : blk - bi * (bi + 1) / 2;
  };
  for (int t = 0; t < g.steps; ++t) {
    const float a = g.coefs[3 * t], b = g.coefs[3 * t + 1], c = g.coefs[3 * t + 2];
    asm volatile("" : "+v"(lane));   // the LDS addresses are formed in every step: all of them do not fit the registers
    const int lr = lane & 15, lk = (lane >> 4) * 8, lq = (lane >> 4) * 4;   // a fragment's row, its first k; a result's first row
    // A block (bi, bj) of A or C, symmetric: the lane's four rows of a column as four
    // columns of a row, and, off the diagonal, as they are.
    auto store = [&](acc4 w, int bi, int bj) {
      const int at = s_at<KP>(bj + lr, bi + lq);
      h4 h, l;
      split4(w, &h, &l);
      *reinterpret_cast<h4*>(sh + at) = h;
      *reinterpret_cast<h4*>(sl + at) = l;
      if (kSplits == 1 && bi != bj) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int to = s_at<KP>(bi + lq + q, bj + lr);
          sh[to] = h[q];
          sl[to] = l[q];
        }
      }
    };
    // A = X X^T, the wave's blocks
    acc4 am[kMine];
    if constexpr (kSplits > 1) {
      const int blk = wave % kBlocks, part_k = wave / kBlocks;
      const int bi = block_row(blk) * 16, bj = block_col(blk) * 16;
      Acc3 s;
#pragma unroll 2
      for (int k0 = part_k * 32 + lk; k0 < lp; k0 += kSplits * 32)
        s.add(row8(xh, x_at<XP>(bi + lr, k0)), row8(xl, x_at<XP>(bi + lr, k0)), row8(xh, x_at<XP>(bj + lr, k0)),
              row8(xl, x_at<XP>(bj + lr, k0)));
      const acc4 w = s.sum();
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[(part_k * KP + bi + lq + q) * KP + bj + lr] = w[q];
      __syncthreads();
      am[0] = acc4{0, 0, 0, 0};
      if (wave < kBlocks)
#pragma unroll
        for (int n = 0; n < kSplits; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) am[0][q] += sums[(n * KP + bi + lq + q) * KP + bj + lr];
    } else {
#pragma unroll
      for (int n = 0; n < kMine; ++n) {
        const int blk = wave + n * kSmallWaves;
        Acc3 s;
        if (blk < kBlocks) {
          const int bi = block_row(blk) * 16 + lr, bj = block_col(blk) * 16 + lr;
#pragma unroll 4
          for (int k0 = lk; k0 < lp; k0 += 32)
            s.add(row8(xh, x_at<XP>(bi, k0)), row8(xl, x_at<XP>(bi, k0)), row8(xh, x_at<XP>(bj, k0)),
                  row8(xl, x_at<XP>(bj, k0)));
        }
        am[n] = s.sum();
        __builtin_amdgcn_sched_barrier(0);   // one block's fragments at a time: all of them do not fit the registers
      }
    }
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      const int blk = wave + n * kSmallWaves;
      if (blk < kBlocks) {
        am[n] *= kScaleA / (kScaleX * kScaleX);
        store(am[n], block_row(blk) * 16, block_col(blk) * 16);
      }
    }
    __syncthreads();
    // C = a I + b A + c A A
    acc4 sq[kMine];
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      const int blk = wave + n * kSmallWaves;
      Acc3 s;
      if (blk < kBlocks) {
        const int bi = block_row(blk) * 16 + lr, bj = block_col(blk) * 16 + lr;
#pragma unroll
        for (int k0 = 0; k0 < KP; k0 += 32)
          s.add(row8(sh, s_at<KP>(bi, k0 + lk)), row8(sl, s_at<KP>(bi, k0 + lk)), row8(sh, s_at<KP>(bj, k0 + lk)),
                row8(sl, s_at<KP>(bj, k0 + lk)));
      }
      sq[n] = s.sum();
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();   // A is read
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      const int blk = wave + n * kSmallWaves;
      if (blk < kBlocks) {
        const int bi = block_row(blk) * 16, bj = block_col(blk) * 16, r = bj + lr, col = bi + lq;
        acc4 w = c * (kScaleC / (kScaleA * kScaleA)) * sq[n] + b * (kScaleC / kScaleA) * am[n];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r == col + q && r < g.k) w[q] += a * kScaleC;
        store(w, bi, bj);
      }
    }
    __syncthreads();
    // X = C X in place: a wave reads a block of columns whole before it writes it
    const bool last = t == g.steps - 1;
#pragma unroll 1
    for (int c0 = wave * 16; c0 < lp; c0 += kSmallWaves * 16) {
      asm volatile("" : "+v"(lane)::"memory");   // nor C, which is read again for every block of columns
      const int lr = lane & 15, lk = (lane >> 4) * 8, lq = (lane >> 4) * 4;
      h8 ph[KP / 32], pl[KP / 32];
#pragma unroll
      for (int k0 = 0; k0 < KP / 32; ++k0) {
        ph[k0] = column8<XP>(xh, k0 * 32, c0, lane);
        pl[k0] = column8<XP>(xl, k0 * 32, c0, lane);
      }
#pragma unroll
      for (int bi = 0; bi < kSide; ++bi) {
        Acc3 s;
#pragma unroll
        for (int k0 = 0; k0 < KP / 32; ++k0) {
          const int at = s_at<KP>(bi * 16 + lr, k0 * 32 + lk);
          s.add(ph[k0], pl[k0], row8(sh, at), row8(sl, at));
        }
        acc4 w = s.sum();   // of X^T C: four columns of row bi * 16 + lr
        const int at = x_at<XP>(bi * 16 + lr, c0 + lq);
        if (!last) {
          split4(w * (1.0f / kScaleC), reinterpret_cast<h4*>(xh + at), reinterpret_cast<h4*>(xl + at));
        } else {   // the result, BF16, in place of hi
          u16x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = bf16_rne(w[q] * (g.scale / (kScaleC * kScaleX)));
          *reinterpret_cast<u16x4*>(xh + at) = o;
        }
        if constexpr (KP > 64) __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
  }
  // Out in 16-byte pieces.
  uint16_t* out = g.out + blockIdx.x * g.out_mat;
  if (!g.tall) {
    const int pieces = lp >> 3;
    for (int i = threadIdx.x; i < g.k * pieces; i += kSmallThreads) {
      const int r = i / pieces, c = (i - r * pieces) * 8;
      store8(out + r * g.out_row + c, *reinterpret_cast<const u32x4*>(xh + x_at<XP>(r, c)), g.out_vec, g.l - c);
    }
  } else {
    for (int c0 = wave * 16; c0 < lp; c0 += kSmallWaves * 16)
#pragma unroll
      for (int k0 = 0; k0 < KP; k0 += 32) {
        const int c = c0 + (lane & 15), r = k0 + (lane >> 4) * 8;
        const u32x4 piece = __builtin_bit_cast(u32x4, column8<XP>(xh, k0, c0, lane));
        if (c < g.l) store8(out + c * g.out_row + r, piece, g.out_vec, g.k - r);
      }
  }
}

template <int KP, int XP>
hipError_t small_launch(const SmallNs& g, int64_t mats, hipStream_t s) {
  constexpr int bytes = small_lds(KP, XP);
  static_assert(bytes <= kLdsBytes, "fits the LDS");
  hipLaunchKernelGGL((ns_small_kernel<KP, XP>), dim3(static_cast<unsigned>(mats)), dim3(kSmallThreads), bytes, s, g);
  return hipGetLastError();
}

// The pitch of X in the small kernel for a k x l matrix, 0 if it is not small.
constexpr int kPitches[3][2] = {{256, 1024}, {256, 512}, {128, 256}};
int small_pitch(int64_t k, int64_t l) {
  if (k > 96) return 0;
  for (int xp : kPitches[(k - 1) / 32])
    if (l <= xp) return xp;
  return 0;
}

hipError_t launch_small(const NsParams& p, const NsInput& in, hipStream_t s) {
  SmallNs g = {};
  g.in = in;
  g.out = p.out;
  g.out_row = p.out_row;
  g.out_mat = p.out_mat;
  g.tall = p.rows > p.cols;
  g.out_vec = (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0 && p.out_row % 8 == 0 && p.out_mat % 8 == 0;
  g.k = static_cast<int>(g.tall ? p.cols : p.rows);
  g.l = static_cast<int>(g.tall ? p.rows : p.cols);
  g.lp = (g.l + 31) / 32 * 32;
  g.steps = p.steps;
  g.scale = p.scale;
  for (int i = 0; i < 3 * p.steps; ++i) g.coefs[i] = p.coefs[i];
  const bool narrow = small_pitch(g.k, g.l) == kPitches[(g.k - 1) / 32][0];
  switch ((g.k + 31) / 32) {
    case 1: return narrow ? small_launch<32, kPitches[0][0]>(g, p.mats, s) : small_launch<32, kPitches[0][1]>(g, p.mats, s);
    case 2: return narrow ? small_launch<64, kPitches[1][0]>(g, p.mats, s) : small_launch<64, kPitches[1][1]>(g, p.mats, s);
    default: return narrow ? small_launch<96, kPitches[2][0]>(g, p.mats, s) : small_launch<96, kPitches[2][1]>(g, p.mats, s);
  }
}

}  // namespace

int64_t ns_workspace_bytes(int64_t mats, int64_t rows, int64_t cols) {
  if (mats == 0 || rows == 0 || cols == 0) return 0;
  return Layout(mats, rows, cols).bytes;
}

hipError_t launch_newton_schulz(const NsParams& p, hipStream_t s) {
  NsInput in{p.in, p.in_row, p.in_mat, static_cast<int>(p.rows), static_cast<int>(p.cols), p.in_f32, 0};
  const int64_t per16 = p.in_f32 ? 4 : 8;
  in.vec = (reinterpret_cast<uintptr_t>(p.in) & 15u) == 0 && p.in_row % per16 == 0 && p.in_mat % per16 == 0;
  if (small_pitch(p.rows < p.cols ? p.rows : p.cols, p.rows < p.cols ? p.cols : p.rows)) return launch_small(p, in, s);
  const Layout w(p.mats, p.rows, p.cols);
  char* ws = static_cast<char*>(p.workspace);
  const bool tall = p.rows > p.cols;
  const int k = static_cast<int>(w.k), l = static_cast<int>(w.l), kp = static_cast<int>(w.kp),
            lp = static_cast<int>(w.lp);
  half_t* x[2] = {reinterpret_cast<half_t*>(ws + w.x[0]), reinterpret_cast<half_t*>(ws + w.x[1])};
  half_t* sq[4] = {reinterpret_cast<half_t*>(ws + w.sq[0]), reinterpret_cast<half_t*>(ws + w.sq[1]),
                   reinterpret_cast<half_t*>(ws + w.sq[2]), reinterpret_cast<half_t*>(ws + w.sq_low)};
  float* f = reinterpret_cast<float*>(ws + w.f);
  half_t* e = reinterpret_cast<half_t*>(ws + w.e);
  half_t* low = p.in_f32 || p.pairs ? reinterpret_cast<half_t*>(ws + w.low) : nullptr;
  const int64_t x_mat = w.kp * w.lp, sq_mat = w.k * w.kp;

  double* partials = reinterpret_cast<double*>(ws + w.partials);
  const int64_t rows4 = (p.rows + kNormThreads / 64 - 1) / (kNormThreads / 64);
  const int parts = static_cast<int>(rows4 < kNormParts ? rows4 : kNormParts);
  hipLaunchKernelGGL(ns_norm_kernel, dim3(parts, static_cast<unsigned>(p.mats)), dim3(kNormThreads), 0, s, in, partials);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  NsX nx;
  nx.x = x[0];
  nx.next = x[1];
  nx.low = low;
  nx.next_low = p.pairs ? e : nullptr;
  nx.mat = x_mat;
  nx.tall = tall;
  nx.partials = partials;
  nx.parts = parts;
  nx.f = f;
  const dim3 turns(static_cast<unsigned>(pad_up(p.cols) / kTurn), static_cast<unsigned>(pad_up(p.rows) / kTurn),
                   static_cast<unsigned>(p.mats));
  if (low)
    hipLaunchKernelGGL(ns_prepare_kernel<true>, turns, dim3(kNormThreads), 0, s, in, nx);
  else
    hipLaunchKernelGGL(ns_prepare_kernel<false>, turns, dim3(kNormThreads), 0, s, in, nx);
  err = hipGetLastError();
  if (err != hipSuccess) return err;

  // k x k product u v^T into d, symmetric or not
  auto square = [&](bool sym, const half_t* u, const half_t* v, half_t* d, float alpha, const half_t* add, float beta,
                    float diag) {
    Product g = {};
    g.p = u;
    g.q = v;
    g.p_mat = g.q_mat = g.d_mat = sq_mat;
    g.p_ld = g.q_ld = g.d_ld = kp;
    g.m = g.n = k;
    g.kk = kp;
    g.d = d;
    g.alpha = alpha;
    g.add = add;
    g.beta = beta;
    g.diag = diag;
    if (add) return product<kRide, kPoly>(g, p.mats, s);
    return sym ? product<kSym, kPlain>(g, p.mats, s) : product<kFull, kPlain>(g, p.mats, s);
  };
  auto poly = [&](const half_t* a, half_t* d, int t) {
    const float* c = p.coefs + 3 * t;
    return square(true, a, a, d, c[2] * (kScaleC / (kScaleA * kScaleA)), a, c[1] * (kScaleC / kScaleA), c[0] * kScaleC);
  };

  // A = X X^T of the stored X (first: still short of the factor f)
  auto gram = [&](const half_t* from, half_t* d, bool first) {
    Product g = {};
    g.p = g.q = from;
    g.p_mat = g.q_mat = x_mat;
    g.p_ld = g.q_ld = lp;
    g.m = g.n = k;
    g.kk = lp;
    g.d = d;
    g.d_mat = sq_mat;
    g.d_ld = kp;
    g.alpha = kScaleA / (kScaleX * kScaleX);
    g.f = first ? f : nullptr;
    g.f_pow = 2;
    return product<kRide, kPlain>(g, p.mats, s);
  };
  // The last product with X goes to the output.
  auto result = [&](Product g, float c_scale) {
    g.alpha = p.scale / (c_scale * kScaleX);
    g.out = p.out;
    g.out_row = p.out_row;
    g.out_mat = p.out_mat;
    g.out_vec = (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0 && p.out_row % 8 == 0 && p.out_mat % 8 == 0;
    g.out_turned = tall;
    return g;
  };
  // X = C X into the other X, the last step's into the output.
  auto apply = [&](const half_t* c, float c_scale, int from, bool first, bool last, Epilogue carry) {
    Product g = {};
    g.f = first ? f : nullptr;
    g.f_pow = 1;
    g.p = c;
    g.p_mat = sq_mat;
    g.p_ld = kp;
    g.q = x[from];
    g.q_mat = x_mat;
    g.q_ld = lp;
    g.m = k;
    g.n = l;
    g.kk = kp;
    if (last) {
      g = result(g, c_scale);
    } else {
      g.alpha = 1.0f / c_scale;
      g.d = x[from ^ 1];
      g.d_mat = x_mat;
      g.d_ld = lp;
    }
    g.carry_out = e;
    g.carry_in = e;
    g.carry_mat = w.e_mat;
    if (first && low) {
      g.q_lo = low - x[0];
      if (last) return product<kTimesX, kOut, 2>(g, p.mats, s);
      if (carry == kCarryOut) return product<kTimesX, kCarryOut, 2>(g, p.mats, s);
      return product<kTimesX, kPlain, 2>(g, p.mats, s);
    }
    if (last) return product<kTimesX, kOut>(g, p.mats, s);
    if (carry == kCarryOut) return product<kTimesX, kCarryOut>(g, p.mats, s);
    if (carry == kCarryIn) return product<kTimesX, kCarryIn>(g, p.mats, s);
    return product<kTimesX, kPlain>(g, p.mats, s);
  };

  // Every launch in order, until one fails.
  hipError_t st = hipSuccess;
  auto run = [&](auto&& launch) {
    if (st == hipSuccess) st = launch();
  };
  if (p.pairs) {
    // Step by step, every matrix a pair: A in sq[0] and sq[2], C in sq[1] and sq[3].
    half_t* x_low[2] = {low, e};
    for (int t = 0; t < p.steps; ++t) {
      const int cur = t & 1;
      const float* c = p.coefs + 3 * t;
      Product a = {};
      a.p = a.q = x[cur];
      a.p_lo = a.q_lo = x_low[cur] - x[cur];
      a.p_mat = a.q_mat = x_mat;
      a.p_ld = a.q_ld = lp;
      a.m = a.n = k;
      a.kk = lp;
      a.d = sq[0];
      a.d_lo = sq[2] - sq[0];
      a.d_mat = sq_mat;
      a.d_ld = kp;
      a.alpha = kScaleA / (kScaleX * kScaleX);
      a.f = t == 0 ? f : nullptr;
      a.f_pow = 2;
      Product q = a;
      q.p = q.q = q.add = sq[0];
      q.p_lo = q.q_lo = q.add_lo = sq[2] - sq[0];
      q.p_mat = q.q_mat = sq_mat;
      q.p_ld = q.q_ld = q.kk = kp;
      q.d = sq[1];
      q.d_lo = sq[3] - sq[1];
      q.alpha = c[2] * (kScaleC / (kScaleA * kScaleA));
      q.beta = c[1] * (kScaleC / kScaleA);
      q.diag = c[0] * kScaleC;
      q.f = nullptr;
      Product y = {};
      y.p = sq[1];
      y.p_lo = sq[3] - sq[1];
      y.p_mat = sq_mat;
      y.p_ld = y.kk = kp;
      y.q = x[cur];
      y.q_lo = x_low[cur] - x[cur];
      y.q_mat = x_mat;
      y.q_ld = lp;
      y.m = k;
      y.n = l;
      y.f = t == 0 ? f : nullptr;
      y.f_pow = 1;
      y.alpha = 1.0f / kScaleC;
      y.d = x[cur ^ 1];
      y.d_lo = x_low[cur ^ 1] - x[cur ^ 1];
      y.d_mat = x_mat;
      y.d_ld = lp;
      run([&] { return product<kSym, kPlain, 3>(a, p.mats, s); });
      run([&] { return product<kSym, kPoly, 3>(q, p.mats, s); });
      if (t < p.steps - 1)
        run([&] { return product<kTimesX, kPlain, 3>(y, p.mats, s); });
      else
        run([&] { return product<kTimesX, kOut, 3>(result(y, kScaleC), p.mats, s); });
    }
    return st;
  }
  // Steps t and t + 1 as one product with X: its factor C' C into sq[0].
  auto pair = [&](int t, int from, bool first) {
    run([&] { return gram(x[from], sq[0], first); });
    run([&] { return poly(sq[0], sq[1], t); });
    run([&] { return square(true, sq[1], sq[0], sq[2], 1.0f / kScaleC, nullptr, 0, 0); });   // C A
    run([&] { return square(true, sq[1], sq[2], sq[0], 1.0f / kScaleC, nullptr, 0, 0); });   // A' = C (C A)^T
    run([&] { return poly(sq[0], sq[2], t + 1); });
    // C' C: its factors hold rounding errors, so it is not quite symmetric.  Half
    // of it will do for the first steps; after them the singular values are
    // spread wide enough that the other half is computed too (low-rank inputs
    // came out at 4.4e-3 instead of 6.7e-3 of their norm).
    run([&] { return square(first, sq[2], sq[1], sq[0], kScaleQ / (kScaleC * kScaleC), nullptr, 0, 0); });
  };

  const bool wide = l >= 2 * k;
  int t = 0, cur = 0;
  if (p.steps == 1) {
    run([&] { return gram(x[0], sq[0], true); });
    run([&] { return poly(sq[0], sq[1], 0); });
    run([&] { return apply(sq[1], kScaleC, 0, true, true, kPlain); });
    return st;
  }
  // The first two steps together: X is still exact, and the second step's X
  // need not be rounded.
  pair(0, 0, true);
  t = 2;
  // X after two steps: its rounding errors are carried into the next product.
  const bool carries = p.steps >= 4 && !(wide && p.steps == 4);
  run([&] { return apply(sq[0], kScaleQ, 0, true, t == p.steps, carries ? kCarryOut : kPlain); });
  cur = 1;
  while (t < p.steps) {
    // The last two together where X is long: one product with X less for two
    // more k x k products.
    if (wide && p.steps - t == 2) {
      pair(t, cur, false);
      t += 2;
      run([&] { return apply(sq[0], kScaleQ, cur, false, true, kPlain); });
    } else {
      const Epilogue carry = carries && t == 2 ? kCarryIn : kPlain;
      run([&] { return gram(x[cur], sq[0], false); });
      run([&] { return poly(sq[0], sq[1], t); });
      ++t;
      run([&] { return apply(sq[1], kScaleC, cur, false, t == p.steps, carry); });
    }
    cur ^= 1;
  }
  return st;
}

}  // namespace zero
