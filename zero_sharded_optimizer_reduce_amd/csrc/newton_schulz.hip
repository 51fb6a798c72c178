// gfx950 kernels of zero_newton_schulz: X = G/||G||_F, then per step
//   A = X X^T,  C = a I + b A + c A A,  X = C X.
//
// Shapes.  k = the smaller side, l = the larger: X is taken k x l (a tall
// input is its transpose), so A and C are k x k.  Every product is written
// with both operands' summed index contiguous in memory, D = P Q^T: A = X X^T
// and A A = A A^T as they stand, X' = C (X^T)^T from a second copy of X kept
// transposed.  Products of commuting polynomials of one symmetric matrix are
// symmetric: only tiles on and below the diagonal are computed, and written
// twice.
//
// Blocks of steps.  With C_0, C_1 polynomials of A, two steps are
//   A' = C_0 A C_0,  C_1 = a I + b A' + c A' A',  X'' = (C_1 C_0) X:
// a Gram product and a product with X (3 k k l) less and three symmetric k x k
// products (3 k k k) more than step by step.
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
#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"

namespace zero {
namespace {

typedef _Float16 half_t;
typedef half_t h8 __attribute__((ext_vector_type(8)));
typedef half_t h4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
constexpr int kNormParts = 256;  // partial sums per matrix, at most

struct NsInput {
  const void* in;
  int64_t row, mat;   // strides in elements
  int rows, cols;
  int f32;
};

__device__ __forceinline__ float load_in(const NsInput& g, int64_t at) {
  if (g.f32) return static_cast<const float*>(g.in)[at];
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(g.in)[at]) << 16);
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

// Partial sums of squares, in FP64 and in an order fixed by the shape: block b
// of a matrix takes its rows b, b + parts, ...
__global__ __launch_bounds__(kNormThreads) void ns_norm_kernel(NsInput g, double* partials) {
  const int64_t base = static_cast<int64_t>(blockIdx.y) * g.mat;
  double acc = 0.0;
  for (int r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const int64_t row = base + static_cast<int64_t>(r) * g.row;
    for (int c = threadIdx.x; c < g.cols; c += kNormThreads) {
      const double v = load_in(g, row + c);
      acc += v * v;
    }
  }
  const double t = block_sum(acc);
  if (threadIdx.x == 0) partials[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = t;
}

// ------------------------------------------------------------------ X
// X * kScaleX = f * (G * 2^e) with f in [1/2, 1): the stored G * 2^e is exact
// for BF16 inputs (8 bits in 11), and the factor f joins the products' scales,
// so that nothing is lost before the first product.
struct NsX {
  half_t* same;      // G's own orientation, rows x cols, pitch pad(cols)
  half_t* turned;    // cols x rows, pitch pad(rows)
  int64_t same_mat, turned_mat;
  float* f;          // per matrix
  const double* partials;
  int parts;
};

constexpr int kTurn = 64;

__global__ __launch_bounds__(kNormThreads) void ns_prepare_kernel(NsInput g, NsX x) {
  __shared__ half_t tile[kTurn][kTurn + 2];
  const int mat = blockIdx.z;
  double sum = 0.0;
  for (int i = threadIdx.x; i < x.parts; i += kNormThreads) sum += x.partials[static_cast<int64_t>(mat) * x.parts + i];
  sum = block_sum(sum);
  // 2^e and f from kScaleX / norm = f * 2^e; a zero matrix stays zero, and a
  // sum that is not finite makes everything NaN
  int e = 0;
  double f = 1.0, mult = 0.0;
  if (sum > 0.0 && sum < __builtin_huge_val()) {
    f = frexp(static_cast<double>(kScaleX) / sqrt(sum), &e);
    mult = ldexp(1.0, e);
  } else if (sum != 0.0) {
    mult = __builtin_nan("");
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) x.f[mat] = static_cast<float>(f);
  const int r0 = blockIdx.y * kTurn, c0 = blockIdx.x * kTurn;
  const int pc = static_cast<int>(pad_up(g.cols)), pr = static_cast<int>(pad_up(g.rows));
  half_t* same = x.same + mat * x.same_mat;
  half_t* turned = x.turned + mat * x.turned_mat;
  const int64_t base = static_cast<int64_t>(mat) * g.mat;
  const int c = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < kTurn; i += kNormThreads / 64) {
    const int r = r0 + i;
    half_t v = 0;
    if (r < g.rows && c0 + c < g.cols) {
      const double w = load_in(g, base + static_cast<int64_t>(r) * g.row + c0 + c);
      v = static_cast<half_t>(static_cast<float>(w * mult));
    }
    tile[i][c] = v;
    if (r < g.rows && c0 + c < pc) same[static_cast<int64_t>(r) * pc + c0 + c] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x >> 6; i < kTurn; i += kNormThreads / 64)
    if (c0 + i < g.cols && r0 + c < pr) turned[static_cast<int64_t>(c0 + i) * pr + r0 + c] = tile[c][i];
}

// ------------------------------------------------------------------ products
// D = alpha' P Q^T with P m x kk, Q n x kk (pitches p_ld, q_ld; kk a multiple of
// kPad, the padding zero).
struct Product {
  const half_t* p;
  const half_t* q;
  int64_t p_mat, q_mat;
  int p_ld, q_ld;
  int m, n, kk;
  int tiles_n, tiles;       // per matrix
  // FP16 results: d row-major (columns n up to d_ld written, the padding as
  // zeros) and dt its transpose; either may be NULL.  For a symmetric product
  // both are the same matrix.
  half_t* d;
  half_t* dt;
  int64_t d_mat, dt_mat;
  int d_ld, dt_ld;
  const half_t* add;        // polynomial: beta * add + diag * I joins (symmetric, pitch d_ld)
  float alpha, beta, diag;
  const float* f;           // per-matrix factor of alpha, or NULL
  int f_pow;
  uint16_t* out;            // BF16 result instead of d, dt
  int64_t out_row, out_mat;
  int out_vec;              // 16-byte stores are aligned
  half_t* carry_out;        // the FP16 roundings of d, in the lanes' own order, or NULL
  const half_t* carry_in;   // those of the X this product reads, or NULL
  int64_t carry_mat;
};

constexpr int kTile = 128;
constexpr int kBk = 64;     // summed index per stage: rows of 128 bytes in LDS

// Rows [row0, row0 + R) of an operand, columns [k0, k0 + 64), into LDS as R rows
// of 128 bytes; the 16-byte piece c of row r lies at piece c ^ (r & 7), so that
// the 16 rows of a fragment read fall into different banks.  Each wave moves
// 1 KiB (8 rows) per instruction, straight to LDS.  Rows past the end read the
// last row again (their results are dropped).
template <int R, int NW>
struct Stager {
  static constexpr int kN = R / 8 / NW;
  static_assert(kN * 8 * NW == R, "every wave moves the same number of pieces");
  __amdgpu_buffer_rsrc_t rsrc;
  int voff[kN];
  int wave;
  __device__ __forceinline__ Stager(const half_t* mat, int ld, int rows, int row0, int wave_, int lane) : wave(wave_) {
    const half_t* base = mat + static_cast<int64_t>(row0) * ld;
    const int left = rows - row0;
    const int64_t bytes = static_cast<int64_t>(left < R ? left : R) * ld * 2;
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<half_t*>(base), 0, static_cast<int>(bytes), 0x00020000);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = (wave * kN + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ (r & 7);
      const int rr = r < left ? r : left - 1;
      voff[i] = rr * ld * 2 + c * 16;
    }
  }
  __device__ __forceinline__ void issue(half_t* lds, int k0) const {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (wave * kN + i) * 8 * kBk), 16, voff[i],
                                               k0 * 2, 0, 0);
  }
};

template <int R>
__device__ __forceinline__ h8 frag(const half_t* lds, int row, int piece) {
  return *reinterpret_cast<const h8*>(lds + row * kBk + ((piece ^ (row & 7)) << 3));
}

template <int NW>
__device__ __forceinline__ float block_sum_f32(float x, float* lds) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) t += lds[i];
  return t;
}

// One tile BM x BN by WR x WC waves.  SYM: lower tiles of a symmetric product.
template <int BM, int BN, int WR, int WC, bool SYM>
__global__ __launch_bounds__(WR * WC * 64) void ns_product_kernel(Product g) {
  constexpr int NW = WR * WC;
  constexpr int TM = BM / WR / 16, TN = BN / WC / 16;
  constexpr int kStage = (BM + BN) * kBk;
  constexpr int kOut = BM * (BN + 8) > BN * (BM + 8) ? BM * (BN + 8) : BN * (BM + 8);
  __shared__ __align__(16) half_t lds[2 * kStage > kOut ? 2 * kStage : kOut];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int mat = blockIdx.x / g.tiles;
  const int t = blockIdx.x - mat * g.tiles;
  int ti, tj;
  if (SYM) {
    ti = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > t) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    tj = t - ti * (ti + 1) / 2;
  } else {
    ti = t / g.tiles_n;
    tj = t - ti * g.tiles_n;
  }
  const int row0 = ti * BM, col0 = tj * BN;
  const Stager<BM, NW> sp(g.p + mat * g.p_mat, g.p_ld, g.m, row0, wave, lane);
  const Stager<BN, NW> sq(g.q + mat * g.q_mat, g.q_ld, g.n, col0, wave, lane);
  const int wr = wave / WC, wc = wave - wr * WC;
  f4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f4{0, 0, 0, 0};

  sp.issue(lds, 0);
  sq.issue(lds + BM * kBk, 0);
  for (int k0 = 0, s = 0; k0 < g.kk; k0 += kBk, s ^= 1) {
    __syncthreads();   // stage s has arrived; the other is free
    half_t* cur = lds + s * kStage;
    half_t* nxt = lds + (s ^ 1) * kStage;
    if (k0 + kBk < g.kk) {
      sp.issue(nxt, k0 + kBk);
      sq.issue(nxt + BM * kBk, k0 + kBk);
    }
#pragma unroll
    for (int h = 0; h < kBk / 32; ++h) {
      h8 a[TM], b[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        a[i] = frag<BM>(cur, wr * TM * 16 + i * 16 + (lane & 15), h * 4 + (lane >> 4));
#pragma unroll
      for (int j = 0; j < TN; ++j)
        b[j] = frag<BN>(cur + BM * kBk, wc * TN * 16 + j * 16 + (lane & 15), h * 4 + (lane >> 4));
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }

  // The lane's values: rows row0 + wr*.. + i*16 + (lane>>4)*4 + 0..3, one column.
  float alpha = g.alpha;
  if (g.f) {
    const float f = g.f[mat];
    alpha *= g.f_pow == 2 ? f * f : f;
  }
  const half_t* add = g.add ? g.add + mat * g.d_mat : nullptr;
  float gain = 0.0f;
  if (g.carry_in) {
    const half_t* c = g.p + mat * g.p_mat;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < g.m; i += NW * 64) sum += static_cast<float>(c[static_cast<int64_t>(i) * g.p_ld + i]);
    gain = block_sum_f32<NW>(sum, reinterpret_cast<float*>(lds)) * g.alpha / (static_cast<float>(g.m) * kScaleE);
  }
  const int lr = wr * TM * 16 + ((lane >> 4) << 2), lc = wc * TN * 16 + (lane & 15);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int r = row0 + lr + i * 16, c = col0 + lc + j * 16;
      f4 v = acc[i][j] * alpha;
      if (add && c < g.n && r < g.m) {
        // add is symmetric: the lane's four rows of column c are four columns of row c
        const h4 w = *reinterpret_cast<const h4*>(add + static_cast<int64_t>(c) * g.d_ld + r);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] += g.beta * static_cast<float>(w[q]);
          if (r + q == c) v[q] += g.diag;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (r + q >= g.m || c >= g.n) v[q] = 0.0f;
      const int64_t at = mat * g.carry_mat + ((static_cast<int64_t>(t) * TM + i) * TN + j) * (NW * 256) + threadIdx.x * 4;
      if (g.carry_in) {
        const h4 w = *reinterpret_cast<const h4*>(g.carry_in + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += gain * static_cast<float>(w[q]);
      }
      if (g.carry_out) {
        h4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = static_cast<half_t>((v[q] - static_cast<float>(static_cast<half_t>(v[q]))) * kScaleE);
        *reinterpret_cast<h4*>(g.carry_out + at) = w;
      }
      acc[i][j] = v;
    }

  // Results go through LDS so that rows leave in whole lines.
  uint16_t* o16 = reinterpret_cast<uint16_t*>(lds);
  auto bits = [&](float v) {
    return g.out ? bf16_rne(v) : __builtin_bit_cast(uint16_t, static_cast<half_t>(v));
  };
  if (g.d || g.out) {
    constexpr int pitch = BN + 8;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) o16[(lr + i * 16 + q) * pitch + lc + j * 16] = bits(acc[i][j][q]);
    __syncthreads();
    for (int at = threadIdx.x; at < BM * (BN / 8); at += NW * 64) {
      const int r = at / (BN / 8), c = (at - r * (BN / 8)) * 8;
      if (row0 + r >= g.m) continue;
      const uint16_t* src = o16 + r * pitch + c;
      if (!g.out) {
        if (col0 + c < g.d_ld)
          *reinterpret_cast<u32x4*>(g.d + mat * g.d_mat + static_cast<int64_t>(row0 + r) * g.d_ld + col0 + c) =
              *reinterpret_cast<const u32x4*>(src);
      } else {
        uint16_t* dst = g.out + mat * g.out_mat + static_cast<int64_t>(row0 + r) * g.out_row + col0 + c;
        if (g.out_vec && col0 + c + 8 <= g.n) {
          *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
        } else {
          for (int q = 0; q < 8; ++q)
            if (col0 + c + q < g.n) dst[q] = src[q];
        }
      }
    }
  }
  if (g.dt && !(SYM && ti == tj)) {
    constexpr int pitch = BM + 8;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        h4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = static_cast<half_t>(acc[i][j][q]);
        *reinterpret_cast<h4*>(reinterpret_cast<half_t*>(lds) + (lc + j * 16) * pitch + lr + i * 16) = w;
      }
    __syncthreads();
    for (int at = threadIdx.x; at < BN * (BM / 8); at += NW * 64) {
      const int c = at / (BM / 8), r = (at - c * (BM / 8)) * 8;
      if (col0 + c >= g.n || row0 + r >= g.dt_ld) continue;
      *reinterpret_cast<u32x4*>(g.dt + mat * g.dt_mat + static_cast<int64_t>(col0 + c) * g.dt_ld + row0 + r) =
          *reinterpret_cast<const u32x4*>(o16 + c * pitch + r);
    }
  }
}

// (named here because clang's host pass leaves out the second stub otherwise)
template __global__ void ns_product_kernel<128, 128, 2, 2, true>(Product);
template __global__ void ns_product_kernel<128, 128, 2, 2, false>(Product);

// ------------------------------------------------------------------ launches
template <bool SYM>
hipError_t product(Product g, int64_t mats, hipStream_t s) {
  const int tm = (g.m + kTile - 1) / kTile;
  g.tiles_n = (g.n + kTile - 1) / kTile;
  g.tiles = SYM ? tm * (tm + 1) / 2 : tm * g.tiles_n;
  hipLaunchKernelGGL((ns_product_kernel<kTile, kTile, 2, 2, SYM>), dim3(static_cast<unsigned>(g.tiles * mats)),
                     dim3(256), 0, s, g);
  return hipGetLastError();
}

// The workspace: partial sums and factors, two turns of X^T and one X, three
// k x k matrices, each for all matrices.
struct Layout {
  int64_t k, l, kp, lp;
  int64_t e_mat;                                   // rounding errors of one matrix: whole tiles
  int64_t partials, f, x, xt[2], sq[3], e, bytes;  // byte offsets
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
    x = take(mats * k * lp * 2);
    for (int64_t& o : xt) o = take(mats * l * kp * 2);
    for (int64_t& o : sq) o = take(mats * k * kp * 2);
    e_mat = (k + kTile - 1) / kTile * kTile * ((l + kTile - 1) / kTile * kTile);
    e = take(mats * e_mat * 2);
    bytes = at;
  }
};

}  // namespace

int64_t ns_workspace_bytes(int64_t mats, int64_t rows, int64_t cols) {
  if (mats == 0 || rows == 0 || cols == 0) return 0;
  return Layout(mats, rows, cols).bytes;
}

hipError_t launch_newton_schulz(const NsParams& p, hipStream_t s) {
  const Layout w(p.mats, p.rows, p.cols);
  char* ws = static_cast<char*>(p.workspace);
  const bool tall = p.rows > p.cols;
  const int k = static_cast<int>(w.k), l = static_cast<int>(w.l), kp = static_cast<int>(w.kp),
            lp = static_cast<int>(w.lp);
  half_t* x = reinterpret_cast<half_t*>(ws + w.x);
  half_t* xt[2] = {reinterpret_cast<half_t*>(ws + w.xt[0]), reinterpret_cast<half_t*>(ws + w.xt[1])};
  half_t* sq[3] = {reinterpret_cast<half_t*>(ws + w.sq[0]), reinterpret_cast<half_t*>(ws + w.sq[1]),
                   reinterpret_cast<half_t*>(ws + w.sq[2])};
  float* f = reinterpret_cast<float*>(ws + w.f);
  half_t* e = reinterpret_cast<half_t*>(ws + w.e);
  const int64_t x_mat = w.k * w.lp, xt_mat = w.l * w.kp, sq_mat = w.k * w.kp;

  NsInput in{p.in, p.in_row, p.in_mat, static_cast<int>(p.rows), static_cast<int>(p.cols), p.in_f32};
  double* partials = reinterpret_cast<double*>(ws + w.partials);
  const int parts = static_cast<int>(p.rows < kNormParts ? p.rows : kNormParts);
  hipLaunchKernelGGL(ns_norm_kernel, dim3(parts, static_cast<unsigned>(p.mats)), dim3(kNormThreads), 0, s, in, partials);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  NsX nx;
  nx.same = tall ? xt[0] : x;
  nx.turned = tall ? x : xt[0];
  nx.same_mat = tall ? xt_mat : x_mat;
  nx.turned_mat = tall ? x_mat : xt_mat;
  nx.f = f;
  nx.partials = partials;
  nx.parts = parts;
  hipLaunchKernelGGL(ns_prepare_kernel,
                     dim3(static_cast<unsigned>(pad_up(p.cols) / kTurn), static_cast<unsigned>(pad_up(p.rows) / kTurn),
                          static_cast<unsigned>(p.mats)),
                     dim3(kNormThreads), 0, s, in, nx);
  err = hipGetLastError();
  if (err != hipSuccess) return err;

  // symmetric k x k product of u and v into d
  auto square = [&](const half_t* u, const half_t* v, half_t* d, float alpha, const half_t* add, float beta, float diag) {
    Product g = {};
    g.p = u;
    g.q = v;
    g.p_mat = g.q_mat = g.d_mat = g.dt_mat = sq_mat;
    g.p_ld = g.q_ld = g.d_ld = g.dt_ld = kp;
    g.m = g.n = k;
    g.kk = kp;
    g.d = g.dt = d;
    g.alpha = alpha;
    g.add = add;
    g.beta = beta;
    g.diag = diag;
    return product<true>(g, p.mats, s);
  };
  auto poly = [&](const half_t* a, half_t* d, int t) {
    const float* c = p.coefs + 3 * t;
    return square(a, a, d, c[2] * (kScaleC / (kScaleA * kScaleA)), a, c[1] * (kScaleC / kScaleA), c[0] * kScaleC);
  };

  // A = X X^T of the stored X (first: still short of the factor f)
  auto gram = [&](half_t* d, bool first) {
    Product g = {};
    g.p = g.q = x;
    g.p_mat = g.q_mat = x_mat;
    g.p_ld = g.q_ld = lp;
    g.m = g.n = k;
    g.kk = lp;
    g.d = g.dt = d;
    g.d_mat = g.dt_mat = sq_mat;
    g.d_ld = g.dt_ld = kp;
    g.alpha = kScaleA / (kScaleX * kScaleX);
    g.f = first ? f : nullptr;
    g.f_pow = 2;
    return product<true>(g, p.mats, s);
  };
  // X = C X from the transposed copy xt[from]: into x and xt[to], the last
  // step's into the output.
  enum { kCarryOut = 1, kCarryIn = 2 };
  auto apply = [&](const half_t* c, float c_scale, int from, bool first, int to, bool last, int carry) {
    Product g = {};
    g.f = first ? f : nullptr;
    g.f_pow = 1;
    g.kk = kp;
    const bool turned = last && tall;   // the result's own orientation
    g.p = turned ? xt[from] : c;
    g.q = turned ? c : xt[from];
    g.p_mat = turned ? xt_mat : sq_mat;
    g.q_mat = turned ? sq_mat : xt_mat;
    g.p_ld = g.q_ld = kp;
    g.m = turned ? l : k;
    g.n = turned ? k : l;
    if (last) {
      g.alpha = p.scale / (c_scale * kScaleX);
      g.out = p.out;
      g.out_row = p.out_row;
      g.out_mat = p.out_mat;
      g.out_vec = (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0 && p.out_row % 8 == 0 && p.out_mat % 8 == 0;
    } else {
      g.alpha = 1.0f / c_scale;
      g.d = x;
      g.d_mat = x_mat;
      g.d_ld = lp;
      g.dt = xt[to];
      g.dt_mat = xt_mat;
      g.dt_ld = kp;
    }
    g.carry_out = carry == kCarryOut ? e : nullptr;
    g.carry_in = carry == kCarryIn ? e : nullptr;
    g.carry_mat = w.e_mat;
    return product<false>(g, p.mats, s);
  };

  // Every launch in order, until one fails.
  hipError_t st = hipSuccess;
  auto run = [&](auto&& launch) {
    if (st == hipSuccess) st = launch();
  };
  // Steps t and t + 1 as one product with X: its factor C' C into sq[0].
  auto pair = [&](int t, bool first) {
    run([&] { return gram(sq[0], first); });
    run([&] { return poly(sq[0], sq[1], t); });
    run([&] { return square(sq[0], sq[1], sq[2], 1.0f / kScaleC, nullptr, 0, 0); });   // A C
    run([&] { return square(sq[2], sq[1], sq[0], 1.0f / kScaleC, nullptr, 0, 0); });   // A' = A C C
    run([&] { return poly(sq[0], sq[2], t + 1); });
    run([&] { return square(sq[2], sq[1], sq[0], kScaleQ / (kScaleC * kScaleC), nullptr, 0, 0); });
  };

  const bool wide = l >= 2 * k;
  int t = 0, cur = 0;
  if (p.steps == 1) {
    run([&] { return gram(sq[0], true); });
    run([&] { return poly(sq[0], sq[1], 0); });
    run([&] { return apply(sq[1], kScaleC, 0, true, 1, true, 0); });
    return st;
  }
  // The first two steps together: X is still exact, and the second step's X
  // need not be rounded.
  pair(0, true);
  t = 2;
  // X after two steps: its rounding errors are carried into the next product.
  const bool carries = p.steps >= 4 && !(wide && p.steps == 4);
  run([&] { return apply(sq[0], kScaleQ, 0, true, 1, t == p.steps, carries ? kCarryOut : 0); });
  cur = 1;
  while (t < p.steps) {
    // The last two together where X is long: one product with X less for two
    // more k x k products.
    if (wide && p.steps - t == 2) {
      pair(t, false);
      t += 2;
      run([&] { return apply(sq[0], kScaleQ, cur, false, cur ^ 1, true, 0); });
    } else {
      const int carry = carries && t == 2 ? kCarryIn : 0;
      run([&] { return gram(sq[0], false); });
      run([&] { return poly(sq[0], sq[1], t); });
      ++t;
      run([&] { return apply(sq[1], kScaleC, cur, false, cur ^ 1, t == p.steps, carry); });
    }
    cur ^= 1;
  }
  return st;
}

}  // namespace zero
