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
constexpr int kNormParts = 1024;  // partial sums per matrix, at most

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

// Per matrix kScaleX / norm = f * 2^e with f in [1/2, 1).  A zero matrix stays
// zero; `add` makes everything NaN when the sum of squares is not finite.
struct NsScale {
  float f, add;
  int e, unused;
};

__global__ __launch_bounds__(kNormThreads) void ns_scale_kernel(const double* partials, int parts, NsScale* scales) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kNormThreads) sum += partials[static_cast<int64_t>(blockIdx.x) * parts + i];
  sum = block_sum(sum);
  if (threadIdx.x != 0) return;
  NsScale s = {1.0f, 0.0f, 0, 0};
  if (sum > 0.0 && sum < __builtin_huge_val())
    s.f = static_cast<float>(frexp(static_cast<double>(kScaleX) / sqrt(sum), &s.e));
  else if (sum != 0.0)
    s.add = __builtin_nanf("");
  scales[blockIdx.x] = s;
}

// ------------------------------------------------------------------ X
// X * kScaleX = f * (G * 2^e): the stored G * 2^e is exact for BF16 inputs (8
// bits in 11), and the factor f joins the products' scales, so that nothing is
// lost before the first product.
struct NsX {
  half_t* same;      // G's own orientation, rows x cols, pitch pad(cols)
  half_t* turned;    // cols x rows, pitch pad(rows)
  int64_t same_mat, turned_mat;
  const NsScale* scales;
};

constexpr int kTurn = 64;

// One 64 x 64 tile to both copies; the padding is written as zeros.
__global__ __launch_bounds__(kNormThreads) void ns_prepare_kernel(NsInput g, NsX x) {
  // 33 words a row: the eight rows a lane group gathers lie in different banks
  __shared__ uint32_t tile[kTurn][kTurn / 2 + 1];
  const int mat = blockIdx.z;
  const NsScale s = x.scales[mat];
  const int r0 = blockIdx.y * kTurn, c0 = blockIdx.x * kTurn;
  const int pc = static_cast<int>(pad_up(g.cols)), pr = static_cast<int>(pad_up(g.rows));
  half_t* same = x.same + mat * x.same_mat;
  half_t* turned = x.turned + mat * x.turned_mat;
  const int64_t base = static_cast<int64_t>(mat) * g.mat;
  const int line = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
#pragma unroll
  for (int i = line; i < kTurn; i += kNormThreads / 8) {
    const int r = r0 + i;
    f8 v = {};
    if (r < g.rows) v = load8(g, base + static_cast<int64_t>(r) * g.row, c0 + c);
    h8 h;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      h[q] = r < g.rows && c0 + c + q < g.cols ? static_cast<half_t>(ldexpf(v[q], s.e) + s.add) : half_t(0);
    if (r < g.rows) *reinterpret_cast<h8*>(same + static_cast<int64_t>(r) * pc + c0 + c) = h;
    const u32x4 w = __builtin_bit_cast(u32x4, h);
#pragma unroll
    for (int q = 0; q < 4; ++q) tile[i][c / 2 + q] = w[q];
  }
  __syncthreads();
#pragma unroll
  for (int i = line; i < kTurn; i += kNormThreads / 8) {
    if (c0 + i >= g.cols) continue;
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a = tile[c + 2 * q][i >> 1], b = tile[c + 2 * q + 1][i >> 1];
      w[q] = i & 1 ? (a >> 16) | (b & 0xFFFF0000u) : (a & 0xFFFFu) | (b << 16);
    }
    *reinterpret_cast<u32x4*>(turned + static_cast<int64_t>(c0 + i) * pr + r0 + c) = w;
  }
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
  const NsScale* scales;    // per-matrix factor f of alpha, or NULL
  int f_pow;
  uint16_t* out;            // BF16 result instead of d, dt
  int64_t out_row, out_mat;
  int out_vec;              // 16-byte stores are aligned
  half_t* carry_out;        // the FP16 roundings of d, in the lanes' own order, or NULL
  const half_t* carry_in;   // those of the X this product reads, or NULL
  int64_t carry_mat;
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
template <int R, int NW>
struct Stager {
  static constexpr int kN = R / 8 / NW;
  static_assert(kN * 8 * NW == R && kN % 2 == 0, "every wave moves the same number of pieces, an even one");
  __amdgpu_buffer_rsrc_t rsrc;
  int voff[2], step, wave;   // even and odd groups of 8 rows
  __device__ __forceinline__ Stager(const half_t* mat, int ld, int row0, int wave_, int lane) : wave(wave_) {
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<half_t*>(mat + static_cast<int64_t>(row0) * ld), 0, R * ld * 2,
                                             0x00020000);
    const int r = wave * kN * 8 + (lane >> 3);
    voff[0] = r * ld * 2 + ((lane & 7) ^ (lane >> 4)) * 16;
    voff[1] = voff[0] ^ 64;   // ld is a multiple of 64
    step = 8 * ld * 2;
  }
  __device__ __forceinline__ void one(half_t* lds, int k0, int i) const {
#ifdef __HIP_DEVICE_COMPILE__   // the builtin is unknown to the host pass
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (wave * kN + i) * 8 * kBk), 16, voff[i & 1],
                                             k0 * 2 + i * step, 0, 0);
#endif
  }
  __device__ __forceinline__ void all(half_t* lds, int k0) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) one(lds, k0, i);
  }
};

// A wave's operands for half a stage: two 16-wide pieces of the summed index.
template <int TM, int TN>
struct Frags {
  static constexpr int kReads = 2 * (TM + TN);
  h8 a[2][TM], b[2][TN];
  // Read number n of kReads; at_p, at_q: the lane's byte offsets in a slot (see
  // lane_at); half 0 or 1.
  __device__ __forceinline__ void one(const half_t* p, const half_t* q, int at_p, int at_q, int half, int n) {
    const int u = n / (TM + TN), i = n - u * (TM + TN);
    if (i < TM)
      a[u][i] = *reinterpret_cast<const h8*>(reinterpret_cast<const char*>(p) + (at_p ^ (half * 64 + u * 32)) +
                                             i * 32 * kBk * 2);
    else
      b[u][i - TM] = *reinterpret_cast<const h8*>(reinterpret_cast<const char*>(q) + (at_q ^ (half * 64 + u * 32)) +
                                                  (i - TM) * 32 * kBk * 2);
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

// One tile BM x BN by WR x WC waves.  SYM: lower tiles of a symmetric product.
//
// The loop over the summed index keeps one to one and a half stages on their
// way to LDS and half a stage ahead in registers: while the matrix cores work
// on one half the wave reads the next one's fragments, and the loads are issued
// evenly between the products (a wave issues in order: loads in a row
// hold its products up while the CU takes them in, about 26 clocks each).
template <int BM, int BN, int WR, int WC, bool SYM>
__global__ __launch_bounds__(WR * WC * 64) void ns_product_kernel(Product g) {
  constexpr int NW = WR * WC;
  constexpr int TM = BM / WR / 32, TN = BN / WC / 32;   // 32 x 32 blocks of a wave
  constexpr int kSlot = (BM > BN ? BM : BN) * kBk;
  // Five places for an operand's rows of one stage.  Separate arrays, so that
  // the compiler can tell a load on its way into one from a read of another.
  __shared__ __align__(16) half_t slot0[kSlot];
  __shared__ __align__(16) half_t slot1[kSlot];
  __shared__ __align__(16) half_t slot2[kSlot];
  __shared__ __align__(16) half_t slot3[kSlot];
  __shared__ __align__(16) half_t slot4[kSlot];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int id = xcd_order(blockIdx.x, gridDim.x);
  const int mat = id / g.tiles;
  const int t = id - mat * g.tiles;
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
  const Stager<BM, NW> sp(g.p + mat * g.p_mat, g.p_ld, row0, wave, lane);
  const Stager<BN, NW> sq(g.q + mat * g.q_mat, g.q_ld, col0, wave, lane);
  const int wr = wave / WC, wc = wave - wr * WC;
  int at_p = lane_at(wr * (BM / WR), lane), at_q = lane_at(wc * (BN / WC), lane);
  f16 acc[TM][TN] = {};
  Frags<TM, TN> f0, f1;
  constexpr int kP = Stager<BM, NW>::kN, kQ = Stager<BN, NW>::kN;
  constexpr int kProducts = 2 * TM * TN, kReads = Frags<TM, TN>::kReads;
  auto past_end = [&](int k) { return k < g.kk ? k : g.kk - kBk; };   // the last stage again, never read
  // Half a stage: the products of `now`, and between them, evenly, the reads of
  // `then` and the loads of one operand.  The compiler keeps the groups apart.
  auto half = [&](const auto& loads, int n_loads, const Frags<TM, TN>& now, Frags<TM, TN>& then, const half_t* p,
                  const half_t* q, int which) {
    // Addresses are formed anew: kept over the loop for every slot they would
    // not fit the registers.
    asm volatile("" : "+v"(at_p), "+v"(at_q));
#pragma unroll
    for (int s = 0; s < n_loads; ++s) {
#pragma unroll
      for (int k = s * kProducts / n_loads; k < (s + 1) * kProducts / n_loads; ++k) {
        const int u = k / (TM * TN), i = (k - u * TM * TN) / TN, j = k % TN;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(now.a[u][i], now.b[u][j], acc[i][j], 0, 0, 0);
      }
      loads(s);
#pragma unroll
      for (int k = s * kReads / n_loads; k < (s + 1) * kReads / n_loads; ++k) then.one(p, q, at_p, at_q, which, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // One stage: P and Q rows in p0 and q0, the next stage's in p1 and q1; the
  // stage after that goes to p2 and, once every wave has read this one, p0.
  auto stage = [&](half_t* p0, half_t* q0, half_t* p1, half_t* q1, half_t* p2, int k0) {
    const int k2 = past_end(k0 + 2 * kBk);
    half([&](int s) { sp.one(p2, k2, s); }, kP, f0, f1, p0, q0, 1);
    // the next stage has arrived (all but p2's loads), and this one is read
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(kP));
    wave_barrier();
    half([&](int s) { sq.one(p0, k2, s); }, kQ, f1, f0, p1, q1, 0);
  };
  sp.all(slot0, 0);
  sq.all(slot1, 0);
  sp.all(slot2, past_end(kBk));
  sq.all(slot3, past_end(kBk));
  __builtin_amdgcn_s_waitcnt(wait_vm(kP + kQ));
  wave_barrier();
#pragma unroll
  for (int k = 0; k < kReads; ++k) f0.one(slot0, slot1, at_p, at_q, 0, k);
  for (int k0 = 0;;) {
    stage(slot0, slot1, slot2, slot3, slot4, k0);
    if ((k0 += kBk) >= g.kk) break;
    stage(slot2, slot3, slot4, slot0, slot1, k0);
    if ((k0 += kBk) >= g.kk) break;
    stage(slot4, slot0, slot1, slot2, slot3, k0);
    if ((k0 += kBk) >= g.kk) break;
    stage(slot1, slot2, slot3, slot4, slot0, k0);
    if ((k0 += kBk) >= g.kk) break;
    stage(slot3, slot4, slot0, slot1, slot2, k0);
    if ((k0 += kBk) >= g.kk) break;
  }
  __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
  wave_barrier();   // nothing is on its way into LDS any more

  // The lane's values of block (i, j): one column, rows 8*u + 4*(lane >> 5) + q.
  float alpha = g.alpha;
  if (g.scales) {
    const float f = g.scales[mat].f;
    alpha *= g.f_pow == 2 ? f * f : f;
  }
  const half_t* add = g.add ? g.add + mat * g.d_mat : nullptr;
  float gain = 0.0f;
  if (g.carry_in) {
    const half_t* c = g.p + mat * g.p_mat;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < g.m; i += NW * 64) sum += static_cast<float>(c[static_cast<int64_t>(i) * g.p_ld + i]);
    gain = block_sum_f32<NW>(sum, reinterpret_cast<float*>(slot4)) * g.alpha / (static_cast<float>(g.m) * kScaleE);
  }
  const int lr = (lane >> 5) << 2, lc = lane & 31;
  const int wrow = row0 + wr * (BM / WR), wcol = col0 + wc * (BN / WC);
  auto four = [&](int i, int j, int u) {   // four values, as the 16-bit words that are stored
    const int r = wrow + i * 32 + u * 8 + lr, c = wcol + j * 32 + lc;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = acc[i][j][u * 4 + q] * alpha;
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
    const int64_t at =
        mat * g.carry_mat + (((static_cast<int64_t>(t) * TM + i) * TN + j) * 4 + u) * (NW * 256) + threadIdx.x * 4;
    if (g.carry_in) {
      const h4 w = *reinterpret_cast<const h4*>(g.carry_in + at);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += gain * static_cast<float>(w[q]);
    }
    u16x4 o;
    if (g.out) {
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = bf16_rne(v[q]);
    } else {
      h4 h;
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = static_cast<half_t>(v[q]);
      o = __builtin_bit_cast(u16x4, h);
      if (g.carry_out) {
        h4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = static_cast<half_t>((v[q] - static_cast<float>(h[q])) * kScaleE);
        *reinterpret_cast<h4*>(g.carry_out + at) = w;
      }
    }
    return o;
  };

  // Results pass through the wave's own part of LDS, kBand blocks of rows at a
  // time, so that they leave as rows of 16-byte pieces.  A wave's LDS
  // operations are carried out in order, so no barrier is needed.
  constexpr int kBand = NW == 8 ? 1 : TM % 2 == 0 ? 2 : TM;
  constexpr int kRows = kBand * 32, kCols = TN * 32;
  static_assert(TM % kBand == 0, "whole bands");
  constexpr int kPart = kSlot / (NW / 4);
  static_assert(kRows * (kCols + 8) <= kPart && kCols * (kRows + 8) <= kPart, "a band fits the wave's part");
  uint16_t* mine = reinterpret_cast<uint16_t*>((wave & 3) == 0 ? slot0 : (wave & 3) == 1 ? slot1 : (wave & 3) == 2 ? slot2 : slot3) +
                   (wave >> 2) * kPart;
  // A tile on the diagonal of a symmetric product: only what lies below the
  // diagonal of its 32 x 32 blocks is kept, as for the tiles.
  const bool diagonal = SYM && ti == tj;
#pragma unroll
  for (int ib = 0; ib < TM; ib += kBand) {
    u16x4 o[kBand][TN][4];
#pragma unroll
    for (int i = 0; i < kBand; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[i][j][u] = four(ib + i, j, u);
    constexpr int pitch = kCols + 8;
#pragma unroll
    for (int i = 0; i < kBand; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int q = 0; q < 4; ++q) mine[(i * 32 + u * 8 + lr + q) * pitch + j * 32 + lc] = o[i][j][u][q];
    if (diagonal) {
#pragma unroll
      for (int i = 0; i < kBand; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (wrow + (ib + i) * 32 == wcol + j * 32) {   // a block on the diagonal: its upper half from the lower
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const int r = (u >> 2) * 8 + lr + (u & 3);
              const uint16_t low = mine[(i * 32 + lc) * pitch + j * 32 + r];
              if (r < lc) mine[(i * 32 + r) * pitch + j * 32 + lc] = low;
            }
          }
    }
#pragma unroll
    for (int k = 0; k < kRows * kCols / 512; ++k) {
      const int at = k * 64 + lane;
      const int lrow = at / (kCols / 8), lcol = (at - lrow * (kCols / 8)) * 8;
      const int r = wrow + ib * 32 + lrow, c = wcol + lcol;
      const u32x4 piece = *reinterpret_cast<const u32x4*>(mine + lrow * pitch + lcol);
      if (r >= g.m || (diagonal && (c >> 5) > (r >> 5))) continue;
      if (!g.out) {
        if (c < g.d_ld) *reinterpret_cast<u32x4*>(g.d + mat * g.d_mat + static_cast<int64_t>(r) * g.d_ld + c) = piece;
      } else {
        uint16_t* dst = g.out + mat * g.out_mat + static_cast<int64_t>(r) * g.out_row + c;
        if (g.out_vec && c + 8 <= g.n) {
          *reinterpret_cast<u32x4*>(dst) = piece;
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (c + q < g.n) dst[q] = static_cast<uint16_t>(piece[q >> 1] >> ((q & 1) * 16));
        }
      }
    }
    if (g.dt) {
      constexpr int turned = kRows + 8;
#pragma unroll
      for (int i = 0; i < kBand; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<u16x4*>(mine + (j * 32 + lc) * turned + i * 32 + u * 8 + lr) = o[i][j][u];
#pragma unroll
      for (int k = 0; k < kRows * kCols / 512; ++k) {
        const int at = k * 64 + lane;
        const int lcol = at / (kRows / 8), lrow = (at - lcol * (kRows / 8)) * 8;
        const int c = wcol + lcol, r = wrow + ib * 32 + lrow;
        const u32x4 piece = *reinterpret_cast<const u32x4*>(mine + lcol * turned + lrow);
        if (c < g.n && r < g.dt_ld && !(diagonal && (c >> 5) >= (r >> 5)))
          *reinterpret_cast<u32x4*>(g.dt + mat * g.dt_mat + static_cast<int64_t>(c) * g.dt_ld + r) = piece;
      }
    }
  }
  // The padding past the last tile, as zeros.
  if (g.d && col0 + BN >= g.n)
    for (int c = col0 + BN + lane; c < g.d_ld; c += 64)
      for (int r = row0 + wave; r < g.m && r < row0 + BM; r += NW)
        g.d[mat * g.d_mat + static_cast<int64_t>(r) * g.d_ld + c] = 0;
  if (g.dt && row0 + BM >= g.m)
    for (int r = row0 + BM + lane; r < g.dt_ld; r += 64)
      for (int c = col0 + wave; c < g.n && c < col0 + BN; c += NW)
        g.dt[mat * g.dt_mat + static_cast<int64_t>(c) * g.dt_ld + r] = 0;
}

// ------------------------------------------------------------------ launches
template <int BM, int BN, int WR, int WC, bool SYM>
hipError_t product_tiles(Product g, int64_t mats, hipStream_t s) {
  const int tm = (g.m + BM - 1) / BM;
  g.tiles_n = (g.n + BN - 1) / BN;
  g.tiles = SYM ? tm * (tm + 1) / 2 : tm * g.tiles_n;
  hipLaunchKernelGGL((ns_product_kernel<BM, BN, WR, WC, SYM>), dim3(static_cast<unsigned>(g.tiles * mats)),
                     dim3(WR * WC * 64), 0, s, g);
  return hipGetLastError();
}

// The tile for a product, by its modelled time: rounds of one tile per CU, each
// of the time measured for a summed index of 4096 (256 CUs busy) and a fixed
// part.  256: 115 us; 192 (symmetric only): 72; 128: 38; 64: 16.  A symmetric
// 4096 x 4096 product has 253 tiles of 192 (72 us) against 136 of 256 (110), a
// full one 256 of 256 (115) against 1024 of 128 (150).
template <bool SYM>
hipError_t product(const Product& g, int64_t mats, hipStream_t s) {
  auto time = [&](int side, double us) {
    const int64_t tm = (g.m + side - 1) / side, tn = (g.n + side - 1) / side;
    const int64_t tiles = (SYM ? tm * (tm + 1) / 2 : tm * tn) * mats;
    return static_cast<double>((tiles + 255) / 256) * (us * g.kk / 4096.0 + 4.0);
  };
  const double t256 = time(256, 115.0), t192 = SYM ? time(192, 72.0) : t256, t128 = time(128, 38.0), t64 = time(64, 16.0);
  const double best = fmin(fmin(t256, t192), fmin(t128, t64));
  if (t256 == best) return product_tiles<256, 256, 2, 4, SYM>(g, mats, s);
  if (t192 == best) return product_tiles<192, 192, 2, 2, true>(g, mats, s);
  if (t128 == best) return product_tiles<128, 128, 2, 2, SYM>(g, mats, s);
  return product_tiles<64, 64, 2, 2, SYM>(g, mats, s);
}

// The workspace: partial sums and factors, two turns of X^T and one X, three
// k x k matrices, each for all matrices.
struct Layout {
  int64_t k, l, kp, lp;
  int64_t e_mat;                                   // rounding errors of one matrix: whole tiles
  int64_t partials, scales, x, xt[2], sq[3], e, bytes;  // byte offsets
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
    scales = take(mats * static_cast<int64_t>(sizeof(NsScale)));
    x = take(mats * k * lp * 2);
    for (int64_t& o : xt) o = take(mats * l * kp * 2);
    for (int64_t& o : sq) o = take(mats * k * kp * 2);
    e_mat = (k + kTile - 1) / kTile * kTile * ((l + kTile - 1) / kTile * kTile);
    e = take(mats * e_mat * 2);
    bytes = at + kTile * (lp > kp ? lp : kp) * 2;   // rows that the last tiles read past their matrix
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
  NsScale* scales = reinterpret_cast<NsScale*>(ws + w.scales);
  half_t* e = reinterpret_cast<half_t*>(ws + w.e);
  const int64_t x_mat = w.k * w.lp, xt_mat = w.l * w.kp, sq_mat = w.k * w.kp;

  NsInput in{p.in, p.in_row, p.in_mat, static_cast<int>(p.rows), static_cast<int>(p.cols), p.in_f32, 0};
  const int64_t per16 = p.in_f32 ? 4 : 8;
  in.vec = (reinterpret_cast<uintptr_t>(p.in) & 15u) == 0 && p.in_row % per16 == 0 && p.in_mat % per16 == 0;
  double* partials = reinterpret_cast<double*>(ws + w.partials);
  const int64_t rows4 = (p.rows + kNormThreads / 64 - 1) / (kNormThreads / 64);
  const int parts = static_cast<int>(rows4 < kNormParts ? rows4 : kNormParts);
  hipLaunchKernelGGL(ns_norm_kernel, dim3(parts, static_cast<unsigned>(p.mats)), dim3(kNormThreads), 0, s, in, partials);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(ns_scale_kernel, dim3(static_cast<unsigned>(p.mats)), dim3(kNormThreads), 0, s, partials, parts, scales);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  NsX nx;
  nx.same = tall ? xt[0] : x;
  nx.turned = tall ? x : xt[0];
  nx.same_mat = tall ? xt_mat : x_mat;
  nx.turned_mat = tall ? x_mat : xt_mat;
  nx.scales = scales;
  hipLaunchKernelGGL(ns_prepare_kernel,
                     dim3(static_cast<unsigned>(pad_up(p.cols) / kTurn), static_cast<unsigned>(pad_up(p.rows) / kTurn),
                          static_cast<unsigned>(p.mats)),
                     dim3(kNormThreads), 0, s, in, nx);
  err = hipGetLastError();
  if (err != hipSuccess) return err;

  // k x k product u v^T into d, symmetric or not
  auto square = [&](bool sym, const half_t* u, const half_t* v, half_t* d, float alpha, const half_t* add, float beta,
                    float diag) {
    Product g = {};
    g.p = u;
    g.q = v;
    g.p_mat = g.q_mat = g.d_mat = g.dt_mat = sq_mat;
    g.p_ld = g.q_ld = g.d_ld = g.dt_ld = kp;
    g.m = g.n = k;
    g.kk = kp;
    g.d = d;
    g.dt = sym ? d : nullptr;
    g.alpha = alpha;
    g.add = add;
    g.beta = beta;
    g.diag = diag;
    return sym ? product<true>(g, p.mats, s) : product<false>(g, p.mats, s);
  };
  auto poly = [&](const half_t* a, half_t* d, int t) {
    const float* c = p.coefs + 3 * t;
    return square(true, a, a, d, c[2] * (kScaleC / (kScaleA * kScaleA)), a, c[1] * (kScaleC / kScaleA), c[0] * kScaleC);
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
    g.scales = first ? scales : nullptr;
    g.f_pow = 2;
    return product<true>(g, p.mats, s);
  };
  // X = C X from the transposed copy xt[from]: into x and xt[to], the last
  // step's into the output.
  enum { kCarryOut = 1, kCarryIn = 2 };
  auto apply = [&](const half_t* c, float c_scale, int from, bool first, int to, bool last, int carry) {
    Product g = {};
    g.scales = first ? scales : nullptr;
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
