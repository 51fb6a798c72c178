// gfx950 kernels of zero_ffn_forward and zero_ffn_backward: a layer's gated
// feed-forward block on T tokens, D wide, F hidden,
//   forward    g = x Wg^T, u = x Wu^T, h = act(g) * u      one product kernel
//              y = h Wd^T                                   another
//   backward   dh = dy Wd, dg = dh u act'(g), du = dh act(g), h again: one
//              dx = dg Wg + du Wu                           another (one long sum)
//              dWg = dg^T x, dWu = du^T x, dWd = dy^T h     one launch for the three
// with x, g and u of the backward pass read from 8-bit checkpoints: g and u in the
// product's epilogue (2 bytes where BF16 needs 4, and no pass of its own), x once into
// BF16 values, which the two products' tiles then read 2 F / 256 times.
//
// Every product is out[q][p] = sum_k P[p][k] Q[q][k], out's rows contiguous along p.  An
// operand's rows are contiguous along k ("rows") or lie along k ("columns": the
// weights in backward, both operands of the weights' gradients), and then come from
// LDS with transposing reads: nothing is turned in memory.
// Operands are BF16, sums FP32 on the matrix cores.  h, dg and du are rounded to BF16,
// the type in which the next product takes them: that moves y, dx and the gradients by
// about as much as their own rounding (2^-9 of a value, on average less).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <numeric>
#include <type_traits>

#include "act8.h"
#include "kernels.h"

#pragma clang fp contract(off)

namespace zero {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBk = 64;        // summed index per stage: rows of 128 bytes in LDS
constexpr int kPad = 64;       // pitches of the workspace's matrices are multiples of this
constexpr int kRawFlags = 0x00020000;

__host__ __device__ inline int64_t pad_up(int64_t n) { return (n + kPad - 1) / kPad * kPad; }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), b2));
}

// ------------------------------------------------------------------ staging
// Columns [k0, k0 + 64) of R rows of an operand into LDS, as R rows of 128 bytes; the
// 16-byte piece c of row r lies at piece c ^ ((r >> 1) & 7), so that the pieces c
// of any 16 consecutive rows fall into different banks (two rows fill the 64 banks
// once).  Each wave moves 8 rows per instruction, straight to LDS.  Rows past the
// matrix's end read as zeros: the descriptor ends with the matrix.
template <int R, int NW>
struct RowStager {
  static constexpr int kN = R / 8 / NW;   // instructions of a wave
  static_assert(kN * 8 * NW == R, "every wave moves the same number of rows");
  uint16_t* base;
  int voff[kN], wave, bytes;   // bytes: from base on, 0 where the wave has no rows
  // first: the matrix's row that is this wave's first; rows: how many it has from there on.
  __device__ __forceinline__ RowStager(const uint16_t* m, int64_t ld, int64_t first, int64_t rows, int kk, int wave_, int lane)
      : wave(wave_) {
    const int64_t most = kN * 8;
    const int64_t n = rows < most ? rows : most;
    base = const_cast<uint16_t*>(m + (rows > 0 ? first : 0) * ld);
    bytes = rows > 0 ? static_cast<int>(((n - 1) * ld + kk) * 2) : 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = i * 8 + (lane >> 3);   // kN * 8 is a multiple of 16: the wave's first row shifts no piece
      voff[i] = r * static_cast<int>(ld) * 2 + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
    static_assert(kN % 2 == 0, "see voff");
  }
  // A stage past the end is loaded too, so that the loads on their way can be
  // counted, but from nowhere.
  // end: bytes, or 0 for a stage past the end; at: bytes from a row's first column on
  __device__ __forceinline__ void one(uint16_t* lds, int end, int at, int i) const {
#ifdef __HIP_DEVICE_COMPILE__   // the builtin is unknown to the host pass
    __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(base, 0, end, kRawFlags),
                                             (lds_void*)(lds + (wave * kN + i) * 8 * kBk), 16, voff[i], at, 0, 0);
#endif
  }
};

// Rows [k0, k0 + 64) and columns [col0, col0 + C) of an operand whose rows lie along
// k: 64 rows of 2 C bytes, from which transposing reads take the columns.  Those
// read 32 bytes of rows r, r + 1, r + 2, r + 3 and 8 rows on together (r a multiple of 16, or 4 more):
// the 32-byte piece c of row r lies at piece c ^ column_turn(r).  Rows past `end` read as zeros (the descriptor ends there), columns
// past a row's end as the next row's: their results are dropped.
__device__ __forceinline__ int column_turn(int r) { return (r & 3) * 2 + ((r >> 3) & 1); }
template <int C, int NW>
struct ColumnStager {
  static constexpr int kRows = 512 / C, kN = 64 / kRows / NW;   // rows of one instruction, instructions of a wave
  static_assert(C >= 128 && kN * kRows * NW == 64, "every wave moves the same number of pieces");
  int voff[kN], wave;
  __device__ __forceinline__ ColumnStager(int64_t ld, int wave_, int lane) : wave(wave_) {
    const int row = lane / (64 / kRows), piece = lane % (64 / kRows);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = (wave * kN + i) * kRows + row;
      voff[i] = r * static_cast<int>(ld) * 2 + (((piece >> 1) ^ column_turn(r)) << 5) + (piece & 1) * 16;
    }
  }
  __device__ __forceinline__ void one(uint16_t* lds, __amdgpu_buffer_rsrc_t rsrc, int i) const {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (wave * kN + i) * 512), 16, voff[i], 0, 0, 0);
#endif
  }
};
// The rows of a stage: `at` is the first one's first column of the tile, `left` rows are there
// from it on (none or less: nothing is read), `width` values from that column on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t column_rows(const uint16_t* at, int left, int64_t ld, int width) {
  const int rows = left < kBk ? left : kBk;
  const int bytes = ((rows - 1) * static_cast<int>(ld) + width) * 2;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(at), 0, left > 0 ? bytes : 0, kRawFlags);
}

// Byte offset in a slot of the lane's fragment piece in the first half of a stage: row first +
// (lane & 15), piece lane >> 4, moved as RowStager moves it.  The second half's is at
// the offset with bit 6 flipped.
__device__ __forceinline__ int lane_at_row(int first, int lane) {
  return (first + (lane & 15)) * kBk * 2 + (((lane >> 4) ^ ((lane >> 1) & 7)) << 4);
}
// What the lane points a transposing read at: row 8 * (lane >> 4) + ((lane >> 2) & 3),
// columns first + 4 * (lane & 3).  4 rows on, column_turn is the same.
template <int C>
__device__ __forceinline__ int lane_at_column(int first, int lane) {
  const int row = (lane >> 4) * 8 + ((lane >> 2) & 3);
  return row * C * 2 + (((first >> 4) ^ column_turn(row)) << 5) + (lane & 3) * 8;
}

// 4 values down a column, twice: the transposing LDS read hands lane j of 16 the
// component j % 4 of the lanes j / 4 + 4 q, so each lane points at four columns of
// one row and lane j gets column j of four rows.
__device__ __forceinline__ b8 transpose8(const void* at, const void* at4) {
  b8 v = {};
#ifdef __HIP_DEVICE_COMPILE__
  typedef short s4 __attribute__((ext_vector_type(4)));
  typedef short s8 __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s4 lds_s4;
  const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at);
  const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at4);
  v = __builtin_bit_cast(b8, s8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
#endif
  return v;
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

// ------------------------------------------------------------------ activations
constexpr float kGeluIn = 0.7978845608028654f, kGeluCube = 0.044715f;   // sqrt(2 / pi)

// sigma(x) = 1 / (1 + e^-x): 0 and 1 where e^-x overflows or vanishes.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// tanh's GELU is x sigma(2 k (x + c x^3)); past 16 sigma is 0 or 1, and the cube stays finite.
__device__ __forceinline__ float gelu_inner(float x) {
  const float z = x < -16.0f ? -16.0f : x > 16.0f ? 16.0f : x;
  return 2.0f * kGeluIn * z * (1.0f + kGeluCube * z * z);
}

template <int ACT>
__device__ __forceinline__ float activate(float g) {
  if (ACT == ZERO_FFN_SILU) return g * sigmoid(g);
  if (ACT == ZERO_FFN_GELU) return g * sigmoid(gelu_inner(g));
  return g < 0.0f ? 0.0f : g;   // NaN stays
}

// act(g) and its derivative (0 at ReLU's corner).
template <int ACT>
__device__ __forceinline__ void activate_slope(float g, float& a, float& slope) {
  if (ACT == ZERO_FFN_RELU) {
    a = g < 0.0f ? 0.0f : g;
    slope = g > 0.0f ? 1.0f : g <= 0.0f ? 0.0f : g;
    return;
  }
  const float s = sigmoid(ACT == ZERO_FFN_SILU ? g : gelu_inner(g));
  a = g * s;
  if (ACT == ZERO_FFN_SILU) {
    slope = s + a * (1.0f - s);
  } else {
    const float z = g < -16.0f ? -16.0f : g > 16.0f ? 16.0f : g;   // sigma' is 0 there
    slope = s + z * s * (1.0f - s) * (2.0f * kGeluIn) * (1.0f + 3.0f * kGeluCube * z * z);
  }
}

// ------------------------------------------------------------------ products
enum Epilogue {
  kStore,      // out = the sums
  kPartial,    // the FP32 sums of a part of the summed index, for ffn_join_kernel
  kGated,      // P is gate's and up's rows in turn: out = act(g) * u, and both into checkpoints
  kSlopes,     // sums are dh: dg, du and h from the checkpoints of g and u
};

struct Act8Rows {   // a checkpoint of a matrix
  uint8_t* codes;
  uint8_t* scales;
};

struct Product {
  const uint16_t* p;
  const uint16_t* p2;      // kGated: up's rows.  Columns: P of the summed index from `turn` on
  const uint16_t* q;
  int64_t p_ld, q_ld;
  int np, nq, kk;          // results: nq rows of np
  int turn;                // columns: summed index (a multiple of kBk) where p2 takes over; its own starts at 0
  int p_end, q_end;        // columns: rows of p (and p2), of q
  int p_cols, q_cols;      // columns: values of a row that may be read
  int tiles_p, tiles_q;
  uint16_t* out;
  int64_t out_ld;
  int out_cols;            // columns that are written: np, or the pitch, with zeros
};

struct JoinArgs {
  const float* partial;
  int64_t pitch;
  int splits, nq, np;
  uint16_t* out;
  int64_t out_ld;
};

struct Products {
  Product of[3];
  int tiles;               // workgroups of tiles; those behind them do the side work
  int64_t side;            // its pieces, one a thread: of x (kGated: saved, kSlopes: loaded) or of a join (columns of Q)
  Act8Params x;
  JoinArgs join;
  int first[3];            // tile number of each; those past the last have 0x7FFFFFFF
  int begin, quarters;     // the first tile of the launch; whether its workgroups take quarters of tiles
  // kGated and kSlopes
  Act8Rows gate, up;
  uint16_t* du;            // kSlopes: out is dg, both with out_ld
  uint16_t* h;
  int64_t h_ld;
  int blocks;              // scales of a row
  int format, act, save;
  int rows;                // of a workgroup, with a few tokens (`tiles` workgroups have them)
  int alike;               // rows whose sums begin at the same turn, a multiple of `rows`
  int spread;              // rows: whether each tile of P begins at another stage
  int splits, chunk;       // kPartial: parts of the summed index and their length, a multiple of 2 kBk
  float* partial;          // kPartial: [splits][nq][pitch]
  int64_t pitch;
};

constexpr int kGroup = 4;  // tiles of q that one XCD's neighbours share (2, 4 and 8 within 1%, 16 2% slower)

// The first n of 8 values to memory, at any alignment: the memory takes whole pieces as they lie
// (one by one they cost the gradients of 777 x 1301 from 1001 tokens 20 us instead of 13).
__device__ __forceinline__ void store8(uint16_t* dst, const float (&v)[8], int n) {
  const u32x4 w = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
  if (n >= 8) {
    __builtin_memcpy(dst, &w, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) dst[q] = static_cast<uint16_t>(w[q >> 1] >> ((q & 1) * 16));
  }
}

__device__ __forceinline__ void store_codes8(uint8_t* dst, u32x2 w, int n) {
  if (n >= 8) {
    __builtin_memcpy(dst, &w, 8);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) dst[q] = static_cast<uint8_t>(w[q >> 2] >> ((q & 3) * 8));
  }
}
__device__ __forceinline__ u32x2 load_codes8(const uint8_t* src, int n) {
  u32x2 w = {};
  if (n >= 8) {
    __builtin_memcpy(&w, src, 8);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) w[q >> 2] |= static_cast<uint32_t>(src[q]) << ((q & 3) * 8);
  }
  return w;
}

// The first N <= 4 of n bytes, zeros past their end.
template <int N>
__device__ __forceinline__ uint32_t load_bytes(const uint8_t* src, int n) {
  uint32_t w = 0;
  if (n >= N) {
    __builtin_memcpy(&w, src, N);
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (q < n) w |= static_cast<uint32_t>(src[q]) << (8 * q);
  }
  return w;
}

// Two blocks' sums one after the other along p, as the matrix cores leave them: lane l has
// column q = l & 15 and rows p = 4 * (l >> 4) + 0..3 of each.  After the exchange of
// lanes 16 to 31 and 48 to 63 of the first for 0 to 15 and 32 to 47 of the second it has
// 8 neighbours along p, octet_at(lane) + 0..7 of the 32.
__device__ __forceinline__ int octet_at(int lane) { return ((lane >> 4) & 1) * 16 + (lane >> 5) * 8; }
__device__ __forceinline__ void octet(const f4& lo, const f4& hi, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t a = __float_as_uint(lo[q]), b = __float_as_uint(hi[q]);
#ifdef __HIP_DEVICE_COMPILE__
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
#endif
    v[q] = __uint_as_float(a);
    v[4 + q] = __uint_as_float(b);
  }
}

// The largest magnitude of 8 values, as a whole number (NaN is above infinity), and the largest of
// lanes l, l ^ 16, l ^ 32 and l ^ 48.
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const uint32_t m = __float_as_uint(x[n]) & 0x7FFFFFFFu;
    top = m > top ? m : top;
  }
  return top;
}
__device__ __forceinline__ uint32_t across_groups(uint32_t top) {
#ifdef __HIP_DEVICE_COMPILE__
  const auto a = __builtin_amdgcn_permlane16_swap(top, top, false, false);
  top = a[0] > a[1] ? a[0] : a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(top, top, false, false);
  top = b[0] > b[1] ? b[0] : b[1];
#endif
  return top;
}

// ------------------------------------------------------------------ side work
// Small streaming work that the products around it do not wait for goes behind the tiles of a
// launch, where a launch of its own would take 3 to 5 us: x into its checkpoint (beside gate
// and up), x's values from it (beside dh), dx's parts added up (beside the weights' gradients):
// 256 x 512 x 1408 forward with its checkpoint 32.5 -> 29.9 us, backward 44 -> 37.
// Piece k is 8 neighbours of a row.
constexpr int64_t kSideMost = 1 << 18;   // pieces; more have a launch that fills the card (8192 x 4096: 20 us)
__host__ __device__ inline int64_t pieces_of(const Act8Params& a) {   // whole blocks of four
  return a.rows * ((a.cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK * 4);
}
// 8 values from `at` on, of which n are there; any alignment.
__device__ __forceinline__ b8 load_piece(const uint16_t* at, int n) {
  u32x4 w = {};
  if (n >= 8) {
    __builtin_memcpy(&w, at, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) w[q >> 1] |= static_cast<uint32_t>(at[q]) << ((q & 1) * 16);
  }
  return __builtin_bit_cast(b8, w);
}

__device__ __forceinline__ void save_piece(const Act8Params& a, int k) {
  const int blocks = static_cast<int>((a.cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK), row = k / (blocks * 4);
  const int piece = k - row * blocks * 4, n = static_cast<int>(a.cols) - piece * 8;
  const bool there = k < pieces_of(a);
  b8 w = {};
  if (there && n > 0) w = load_piece(static_cast<const uint16_t*>(a.values) + row * a.row + piece * 8, n);
  float v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = static_cast<float>(w[q]);
  uint32_t top = top_of(v);
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    const uint32_t m = __shfl_xor(top, off, 64);
    top = m > top ? m : top;
  }
  if (!there) return;
  const uint32_t byte = act8_scale_byte(top, a.format);
  uint32_t codes[2];
  act8_codes(v, act8_inverse(byte), a.format, codes);
  store_codes8(a.codes + row * a.cols + piece * 8, u32x2{codes[0], codes[1]}, n);
  if ((piece & 3) == 0) a.scales[static_cast<int64_t>(row) * blocks + piece / 4] = static_cast<uint8_t>(byte);
}
__device__ __forceinline__ void read_piece(const Act8Params& a, int k) {
  const int blocks = static_cast<int>((a.cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK), row = k / (blocks * 4);
  const int piece = k - row * blocks * 4, n = static_cast<int>(a.cols) - piece * 8;
  if (k >= pieces_of(a) || n <= 0) return;
  const u32x2 w = load_codes8(a.codes + row * a.cols + piece * 8, n);
  const float scale = act8_scale(a.scales[static_cast<int64_t>(row) * blocks + piece / 4]);
  const uint32_t words[2] = {w.x, w.y};
  float v[8];
  if (a.format == ZERO_ACT8_INT8)
    act8_numbers_int8(words, v);
  else
    act8_numbers_e4m3(words, v);
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] *= scale;   // exact
  store8(static_cast<uint16_t*>(a.values) + row * a.row + piece * 8, v, n);
}
__device__ __forceinline__ void join_piece(const JoinArgs& a, int64_t k) {
  const int64_t pieces = a.pitch / 8, n = a.nq * pieces;
  if (k >= n) return;
  const int64_t q = k / pieces;
  const int p = static_cast<int>(k - q * pieces) * 8;
  f4 lo = {}, hi = {};
  for (int s = 0; s < a.splits; ++s) {
    const f4* from = reinterpret_cast<const f4*>(a.partial + (s * static_cast<int64_t>(a.nq) + q) * a.pitch + p);
    lo += from[0];
    hi += from[1];
  }
  const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  store8(a.out + q * a.out_ld + p, v, a.np - p);
}

// A tile of BP x BQ results by WP x WQ waves.  ACT: of kGated and kSlopes.  Bound by the matrix
// units, whose clock falls as they fill.  Measured, 8192 x 4096 x 14336 with tiles of 256 x 256, medians
// of 40 passes in a row: gate and up, saved, 1381 us (1393 TFLOP/s, matrix units 77% busy), y 645 (1492,
// 85%), dh 917 (1050, 59%: the epilogue moves 0.95 GB while they wait, since all CUs come to it
// together), dx 1289 (1493, 81%), the weights' gradients 1961 and 145 for the quarters (1370, 77%).  On
// another card 1488, 695, 928, 1292 and 2004.
template <int BP, int BQ, int WP, int WQ, int SLOTS, bool PCOL, bool QCOL, Epilogue EPI, int ACT>
__global__ __launch_bounds__(WP * WQ * 64) void ffn_product_kernel(Products args) {
  constexpr int NW = WP * WQ;
  constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;   // 16 x 16 blocks of a wave
  static_assert(TP % 2 == 0 && (EPI != kGated || (!PCOL && TP % 4 == 0)), "gate's and up's blocks of a wave are side by side");
  // SLOTS places for each operand's part of one stage.  Separate arrays, so that the
  // compiler can tell a load on its way into one from a read of another.
  static_assert(SLOTS == 2 || SLOTS == 4, "see the loop");
  constexpr bool MORE = SLOTS == 4;
  __shared__ __align__(16) uint16_t pslot0[BP * kBk];
  __shared__ __align__(16) uint16_t pslot1[BP * kBk];
  __shared__ __align__(16) uint16_t pslot2[MORE ? BP * kBk : 1];
  __shared__ __align__(16) uint16_t pslot3[MORE ? BP * kBk : 1];
  __shared__ __align__(16) uint16_t qslot0[BQ * kBk];
  __shared__ __align__(16) uint16_t qslot1[BQ * kBk];
  __shared__ __align__(16) uint16_t qslot2[MORE ? BQ * kBk : 1];
  __shared__ __align__(16) uint16_t qslot3[MORE ? BQ * kBk : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if constexpr (EPI == kGated || EPI == kSlopes || QCOL) {
    if (static_cast<int>(blockIdx.x) >= args.tiles) {
      const int k = (blockIdx.x - args.tiles) * (NW * 64) + threadIdx.x;
      if constexpr (EPI == kGated)
        save_piece(args.x, k);
      else if constexpr (EPI == kSlopes)
        read_piece(args.x, k);
      else
        join_piece(args.join, k);
      return;
    }
  }
  int id = xcd_order(blockIdx.x, args.tiles);
  const int split = EPI == kPartial ? id % args.splits : 0;
  if constexpr (EPI == kPartial) id /= args.splits;
  // One of the four quarters of a larger tile, or a tile.
  const int quarter = args.quarters ? id & 3 : 0;
  id = args.begin + (args.quarters ? id >> 2 : id);
  const int which = id >= args.first[2] ? 2 : id >= args.first[1] ? 1 : 0;
  const Product& g = args.of[which];
  const int t = id - args.first[which];
  // Groups of kGroup tiles of q: an XCD's 32 workgroups share their operands' rows.
  const int group = t / (kGroup * g.tiles_p), in = t - group * kGroup * g.tiles_p;
  const int left = g.tiles_q - group * kGroup, height = left < kGroup ? left : kGroup;
  int tp = in / height, tq = group * kGroup + in - tp * height;
  if (args.quarters) {
    tp = 2 * tp + (quarter & 1);
    tq = 2 * tq + (quarter >> 1);
  }
  const int wp = wave / WQ, wq = wave - wp * WQ;

  const int k_first = EPI == kPartial ? split * args.chunk : 0;
  const int kk = EPI == kPartial && g.kk - k_first > args.chunk ? args.chunk : g.kk - k_first;
  constexpr int kOwn = EPI == kGated ? BP / 2 : BP;   // values along p of a tile
  const int p0 = tp * kOwn, q0 = tq * BQ;
  if (p0 >= g.out_cols || q0 >= g.nq) return;   // a quarter past the edge
  using PStager = std::conditional_t<PCOL, ColumnStager<BP, NW>, RowStager<BP, NW>>;
  using QStager = std::conditional_t<QCOL, ColumnStager<BQ, NW>, RowStager<BQ, NW>>;
  auto p_stager = [&] {
    if constexpr (PCOL) {
      return PStager(g.p_ld, wave, lane);
    } else {
      constexpr int kMine = PStager::kN * 8;   // rows of a wave
      const int row = wave * kMine;
      if constexpr (EPI == kGated) {
        // LDS rows of wave row wp: half of them gate's, half up's
        constexpr int kHalf = BP / WP / 2;
        static_assert(kHalf % kMine == 0, "a wave stages rows of one of them");
        const int first = p0 + row / (2 * kHalf) * kHalf + row % kHalf;
        return PStager(row / kHalf % 2 ? g.p2 : g.p, g.p_ld, first, g.np - first, kk, wave, lane);
      } else {
        return PStager(g.p + k_first, g.p_ld, p0 + row, g.np - p0 - row, kk, wave, lane);
      }
    }
  };
  auto q_stager = [&] {
    if constexpr (QCOL) {
      return QStager(g.q_ld, wave, lane);
    } else {
      const int row = wave * QStager::kN * 8;
      return QStager(g.q + k_first, g.q_ld, q0 + row, g.nq - q0 - row, kk, wave, lane);
    }
  };
  const PStager sp = p_stager();
  const QStager sq = q_stager();
  constexpr int kP = PStager::kN, kQ = QStager::kN;
  // Where the stage to load next comes from; next_p and next_q go on to it.
  const bool past_turn = PCOL && k_first >= g.turn;   // a part that starts in p2
  const int p_first = past_turn ? k_first - g.turn : k_first;
  const uint16_t* const p2_at = g.p2 + p0;
  const uint16_t* p_at = (past_turn ? p2_at : g.p + p0) + (PCOL ? p_first * g.p_ld : 0);
  const uint16_t* q_at = g.q + q0;
  const int p_rows = g.p_end, p_ld = static_cast<int>(g.p_ld), q_ld = static_cast<int>(g.q_ld);
  const int p_width = g.p_cols - p0, q_width = g.q_cols - q0;
  int p_left = p_rows - p_first, q_left = g.q_end, p_turn = past_turn ? -kBk : g.turn - k_first, p_byte = 0, q_byte = 0, p_end = 0, q_end = 0;
  // Rows: stages still to load (kk is whole stages), and where the next begins.
  const int stages = QCOL ? 0 : kk / kBk;
  int p_n = stages, q_n = stages, p_k = !PCOL && args.spread ? tp % stages * kBk : 0, q_k = p_k;
  __amdgpu_buffer_rsrc_t p_from, q_from;
  auto next_p = [&] {
    if constexpr (PCOL) {
      const bool turn = p_turn == 0;
      p_at = turn ? p2_at : p_at;
      p_left = turn ? p_rows : p_left;
      p_from = column_rows(p_at, p_left, p_ld, p_width);
      p_at += kBk * static_cast<int64_t>(p_ld);
      p_left -= kBk;
      p_turn -= kBk;
    } else {
      p_end = p_n > 0 ? sp.bytes : 0;
      p_byte = p_end ? p_k * 2 : 0;
      --p_n;
      p_k = p_k + kBk < kk ? p_k + kBk : 0;
    }
  };
  auto next_q = [&] {
    if constexpr (QCOL) {
      q_from = column_rows(q_at, q_left, q_ld, q_width);
      q_at += kBk * static_cast<int64_t>(q_ld);
      q_left -= kBk;
    } else {
      q_end = q_n > 0 ? sq.bytes : 0;
      q_byte = q_end ? q_k * 2 : 0;
      --q_n;
      q_k = q_k + kBk < kk ? q_k + kBk : 0;
    }
  };
  auto load_p = [&](uint16_t* lds, int i) {
    if constexpr (PCOL)
      sp.one(lds, p_from, i);
    else
      sp.one(lds, p_end, p_byte, i);
  };
  auto load_q = [&](uint16_t* lds, int i) {
    if constexpr (QCOL)
      sq.one(lds, q_from, i);
    else
      sq.one(lds, q_end, q_byte, i);
  };

  int at_p = PCOL ? lane_at_column<BP>(wp * (BP / WP), lane) : lane_at_row(wp * (BP / WP), lane);
  int at_q = QCOL ? lane_at_column<BQ>(wq * (BQ / WQ), lane) : lane_at_row(wq * (BQ / WQ), lane);
  auto read_p = [&](const uint16_t* ps, int half, int i) {
    if constexpr (PCOL) {
      const char* at = reinterpret_cast<const char*>(ps) + (at_p ^ (i << 5)) + half * 32 * BP * 2;
      return transpose8(at, at + 4 * BP * 2);
    } else {
      return *reinterpret_cast<const b8*>(reinterpret_cast<const char*>(ps) + (at_p ^ (half * 64)) + i * 16 * kBk * 2);
    }
  };
  auto read_q = [&](const uint16_t* qs, int half, int j) {
    if constexpr (QCOL) {
      const char* at = reinterpret_cast<const char*>(qs) + (at_q ^ (j << 5)) + half * 32 * BQ * 2;
      return transpose8(at, at + 4 * BQ * 2);
    } else {
      return *reinterpret_cast<const b8*>(reinterpret_cast<const char*>(qs) + (at_q ^ (half * 64)) + j * 16 * kBk * 2);
    }
  };

  // A stage is 2 TP steps: step s multiplies P's block s % TP by the TQ blocks of Q, both
  // in half s / TP of the stage.  P's blocks are read two steps ahead (four places), Q's
  // during the half before.  So Q's slot is free, and its next one needed, half-way; P's two
  // steps before the end: a barrier at each, and from there on the loads of the stage
  // SLOTS on into the free slot, a few per step (a wave issues in order: loads in a row
  // hold its products up).  With two slots each load has between half a stage and a whole one to
  // arrive.  Tiles of 128 x 128, two on a CU, gain nothing from four: a CU takes in 55 to 95
  // bytes/ns, and a stage of 32 KiB takes the 0.46 us that says.  Few tiles of 128 x 64, alone on their
  // CU, do: dh's product of 1001 x 1301 x 777 takes 12.7 us with four, 16.5 with two.
  constexpr int kSteps = 2 * TP, kQSpan = TP - 2, kPSpan = TP;   // steps with loads
  static_assert(kSteps % 4 == 0, "a stage starts with the first place");
  f4 acc[TP][TQ] = {};
  b8 fp[4], fq[2][TQ];
  // The stage in ps0 and qs0; the next in ps1 and qs1; the one before was in psp.
  auto stage = [&](uint16_t* ps0, uint16_t* qs0, uint16_t* ps1, uint16_t* qs1, uint16_t* psp) {
    // Addresses are formed anew: kept over the loop for every slot they would
    // not fit the registers.
    asm volatile("" : "+v"(at_p), "+v"(at_q));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s == TP) {   // Q's next stage has arrived (all but the loads after its own), and this one's is read
        __builtin_amdgcn_s_waitcnt(wait_vm_lds((SLOTS - 1) * kP + (SLOTS - 2) * kQ));
        wave_barrier();
        next_q();
      }
      if (s == kSteps - 2) {   // the same of P
        __builtin_amdgcn_s_waitcnt(wait_vm_lds((SLOTS - 1) * kQ + (SLOTS - 2) * kP));
        wave_barrier();
        next_p();
      }
#pragma unroll
      for (int j = s % TP * TQ / TP; j < (s % TP + 1) * TQ / TP; ++j)
        fq[s < TP ? 1 : 0][j] = s < TP ? read_q(qs0, 1, j) : read_q(qs1, 0, j);
      fp[(s + 2) % 4] = s + 2 < kSteps ? read_p(ps0, (s + 2) / TP, (s + 2) % TP) : read_p(ps1, 0, s + 2 - kSteps);
      if (s >= TP && s < TP + kQSpan) {
#pragma unroll
        for (int i = (s - TP) * kQ / kQSpan; i < (s - TP + 1) * kQ / kQSpan; ++i) load_q(qs0, i);
      }
      const int r = s >= kSteps - 2 ? s - (kSteps - 2) : s + 2;   // steps since P's barrier
      if (r < kPSpan) {
#pragma unroll
        for (int i = r * kP / kPSpan; i < (r + 1) * kP / kPSpan; ++i) load_p(s >= kSteps - 2 ? ps0 : psp, i);
      }
#pragma unroll
      for (int j = 0; j < TQ; ++j)
        acc[s % TP][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[s % 4], fq[s / TP][j], acc[s % TP][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);   // the steps stay apart
    }
  };
  // The first SLOTS stages, of P's last one what the two steps before the first would have loaded.
  constexpr int kAhead = 2 * kP / kPSpan;
  auto load_stage = [&](uint16_t* ps, uint16_t* qs, auto n_p) {
    next_q();
#pragma unroll
    for (int i = 0; i < kQ; ++i) load_q(qs, i);
    next_p();
#pragma unroll
    for (int i = 0; i < decltype(n_p)::value; ++i) load_p(ps, i);
  };
  load_stage(pslot0, qslot0, std::integral_constant<int, kP>());
  if constexpr (MORE) {
    load_stage(pslot1, qslot1, std::integral_constant<int, kP>());
    load_stage(pslot2, qslot2, std::integral_constant<int, kP>());
    load_stage(pslot3, qslot3, std::integral_constant<int, kAhead>());
  } else {
    load_stage(pslot1, qslot1, std::integral_constant<int, kAhead>());
  }
  __builtin_amdgcn_s_waitcnt(wait_vm((SLOTS - 1) * kQ + (SLOTS - 2) * kP + kAhead));
  wave_barrier();
#pragma unroll
  for (int j = 0; j < TQ; ++j) fq[0][j] = read_q(qslot0, 0, j);
  fp[0] = read_p(pslot0, 0, 0);
  fp[1] = read_p(pslot0, 0, 1);
  // Two stages each time, the second of zeros where their number is odd: with an exit
  // between them the sums' registers were saved and restored at every turn.
  int k0 = 0;
  if constexpr (MORE) {
    while (true) {
      stage(pslot0, qslot0, pslot1, qslot1, pslot3);
      stage(pslot1, qslot1, pslot2, qslot2, pslot0);
      if ((k0 += 2 * kBk) >= kk) break;
      stage(pslot2, qslot2, pslot3, qslot3, pslot1);
      stage(pslot3, qslot3, pslot0, qslot0, pslot2);
      if ((k0 += 2 * kBk) >= kk) break;
    }
  } else {
    do {
      stage(pslot0, qslot0, pslot1, qslot1, pslot1);
      stage(pslot1, qslot1, pslot0, qslot0, pslot0);
    } while ((k0 += 2 * kBk) < kk);
  }
  __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));   // nothing is on its way into LDS any more

  // Results.  The lane's token (or row) and its neighbours along p; rows 16 apart follow.
  const int np = g.np, nq = g.nq, out_cols = g.out_cols;
  const int64_t out_ld = g.out_ld;
  const int lp = octet_at(lane);
  const int first_q = q0 + wq * (BQ / WQ) + (lane & 15);
  const int first_p = p0 + wp * (kOwn / WP);   // the wave's: a multiple of 32
  uint16_t* out = g.out + first_q * out_ld + first_p + lp;
  if constexpr (EPI == kStore) {
#pragma unroll
    for (int j = 0; j < TQ; ++j, out += 16 * out_ld)
#pragma unroll
      for (int i = 0; i < TP; i += 2) {
        float v[8];
        octet(acc[i][j], acc[i + 1][j], v);
        const int p = first_p + i * 16 + lp;
        if (first_q + j * 16 < nq && p < out_cols) store8(out + i * 16, v, out_cols - p);
      }
  } else if constexpr (EPI == kPartial) {
    const int64_t pitch = args.pitch;
    float* partial = args.partial + (static_cast<int64_t>(split) * nq + first_q) * pitch + first_p + lp;
#pragma unroll
    for (int j = 0; j < TQ; ++j, partial += 16 * pitch)
#pragma unroll
      for (int i = 0; i < TP; i += 2) {
        float v[8];
        octet(acc[i][j], acc[i + 1][j], v);
        if (first_q + j * 16 < nq && first_p + i * 16 + lp < pitch) {
          f4* to = reinterpret_cast<f4*>(partial + i * 16);
          to[0] = f4{v[0], v[1], v[2], v[3]};
          to[1] = f4{v[4], v[5], v[6], v[7]};
        }
      }
  } else if constexpr (EPI == kGated) {
    const int save = args.save, blocks = args.blocks, format = args.format;
    const Act8Rows gate = args.gate, up = args.up;
    int64_t row = static_cast<int64_t>(first_q) * np + first_p + lp, block = static_cast<int64_t>(first_q) * blocks + (first_p >> 5);
#pragma unroll
    for (int j = 0; j < TQ; ++j, out += 16 * out_ld, row += 16 * static_cast<int64_t>(np), block += 16 * static_cast<int64_t>(blocks)) {
      const bool in_q = first_q + j * 16 < nq;
#pragma unroll
      for (int i = 0; i < TP / 2; i += 2) {
        float a[8], b[8], v[8];
        octet(acc[i][j], acc[i + 1][j], a);
        octet(acc[i + TP / 2][j], acc[i + TP / 2 + 1][j], b);
        const int p = first_p + i * 16 + lp;
#pragma unroll
        for (int n = 0; n < 8; ++n) v[n] = activate<ACT>(a[n]) * b[n];
        if (p + 8 > np) {   // past the matrices' rows an infinity in x times their zeros is NaN, which would reach y
#pragma unroll
          for (int n = 0; n < 8; ++n) v[n] = p + n < np ? v[n] : 0.0f;
        }
        if (in_q && p < out_cols) store8(out + i * 16, v, 8);   // the workspace's: whole octets
        if (!save) continue;
        // 32 neighbours are one block: the lane's 8 and those of lanes ^ 16, ^ 32, ^ 48
        auto keep = [&](const float (&x)[8], const Act8Rows& to) {
          const uint32_t byte = act8_scale_byte(across_groups(top_of(x)), format);
          uint32_t w[2];
          act8_codes(x, act8_inverse(byte), format, w);
          if (!in_q || p >= np) return;
          store_codes8(to.codes + row + i * 16, u32x2{w[0], w[1]}, np - p);
          if (lane < 16) to.scales[block + (i >> 1)] = static_cast<uint8_t>(byte);
        };
        keep(a, gate);
        keep(b, up);
      }
    }
  } else {
    // The checkpoints' codes of all rows on their way at once: fetched 16 rows ahead, the product of
    // 8192 x 4096 x 14336 took 952 us instead of 889.
    struct Held {
      u32x2 g[TP / 2], u[TP / 2];
      uint32_t sg, su;   // a scale each byte
    };
    const Act8Rows gate = args.gate, up = args.up;
    const int blocks = args.blocks, format = args.format;
    Held held[TQ];
#pragma unroll
    for (int j = 0; j < TQ; ++j) {
      Held& x = held[j];
      const int q = first_q + j * 16;
      const int64_t row = static_cast<int64_t>(q) * np + first_p + lp, block = static_cast<int64_t>(q) * blocks + (first_p >> 5);
      x.sg = x.su = 0;
      if (q < nq) {
        const int more = blocks - (first_p >> 5);
        x.sg = load_bytes<TP / 2>(gate.scales + block, more);
        x.su = load_bytes<TP / 2>(up.scales + block, more);
      }
#pragma unroll
      for (int i = 0; i < TP / 2; ++i) {
        const int left = np - first_p - i * 32 - lp;   // of this lane's octet on
        x.g[i] = x.u[i] = u32x2{};
        if (q < nq && left > 0) {
          x.g[i] = load_codes8(gate.codes + row + i * 32, left);
          x.u[i] = load_codes8(up.codes + row + i * 32, left);
        }
      }
    }
    uint16_t* du_out = args.du + first_q * out_ld + first_p + lp;
    uint16_t* h_out = args.h + first_q * args.h_ld + first_p + lp;
#pragma unroll
    for (int j = 0; j < TQ; ++j, out += 16 * out_ld, du_out += 16 * out_ld, h_out += 16 * args.h_ld) {
      const Held& x = held[j];
#pragma unroll
      for (int i = 0; i < TP; i += 2) {
        float dh[8];
        octet(acc[i][j], acc[i + 1][j], dh);
        const int p = first_p + i * 16 + lp;
        if (p + 8 > np) {   // past the matrix's columns the sums are of something else
#pragma unroll
          for (int n = 0; n < 8; ++n) dh[n] = p + n < np ? dh[n] : 0.0f;
        }
        const uint32_t wg[2] = {x.g[i / 2].x, x.g[i / 2].y}, wu[2] = {x.u[i / 2].x, x.u[i / 2].y};
        float gv[8], uv[8];
        if (format == ZERO_ACT8_INT8) {
          act8_numbers_int8(wg, gv);
          act8_numbers_int8(wu, uv);
        } else {
          act8_numbers_e4m3(wg, gv);
          act8_numbers_e4m3(wu, uv);
        }
        const float sg = act8_scale(x.sg >> (4 * i) & 255u), su = act8_scale(x.su >> (4 * i) & 255u);
        float dg[8], du[8], hv[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float a, slope;
          const float u = uv[n] * su;
          activate_slope<ACT>(gv[n] * sg, a, slope);
          dg[n] = dh[n] * u * slope;
          du[n] = dh[n] * a;
          hv[n] = a * u;
        }
        if (first_q + j * 16 < nq && p < out_cols) {   // the workspace's: whole octets
          store8(out + i * 16, dg, 8);
          store8(du_out + i * 16, du, 8);
          store8(h_out + i * 16, hv, 8);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ parts of a long sum
// Where a product has fewer tiles than the card has room for, several workgroups share a
// tile's sum and this adds their parts up, in order.  256 rows of 512 alone: 4.4 us, a launch.
__global__ __launch_bounds__(256) void ffn_join_kernel(JoinArgs a) {
  join_piece(a, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x);
}

// ------------------------------------------------------------------ a few tokens
// Up to kFewTokens tokens: the weights' way from memory is all that counts, and every
// weight is used once.  No LDS on the way in: a wave takes RB blocks of 16 rows of P (of gate and
// of up) as the matrix cores want them, a row's 64 bytes by 4 lanes, and the
// tokens' the same way (from L2).  Fewer rows than the blocks have are the last one
// several times, which costs no memory: so the workgroups get equal shares.  The waves of a workgroup
// take turns along the summed index and add up at the end, in order, in LDS.
// Rows and columns of any alignment are read where they lie.
// Measured, medians: 1 token through 4096 x 14336 42 us for gate and up (5.6 TB/s), 21 for down (5.6); 24 tokens
// through 4096 x 11008 38 (4.8) and 28 (3.2: the tokens' rows, which every CU takes in from L2, are
// 1.5 times its share of the weights; with the sum in two, and twice the rows, 21 before the
// parts are added up, which costs as much).
constexpr int kFewTokens = 32;
constexpr int kFewStep = 64;   // summed index of a wave's turn: a cache line of each row

template <int TB, int NW, int RB, bool GATED>
__global__ __launch_bounds__(NW * 64) void ffn_few_kernel(Products args) {
  constexpr int M = GATED ? 2 : 1, kParts = M * RB * TB;
  __shared__ f4 part[NW][kParts][64];
  if constexpr (GATED) {
    if (static_cast<int>(blockIdx.x) >= args.tiles) {
      save_piece(args.x, (blockIdx.x - args.tiles) * (NW * 64) + threadIdx.x);
      return;
    }
  }
  const Product& g = args.of[0];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row0 = blockIdx.x * args.rows, kk = g.kk, nq = g.nq;
  const int np = g.np - row0 < args.rows ? g.np : row0 + args.rows;   // where this workgroup's end
  const uint16_t* w[M][RB];
  const uint16_t* x[TB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    // rows past the end: the last one once more, their results are dropped
    const int row = row0 + r * 16 + (lane & 15);
    const int64_t at = (row < np ? row : np - 1) * g.p_ld + (lane >> 4) * 8;
    w[0][r] = g.p + at;
    if constexpr (GATED) w[1][r] = g.p2 + at;
  }
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    const int q = b * 16 + (lane & 15);
    x[b] = g.q + (q < nq ? q : nq - 1) * g.q_ld + (lane >> 4) * 8;
  }
  f4 acc[M][RB][TB] = {};
  constexpr int kU = kFewStep / 32;
  struct Frags {
    b8 w[M][RB][kU], x[TB][kU];
  };
  auto load = [&](Frags& f, int k, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int at = k + u * 32, n = WHOLE ? 8 : kk - at - (lane >> 4) * 8;
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r) f.w[m][r][u] = load_piece(w[m][r] + at, n);
#pragma unroll
      for (int b = 0; b < TB; ++b) f.x[b][u] = load_piece(x[b] + at, n);
    }
    __builtin_amdgcn_sched_barrier(0);   // all on their way before the first is waited for
  };
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
          for (int b = 0; b < TB; ++b)
            acc[m][r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.w[m][r][u], f.x[b][u], acc[m][r][b], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // The wave's turns, one loaded ahead; the workgroups start at different ones, so that
  // they do not all read the same columns of their rows, which lie in the same few channels.
  // A row's start, and with it the order of its sum, goes by the row and not by the workgroup: y has the
  // same bits whether a checkpoint is saved or not.  Eight turns are common, and with group % turns every
  // eighth group starts alike: 1 token of 4096 x 14336 took 68.2 us, with one more every eight 65.5.
  const int whole = kk / kFewStep, turns = whole > wave ? (whole - wave - 1) / NW + 1 : 0;
  const int group = row0 / args.alike;
  int next = turns ? (group + group / 8) % turns : 0;
  auto place = [&] {
    const int k = (next * NW + wave) * kFewStep;
    next = next + 1 < turns ? next + 1 : 0;
    return k;
  };
  Frags f0, f1;
  if (turns) load(f0, place(), std::true_type());
  int t = 0;
  for (; t + 2 < turns; t += 2) {
    load(f1, place(), std::true_type());
    multiply(f0);
    load(f0, place(), std::true_type());
    multiply(f1);
  }
  if (t + 1 < turns) {
    load(f1, place(), std::true_type());
    multiply(f0);
    multiply(f1);
  } else if (turns) {
    multiply(f0);
  }
  if (whole * kFewStep < kk && wave == whole % NW) {
    load(f0, whole * kFewStep, std::false_type());
    multiply(f0);
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int b = 0; b < TB; ++b) part[wave][(m * RB + r) * TB + b][lane] = acc[m][r][b];
  __syncthreads();
  if (wave >= TB) return;
  // Wave b: tokens 16 b to 16 b + 15, one per lane & 15; 4 neighbours along p of each block.
  const int q = wave * 16 + (lane & 15), lp = (lane >> 4) * 4;
  f4 sum[M][RB];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      f4 v = part[0][(m * RB + r) * TB + wave][lane];
#pragma unroll
      for (int n = 1; n < NW; ++n) v += part[n][(m * RB + r) * TB + wave][lane];
      sum[m][r] = v;
    }
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int p = row0 + r * 16 + lp;
    f4 v = sum[0][r];
    if constexpr (GATED) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float a = args.act == ZERO_FFN_SILU   ? activate<ZERO_FFN_SILU>(v[n])
                        : args.act == ZERO_FFN_GELU ? activate<ZERO_FFN_GELU>(v[n])
                                                    : activate<ZERO_FFN_RELU>(v[n]);
        v[n] = a * sum[1][r][n];
      }
    }
    if (q >= nq || p >= np) continue;
    const u32x2 two = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
    uint16_t* dst = g.out + q * g.out_ld + p;
    if (p + 4 <= np) {
      __builtin_memcpy(dst, &two, 8);
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (p + n < np) dst[n] = static_cast<uint16_t>(two[n >> 1] >> ((n & 1) * 16));
    }
  }
  if constexpr (GATED) {
    static_assert(RB * 16 == ZERO_ACT8_BLOCK, "a workgroup has whole blocks of a checkpoint");
    if (!args.save) return;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const Act8Rows& to = m ? args.up : args.gate;
      // rows past the end are copies of the last one, which is in this block
      float all[RB * 4];
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int n = 0; n < 4; ++n) all[r * 4 + n] = sum[m][r][n];
      const uint32_t byte = act8_scale_byte(across_groups(top_of(all)), args.format);
      uint32_t codes[RB];
      act8_codes(all, act8_inverse(byte), args.format, codes);
      if (q >= nq) continue;
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const int p = row0 + r * 16 + lp;
        const uint32_t c = codes[r];
        uint8_t* dst = to.codes + static_cast<int64_t>(q) * g.np + p;
        if (p + 4 <= np) {
          __builtin_memcpy(dst, &c, 4);
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n)
            if (p + n < np) dst[n] = static_cast<uint8_t>(c >> (8 * n));
        }
      }
      if (lane < 16) to.scales[static_cast<int64_t>(q) * args.blocks + blockIdx.x] = static_cast<uint8_t>(byte);
    }
  }
}

// ------------------------------------------------------------------ operands that the products cannot take
// A matrix whose rows are not 16-byte aligned, or end inside a stage: copied to the
// workspace with a pitch of whole stages, zeros behind each row.  Bound by its launch and the
// unaligned reads: x and the weights of 777 x 1301 x 1999 11 us for 36 MB; of a wide layer by the bytes, three
// weights read and written on every call (256 tokens of 4096 x 11000 forward 205 us, of 4096 x 11008 105).
struct PackArgs {
  struct {
    const uint16_t* from;
    int64_t ld;
    uint16_t* to;
    int64_t pitch, rows;
    int cols;
  } of[4];   // one per blockIdx.y
};
__global__ __launch_bounds__(256) void ffn_pack_kernel(PackArgs args) {
  const auto& a = args.of[blockIdx.y];
  const int64_t pieces = a.pitch / 8, n = a.rows * pieces;
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; k < n; k += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = k / pieces;
    const int c = static_cast<int>(k - r * pieces) * 8;
    *reinterpret_cast<b8*>(a.to + k * 8) = load_piece(a.from + r * a.ld + c, a.cols - c);   // rows follow one another
  }
}

// ------------------------------------------------------------------ launches
struct Matrix {   // as a product takes it
  const uint16_t* at;
  int64_t ld;
};

bool aligned(const uint16_t* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }

// The workspace in order.  take(): the next `elements` BF16 values, 256-byte aligned.
struct Carver {
  char* at;
  uint16_t* take(int64_t elements) {
    char* p = at;
    at += (elements * 2 + 255) / 256 * 256;
    return reinterpret_cast<uint16_t*>(p);
  }
};

// Matrices to copy, in one launch.
struct Packing {
  PackArgs args = {};
  int n = 0;
  int64_t most = 0;
  Matrix add(const uint16_t* from, int64_t ld, uint16_t* to, int64_t pitch, int64_t rows, int64_t cols) {
    args.of[n++] = {from, ld, to, pitch, rows, static_cast<int>(cols)};
    if (rows * pitch / 8 > most) most = rows * pitch / 8;
    return {to, pitch};
  }
  hipError_t go(hipStream_t s) const {
    if (n == 0) return hipSuccess;
    const int64_t grid = (most + 255) / 256;
    hipLaunchKernelGGL(ffn_pack_kernel, dim3(static_cast<unsigned>(grid < 4096 ? grid : 4096), n), dim3(256), 0, s, args);
    return hipGetLastError();
  }
};

// Tiles of bp x bq: numbers a's products' and says how many there are.
template <Epilogue EPI>
int64_t number_tiles(Products& a, int n, int bp, int bq) {
  int64_t total = 0;
  for (int k = 0; k < 3; ++k) {
    a.first[k] = k < n ? static_cast<int>(total) : 0x7FFFFFFF;
    if (k >= n) continue;
    Product& g = a.of[k];
    const int own = EPI == kGated ? bp / 2 : bp;
    const int columns = g.out_cols > g.np ? g.out_cols : g.np;
    g.tiles_p = (columns + own - 1) / own;
    g.tiles_q = (g.nq + bq - 1) / bq;
    total += static_cast<int64_t>(g.tiles_p) * g.tiles_q;
  }
  return total;
}

// `count` workgroups of tiles, from a.begin on, and the side work's.
template <int BP, int BQ, int WP, int WQ, int SLOTS, bool PCOL, bool QCOL, Epilogue EPI, int ACT = 0>
hipError_t launch_tiles(Products& a, int64_t count, hipStream_t s) {
  constexpr int kThreads = WP * WQ * 64;
  a.tiles = static_cast<int>(count);
  const int64_t side = (a.side + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((ffn_product_kernel<BP, BQ, WP, WQ, SLOTS, PCOL, QCOL, EPI, ACT>), dim3(static_cast<unsigned>(count + side)),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int BP, int BQ, int WP, int WQ, int SLOTS, bool PCOL, bool QCOL, Epilogue EPI, int ACT = 0>
hipError_t tiles(Products a, int n, hipStream_t s) {
  const int64_t total = number_tiles<EPI>(a, n, BP, BQ);
  return launch_tiles<BP, BQ, WP, WQ, SLOTS, PCOL, QCOL, EPI, ACT>(a, EPI == kPartial ? total * a.splits : total, s);
}

// Tiles of 256 x 256, one per CU at a time.  What is left over after whole rounds is done in quarters,
// two per CU, where that is half a round at most.
template <bool PCOL, bool QCOL, Epilogue EPI, int ACT>
hipError_t large_tiles(Products a, int n, hipStream_t s) {
  constexpr int64_t kCus = 256;
  const int64_t total = number_tiles<EPI>(a, n, 256, 256), over = total % kCus;
  const bool split = total > kCus && over > 0 && over <= kCus / 2;
  const hipError_t e = launch_tiles<256, 256, 2, 4, 2, PCOL, QCOL, EPI, ACT>(a, split ? total - over : total, s);
  if (e != hipSuccess || !split) return e;
  a.begin = static_cast<int>(total - over);
  a.quarters = 1;
  a.side = 0;
  return launch_tiles<128, 128, 2, 2, 2, PCOL, QCOL, EPI, ACT>(a, over * 4, s);
}

// Gate and up: up to 32 rows of each by 8 waves (over 16 tokens by 4: more registers each);
// down: up to 16 rows by 8.  A CU takes in some 25
// bytes/ns from memory, so the CUs' shares decide: 1 token through gate and up of 4096 x 11008
// takes as long as through 4096 x 14336 where every workgroup has 32 rows (2 on some CUs,
// 1 on the others).
template <bool GATED>
hipError_t few(Products a, hipStream_t s) {
  constexpr int kBlocks = GATED ? 2 : 1, kMost = kBlocks * 16, kCus = 256;
  const int np = a.of[0].np, each = (np + kCus * kMost - 1) / (kCus * kMost);   // workgroups of a CU
  const int share = (np + kCus * each - 1) / (kCus * each), rows = share < 8 ? 8 : share;
  a.rows = a.save ? kMost : rows;
  // Saving takes whole blocks of 32 rows: where both kinds of workgroups begin, the start may change.
  a.alike = GATED ? std::lcm(rows, kMost) : rows;
  a.tiles = (np + a.rows - 1) / a.rows;
  const int waves = GATED && a.of[0].nq > 16 ? 4 : 8, threads = waves * 64;
  const dim3 grid(static_cast<unsigned>(a.tiles + (a.side + threads - 1) / threads));
  if (a.of[0].nq <= 16)
    hipLaunchKernelGGL((ffn_few_kernel<1, 8, kBlocks, GATED>), grid, dim3(threads), 0, s, a);
  else
    hipLaunchKernelGGL((ffn_few_kernel<2, GATED ? 4 : 8, kBlocks, GATED>), grid, dim3(threads), 0, s, a);
  return hipGetLastError();
}

// Modelled times in us of n tiles whose sums have so many stages, fitted to launches with operands of
// 1024 to 4096 x 2816 to 28672, from memory and from caches: up to 256 tiles have a CU each (four stages
// of 128 x 64 on their way, with columns a little less work), up to 512 of 128 x 128 two on each.
double time256(double stages, int64_t n) { return 8.0 + stages * (1.1 + 0.35 * static_cast<double>(n) / 256); }
double time128(double stages, int64_t n) { return 3.0 + stages * (n <= 256 ? 0.64 : n <= 512 ? 1.1 : 1.25 * static_cast<double>(n) / 512); }
// Gate and up of 4096 x 14336, 256 tokens: 67 us in one round, 77 in tiles of 128 x 128, 81 of 256 x 256.
double time128x256(double stages, int64_t n) { return 5.0 + stages * (0.87 + 0.1 * static_cast<double>(n) / 256); }
double time64(double stages, bool columns) { return 3.2 + stages * (columns ? 0.36 : 0.42); }

// How y's and dx's sums (nq rows of np values) are shared out.  Measured, 4096 x 14336 from memory, in
// parts and in the best whole tiles: 64 rows 31 and 121 us, 256 54 and 123, 512 77 and 121, 1024 (four
// parts of tiles of 256) 108 and 161, 2048 (two) 178 and 231; kk = 2816, 256 rows 18 and 19,
// 1024 36 and 27 (whole).
struct Parts {
  int splits, chunk;
  bool large;   // tiles of 256 x 256
  int64_t pitch, bytes;
};
Parts parts_of(int64_t np, int64_t nq, int64_t kk, bool columns) {
  Parts x = {1, 0, false, (np + 7) / 8 * 8, 0};
  auto tiles_of = [&](int64_t bp, int64_t bq) { return (np + bp - 1) / bp * ((nq + bq - 1) / bq); };
  const int64_t n256 = tiles_of(256, 256), n128 = tiles_of(128, 128), n64 = tiles_of(128, 64);
  if (n128 == 0 || n256 >= 256) return x;
  const double stages = static_cast<double>((kk + kBk - 1) / kBk);
  double best = time128(stages, n128);
  if (n64 <= 256 && time64(stages, columns) < best) best = time64(stages, columns);
  if (time256(stages, n256) < best) best = time256(stages, n256);
  for (int64_t splits = 2; splits <= 16; ++splits) {
    const int64_t chunk = ((kk + splits - 1) / splits + 2 * kBk - 1) / (2 * kBk) * (2 * kBk);
    const int64_t parts = (kk + chunk - 1) / chunk;
    if (parts < 2) continue;
    // written, and read by the second launch; the choice looks at whole 64 rows, so that the room that
    // it needs grows within them
    const int64_t bytes = parts * nq * x.pitch * 4, moved = 2 * (parts * ((nq + 63) / 64 * 64) * x.pitch * 4);
    const double st = static_cast<double>(chunk / kBk), join = 4.5 + static_cast<double>(moved) / 5e6;
    for (int large = 0; large < 2; ++large) {
      const int64_t n = (large ? n256 : n128) * parts;
      if (n > (large ? 256 : 512)) continue;
      const double time = join + (large ? time256(st, n) : time128(st, n));
      if (time < best) {
        best = time;
        x.splits = static_cast<int>(parts);
        x.chunk = static_cast<int>(chunk);
        x.large = large;
        x.bytes = bytes;
      }
    }
  }
  return x;
}

// 128 x 128, n workgroups.  With a CU each they keep four stages of rows on their way: gate and up of
// 4096 x 14336 from memory for 128 tokens 55 us instead of 61, of 2048 x 8192 26 instead of 29; y
// of 64 tokens in eight parts 31 instead of 34.  Columns gain nothing on average (dh of 14336 x 4096 35
// instead of 37, of 4096 x 1024 11 instead of 10).
template <bool PCOL, bool QCOL, Epilogue EPI, int ACT = 0>
hipError_t tiles128(const Products& a, int products, int64_t n, hipStream_t s) {
  if constexpr (!PCOL) {
    if (n <= 256) return tiles<128, 128, 2, 2, 4, PCOL, QCOL, EPI, ACT>(a, products, s);
  }
  return tiles<128, 128, 2, 2, 2, PCOL, QCOL, EPI, ACT>(a, products, s);
}

// later: the launch that can add the parts up beside its own work.
template <bool PCOL>
hipError_t product_in_parts(Products a, const Parts& parts, void* room, hipStream_t s, Products* later = nullptr) {
  a.splits = parts.splits;
  a.chunk = parts.chunk;
  a.pitch = parts.pitch;
  a.partial = static_cast<float*>(room);
  const Product& g = a.of[0];
  const int64_t n = (g.np + 127) / 128 * ((g.nq + 127) / 128) * static_cast<int64_t>(parts.splits);
  const hipError_t e = parts.large ? tiles<256, 256, 2, 4, 2, PCOL, false, kPartial>(a, 1, s)
                                   : tiles128<PCOL, false, kPartial>(a, 1, n, s);
  if (e != hipSuccess) return e;
  const JoinArgs j = {a.partial, a.pitch, a.splits, g.nq, g.np, g.out, g.out_ld};
  const int64_t pieces = g.nq * (a.pitch / 8);
  if (later && pieces <= kSideMost) {
    later->join = j;
    later->side = pieces;
    return hipSuccess;
  }
  hipLaunchKernelGGL(ffn_join_kernel, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, s, j);
  return hipGetLastError();
}

template <bool PCOL, bool QCOL, Epilogue EPI, int ACT = 0>
hipError_t product(const Products& a, int n, hipStream_t s) {
  auto count = [&](int bp, int bq) {
    const int64_t own = EPI == kGated ? bp / 2 : bp;
    int64_t t = 0;
    for (int k = 0; k < n; ++k) t += (a.of[k].np + own - 1) / own * ((a.of[k].nq + bq - 1) / bq);
    return t;
  };
  // 256 x 256 where they fill the card or their longer stages take less time than the rounds of 128 x 128
  // (512 rows of 28672 values: 4096 a sum 97 and 142 us; 8192 values, 1024 a sum 24 and 13).
  const int64_t n256 = count(256, 256), n128 = count(128, 128);
  const double stages = (a.of[0].kk + kBk - 1) / kBk;
  if constexpr (!QCOL) {   // (columns of 64 would need another order in LDS)
    if (n256 < 256 && (count(128, 64) <= 256 || a.of[0].nq <= 64) && time64(stages, PCOL) < time256(stages, n256))
      return tiles<128, 64, 2, 2, 4, PCOL, QCOL, EPI, ACT>(a, n, s);
  }
  if constexpr (EPI == kGated) {   // 256 tokens of fewer rows, to bring the weights in once
    const int64_t n = count(128, 256);
    const double time = time128x256(stages, n);
    if (n <= 256 && time < time128(stages, n128) && time < time256(stages, n256))
      return tiles<128, 256, 2, 4, 2, PCOL, QCOL, EPI, ACT>(a, 1, s);
  }
  if (n256 >= 256 || time256(stages, n256) < time128(stages, n128)) return large_tiles<PCOL, QCOL, EPI, ACT>(a, n, s);
  return tiles128<PCOL, QCOL, EPI, ACT>(a, n, n128, s);
}

// The activation is a constant of the kernel: asked for each value, its code was 250 KB and did not
// fit the instruction cache (dh's product of 8192 x 4096 x 14336: 967 us).
template <bool PCOL, Epilogue EPI>
hipError_t activated(const Products& a, hipStream_t s) {
  if (a.act == ZERO_FFN_SILU) return product<PCOL, false, EPI, ZERO_FFN_SILU>(a, 1, s);
  if (a.act == ZERO_FFN_GELU) return product<PCOL, false, EPI, ZERO_FFN_GELU>(a, 1, s);
  return product<PCOL, false, EPI, ZERO_FFN_RELU>(a, 1, s);
}

}  // namespace

#define ZERO_TRY(call)                      \
  do {                                      \
    const hipError_t e_ = (call);           \
    if (e_ != hipSuccess) return e_;        \
  } while (0)

// Forward: h, and room for x and the weights where they have to be packed.
// Backward: dg beside du, h, x's values, and room for dy and the weights.
int64_t ffn_workspace_bytes(int64_t tokens, int64_t model, int64_t hidden, bool backward, bool unaligned) {
  const int64_t dp = pad_up(model), fp = pad_up(hidden);
  auto bytes = [](int64_t elements) { return (elements * 2 + 255) / 256 * 256; };
  if (!backward && tokens <= kFewTokens) return bytes(tokens * fp);
  int64_t n = bytes(tokens * dp);                                   // x or dy
  if (backward)
    n += bytes(tokens * 2 * fp) + bytes(tokens * fp) + bytes(tokens * dp);
  else
    n += bytes(tokens * fp);
  n += bytes(parts_of(model, tokens, backward ? 2 * fp : fp, backward).bytes / 2);
  if (unaligned || model % kPad || hidden % kPad) n += 2 * bytes(hidden * dp) + bytes(model * fp);
  return n;
}

// The room that parts take grows with the rows within 64 of them, and may fall from one 64 to the next;
// from 256 tiles of 256 x 256 on there is none.  So the most that any count up to `tokens` takes is that
// of `tokens` itself or of a multiple of 64 with parts.
int64_t ffn_workspace_room(int64_t tokens, int64_t model, int64_t hidden, bool backward, bool unaligned) {
  int64_t most = ffn_workspace_bytes(tokens, model, hidden, backward, unaligned);
  for (int64_t t = 64; t <= tokens && (model + 255) / 256 * ((t + 255) / 256) < 256; t += 64) {
    const int64_t n = ffn_workspace_bytes(t, model, hidden, backward, unaligned);
    if (n > most) most = n;
  }
  return most;
}

bool ffn_weights_aligned(const FfnParams& p) {
  return aligned(p.w_gate, p.model) && aligned(p.w_up, p.model) && aligned(p.w_down, p.hidden);
}

hipError_t launch_ffn_forward(const FfnParams& p, hipStream_t s) {
  const int64_t t = p.tokens, d = p.model, f = p.hidden, dp = pad_up(d), fp = pad_up(f);
  Carver ws = {static_cast<char*>(p.workspace)};
  uint16_t* h = ws.take(t * fp);
  const bool is_few = t <= kFewTokens;
  const Parts parts = is_few ? Parts{1, 0, false, 0, 0} : parts_of(d, t, fp, false);
  uint16_t* parts_room = ws.take(parts.bytes / 2);
  uint16_t* x_room = is_few ? nullptr : ws.take(t * dp);
  Matrix x = {p.x, p.x_row}, gate = {p.w_gate, d}, up = {p.w_up, d}, down = {p.w_down, f};
  Packing packing;
  if (!is_few && (!aligned(x.at, x.ld) || d % kPad)) x = packing.add(x.at, x.ld, x_room, dp, t, d);
  if (!is_few && (!ffn_weights_aligned(p) || d % kPad || f % kPad)) {
    gate = packing.add(gate.at, d, ws.take(f * dp), dp, f, d);
    up = packing.add(up.at, d, ws.take(f * dp), dp, f, d);
    down = packing.add(down.at, f, ws.take(d * fp), fp, d, f);
  }
  ZERO_TRY(packing.go(s));
  Products a = {};
  if (p.save) {
    a.x = {const_cast<uint16_t*>(p.x), p.x_row, t, d, p.ckpt.x_codes, p.ckpt.x_scales, p.ckpt.format, 0};
    if (pieces_of(a.x) <= kSideMost)
      a.side = pieces_of(a.x);
    else
      ZERO_TRY(launch_act8_save(a.x, s));
  }
  a.gate = {p.ckpt.gate_codes, p.ckpt.gate_scales};
  a.up = {p.ckpt.up_codes, p.ckpt.up_scales};
  a.blocks = static_cast<int>((f + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK);
  a.format = p.ckpt.format;
  a.act = p.activation;
  a.save = p.save;
  // Where x stays in an XCD's L2 (4 MiB) the tiles of the weights need not keep in step: they begin at
  // different columns, which lie in different channels of the memory (4096 x 14336 from memory, 64 tokens:
  // 51 us in step, 46 spread; 128: 55 and 51; 256: 78 and 77).
  a.spread = t * d * 2 <= 4 << 20;
  Product& g = a.of[0];
  g.p = gate.at;
  g.p2 = up.at;
  g.p_ld = gate.ld;
  g.q = x.at;
  g.q_ld = x.ld;
  g.np = static_cast<int>(f);
  g.nq = static_cast<int>(t);
  g.kk = static_cast<int>(is_few ? d : dp);
  g.out = h;
  g.out_ld = fp;
  g.out_cols = static_cast<int>(fp);
  ZERO_TRY((is_few ? few<true>(a, s) : activated<false, kGated>(a, s)));
  Products b = {};
  Product& y = b.of[0];
  y.p = down.at;
  y.p_ld = down.ld;
  y.q = h;
  y.q_ld = fp;
  y.np = static_cast<int>(d);
  y.nq = static_cast<int>(t);
  y.kk = static_cast<int>(is_few ? f : fp);
  y.out = p.y;
  y.out_ld = p.y_row;
  y.out_cols = static_cast<int>(d);
  if (is_few) return few<false>(b, s);
  if (parts.splits > 1) return product_in_parts<false>(b, parts, parts_room, s);
  return product<false, false, kStore>(b, 1, s);
}

hipError_t launch_ffn_backward(const FfnParams& p, hipStream_t s) {
  const int64_t t = p.tokens, d = p.model, f = p.hidden, dp = pad_up(d), fp = pad_up(f);
  Carver ws = {static_cast<char*>(p.workspace)};
  uint16_t* dgu = ws.take(t * 2 * fp);
  uint16_t* h = ws.take(t * fp);
  uint16_t* x = ws.take(t * dp);
  uint16_t* dy_room = ws.take(t * dp);
  const Parts parts = parts_of(d, t, 2 * fp, true);
  uint16_t* parts_room = ws.take(parts.bytes / 2);
  Matrix dy = {p.x, p.x_row}, gate = {p.w_gate, d}, up = {p.w_up, d}, down = {p.w_down, f};
  int dy_cols = static_cast<int>(d), w_cols = static_cast<int>(d), down_cols = static_cast<int>(f);
  Packing packing;
  if (t > 0 && (!aligned(dy.at, dy.ld) || d % kPad)) {
    dy = packing.add(dy.at, dy.ld, dy_room, dp, t, d);
    dy_cols = static_cast<int>(dp);
  }
  if (t > 0 && (!ffn_weights_aligned(p) || d % kPad || f % kPad)) {
    gate = packing.add(gate.at, d, ws.take(f * dp), dp, f, d);
    up = packing.add(up.at, d, ws.take(f * dp), dp, f, d);
    down = packing.add(down.at, f, ws.take(d * fp), fp, d, f);
    w_cols = static_cast<int>(dp);
    down_cols = static_cast<int>(fp);
  }
  ZERO_TRY(packing.go(s));
  // dh, and from it dg, du and h
  Products a = {};
  a.x = {x, dp, t, d, p.ckpt.x_codes, p.ckpt.x_scales, p.ckpt.format, 0};
  if (pieces_of(a.x) <= kSideMost)
    a.side = pieces_of(a.x);
  else
    ZERO_TRY(launch_act8_load(a.x, s));
  a.gate = {p.ckpt.gate_codes, p.ckpt.gate_scales};
  a.up = {p.ckpt.up_codes, p.ckpt.up_scales};
  a.blocks = static_cast<int>((f + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK);
  a.format = p.ckpt.format;
  a.act = p.activation;
  a.du = dgu + fp;
  a.h = h;
  a.h_ld = fp;
  Product& g = a.of[0];
  g.p = g.p2 = down.at;
  g.p_ld = down.ld;
  g.p_cols = down_cols;
  g.p_end = static_cast<int>(d);
  g.turn = 0x7FFFFFFF;
  g.q = dy.at;
  g.q_ld = dy.ld;
  g.np = static_cast<int>(f);
  g.nq = static_cast<int>(t);
  g.kk = static_cast<int>(dp);
  g.out = dgu;
  g.out_ld = 2 * fp;
  g.out_cols = static_cast<int>(fp);
  if (t > 0) ZERO_TRY((activated<true, kSlopes>(a, s)));
  Products c = {};
  if (p.y && t > 0) {   // dx
    Products b = {};
    Product& y = b.of[0];
    y.p = gate.at;
    y.p2 = up.at;
    y.p_ld = gate.ld;
    y.p_cols = w_cols;
    y.p_end = static_cast<int>(f);
    y.turn = static_cast<int>(fp);
    y.q = dgu;
    y.q_ld = 2 * fp;
    y.np = static_cast<int>(d);
    y.nq = static_cast<int>(t);
    y.kk = static_cast<int>(2 * fp);
    y.out = p.y;
    y.out_ld = p.y_row;
    y.out_cols = static_cast<int>(d);
    ZERO_TRY((parts.splits > 1 ? product_in_parts<true>(b, parts, parts_room, s, &c) : product<true, false, kStore>(b, 1, s)));
  }
  // the weights' gradients; without tokens sums of nothing, zeros
  for (int k = 0; k < 3; ++k) {
    Product& w = c.of[k];
    const bool last = k == 2;
    w.p = w.p2 = last ? h : x;
    w.p_ld = last ? fp : dp;
    w.p_cols = static_cast<int>(last ? fp : dp);
    w.q = last ? dy.at : dgu + k * fp;
    w.q_ld = last ? dy.ld : 2 * fp;
    w.q_cols = last ? dy_cols : static_cast<int>(fp);
    w.p_end = w.q_end = static_cast<int>(t);
    w.turn = 0x7FFFFFFF;
    w.np = static_cast<int>(last ? f : d);
    w.nq = static_cast<int>(last ? d : f);
    w.kk = static_cast<int>(t);
    w.out = k == 0 ? p.d_gate : k == 1 ? p.d_up : p.d_down;
    w.out_ld = w.np;
    w.out_cols = w.np;
  }
  return product<true, true, kStore>(c, 3, s);
}

}  // namespace zero
