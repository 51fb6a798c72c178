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
#include <type_traits>

#include "act8.h"
#include "kernels.h"

#pragma clang fp contract(off)

namespace zero {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBk = 64;        // summed index per stage: rows of 128 bytes in LDS
constexpr int kPad = 64;       // pitches of the workspace's matrices are multiples of this
constexpr int kRawFlags = 0x00020000;

__host__ __device__ inline int64_t pad_up(int64_t n) { return (n + kPad - 1) / kPad * kPad; }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(lo))) |
         (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(hi))) << 16);
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
  __amdgpu_buffer_rsrc_t rsrc, none;      // none: no bytes in range, a load through it gives zeros
  int voff[kN], wave;
  bool any;
  // rows: how many of the tile's rows, from the first of this wave's on, the matrix has; lds_row:
  // the wave's first row in LDS, first: the row of the matrix that goes there.
  __device__ __forceinline__ RowStager(const uint16_t* m, int64_t ld, int64_t first, int64_t rows, int kk, int wave_, int lane)
      : wave(wave_), any(rows > 0) {
    const int64_t most = kN * 8;
    const int64_t n = rows < most ? rows : most;
    uint16_t* base = const_cast<uint16_t*>(m + (any ? first : 0) * ld);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, any ? static_cast<int>(((n - 1) * ld + kk) * 2) : 0, kRawFlags);
    none = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(m), 0, 0, kRawFlags);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = i * 8 + (lane >> 3);   // kN * 8 is a multiple of 16: the wave's first row shifts no piece
      voff[i] = r * static_cast<int>(ld) * 2 + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
    static_assert(kN % 2 == 0, "see voff");
  }
  // A stage past the end is loaded too, so that the loads on their way can be
  // counted, but from nowhere.
  __device__ __forceinline__ void one(uint16_t* lds, int k0, bool live, int i) const {
#ifdef __HIP_DEVICE_COMPILE__   // the builtin is unknown to the host pass
    const bool l = live && any;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(l ? rsrc : none, (lds_void*)(lds + (wave * kN + i) * 8 * kBk), 16, voff[i],
                                             l ? k0 * 2 : 0, 0, 0);
#endif
  }
};

// Rows [k0, k0 + 64) and columns [col0, col0 + C) of an operand whose rows lie along
// k: 64 rows of 2 C bytes, from which transposing reads take the columns.  Those
// read 64 bytes of four rows together: the 64-byte piece c of row r lies at piece
// c ^ (r & 3).  Rows past `end` read as zeros (the descriptor ends there), columns
// past a row's end as the next row's: their results are dropped.
template <int C, int NW>
struct ColumnStager {
  static constexpr int kRows = 512 / C, kN = 64 / kRows / NW;   // rows of one instruction, instructions of a wave
  static_assert(kN * kRows * NW == 64 && (kN * kRows) % 4 == 0, "every wave moves the same number of pieces");
  const uint16_t* m;
  int64_t ld;
  int cols, col0, voff[kN], wave;
  __device__ __forceinline__ ColumnStager(const uint16_t* m_, int64_t ld_, int col0_, int cols_, int wave_, int lane)
      : m(m_), ld(ld_), cols(cols_), col0(col0_), wave(wave_) {
    const int row = lane / (64 / kRows), piece = lane % (64 / kRows);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = (wave * kN + i) * kRows + row;
      voff[i] = r * static_cast<int>(ld) * 2 + (((piece >> 2) ^ (r & 3)) << 6) + (piece & 3) * 16;
    }
  }
  __device__ __forceinline__ void one(uint16_t* lds, const uint16_t* from, int k0, int end, bool live, int i) const {
#ifdef __HIP_DEVICE_COMPILE__
    const int left = end - k0 < kBk ? end - k0 : kBk;
    const bool l = live && left > 0;
    uint16_t* base = const_cast<uint16_t*>(l ? from + k0 * ld + col0 : from);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(base, 0, l ? static_cast<int>(((left - 1) * ld + cols - col0) * 2) : 0, kRawFlags),
        (lds_void*)(lds + (wave * kN + i) * 512), 16, voff[i], 0, 0, 0);
#endif
  }
};

// Byte offset in a slot of the lane's first fragment piece: row first + (lane & 31),
// piece lane >> 5, moved as RowStager moves it.  Pieces 2, 4 and 6 further on are at
// the offset with bits 5 and 6 flipped.
__device__ __forceinline__ int lane_at_row(int first, int lane) {
  return (first + (lane & 31)) * kBk * 2 + (((lane >> 5) ^ ((lane >> 1) & 7)) << 4);
}
// What the lane points a transposing read at: row 8 * (lane >> 5) + ((lane >> 2) & 3),
// columns first + 16 * ((lane >> 4) & 1) + 4 * (lane & 3).
template <int C>
__device__ __forceinline__ int lane_at_column(int first, int lane) {
  return ((lane >> 5) * 8 + ((lane >> 2) & 3)) * C * 2 + (((first >> 5) ^ ((lane >> 2) & 3)) << 6) +
         ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
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

__device__ __forceinline__ float activate(float g, int act) {
  if (act == ZERO_FFN_SILU) return g * sigmoid(g);
  if (act == ZERO_FFN_GELU) return g * sigmoid(gelu_inner(g));
  return g < 0.0f ? 0.0f : g;   // NaN stays
}

// act(g) and its derivative (0 at ReLU's corner).
__device__ __forceinline__ void activate_slope(float g, int act, float& a, float& slope) {
  if (act == ZERO_FFN_RELU) {
    a = g < 0.0f ? 0.0f : g;
    slope = g > 0.0f ? 1.0f : g <= 0.0f ? 0.0f : g;
    return;
  }
  if (act == ZERO_FFN_SILU) {
    const float s = sigmoid(g);
    a = g * s;
    slope = s * (1.0f + g * (1.0f - s));
    return;
  }
  const float s = sigmoid(gelu_inner(g));
  const float z = g < -16.0f ? -16.0f : g > 16.0f ? 16.0f : g;   // sigma' is 0 there
  a = g * s;
  slope = s + z * s * (1.0f - s) * (2.0f * kGeluIn) * (1.0f + 3.0f * kGeluCube * z * z);
}

// ------------------------------------------------------------------ products
enum Epilogue {
  kStore,      // out = the sums
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
  int out_vec;             // 16-byte stores are aligned
};

struct Products {
  Product of[3];
  int first[3];            // tile number of each; those past the last have 0x7FFFFFFF
  // kGated and kSlopes
  Act8Rows gate, up;
  uint16_t* du;            // kSlopes: out is dg, both with out_ld
  uint16_t* h;
  int64_t h_ld;
  int blocks;              // scales of a row
  int format, act, save;
};

constexpr int kGroup = 8;  // tiles of q that one XCD's neighbours share

// 8 values to memory, which is 16-byte aligned if vec; the first n of them.
__device__ __forceinline__ void store8(uint16_t* dst, const float (&v)[8], int vec, int n) {
  const u32x4 w = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
  if (vec && n >= 8) {
    *reinterpret_cast<u32x4*>(dst) = w;
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

// A block's sums, as the matrix cores leave them: lane l has column q = l & 31 and rows p = 8 u +
// 4 * (l >> 5) + 0..3, u = 0..3.  After the exchange of halves between u and u + 1
// it has 8 neighbours along p, 16 h + 8 * (l >> 5) + 0..7, h = 0, 1.
__device__ __forceinline__ void octets(const f16& acc, float (&v)[2][8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a = __float_as_uint(acc[8 * h + q]), b = __float_as_uint(acc[8 * h + 4 + q]);
#ifdef __HIP_DEVICE_COMPILE__
      const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
      a = r[0];
      b = r[1];
#endif
      v[h][q] = __uint_as_float(a);
      v[h][4 + q] = __uint_as_float(b);
    }
}

// A tile of BP x BQ results by WP x WQ waves.
template <int BP, int BQ, int WP, int WQ, bool PCOL, bool QCOL, Epilogue EPI>
__global__ __launch_bounds__(WP * WQ * 64) void ffn_product_kernel(Products args) {
  constexpr int NW = WP * WQ;
  constexpr int TP = BP / WP / 32, TQ = BQ / WQ / 32;   // 32 x 32 blocks of a wave
  constexpr int kSlot = (BP > BQ ? BP : BQ) * kBk;
  static_assert(EPI != kGated || (!PCOL && TP % 2 == 0), "gate's and up's blocks of a wave are side by side");
  // Five places for an operand's part of one stage.  Separate arrays, so that the
  // compiler can tell a load on its way into one from a read of another.
  __shared__ __align__(16) uint16_t slot0[kSlot];
  __shared__ __align__(16) uint16_t slot1[kSlot];
  __shared__ __align__(16) uint16_t slot2[kSlot];
  __shared__ __align__(16) uint16_t slot3[kSlot];
  __shared__ __align__(16) uint16_t slot4[kSlot];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int id = xcd_order(blockIdx.x, gridDim.x);
  const int which = id >= args.first[2] ? 2 : id >= args.first[1] ? 1 : 0;
  const Product& g = args.of[which];
  const int t = id - args.first[which];
  // Groups of kGroup tiles of q: an XCD's 32 workgroups share their operands' rows.
  const int group = t / (kGroup * g.tiles_p), in = t - group * kGroup * g.tiles_p;
  const int left = g.tiles_q - group * kGroup, height = left < kGroup ? left : kGroup;
  const int tp = in / height, tq = group * kGroup + in - tp * height;
  const int wp = wave / WQ, wq = wave - wp * WQ;

  constexpr int kOwn = EPI == kGated ? BP / 2 : BP;   // values along p of a tile
  const int p0 = tp * kOwn, q0 = tq * BQ;
  using PStager = std::conditional_t<PCOL, ColumnStager<BP, NW>, RowStager<BP, NW>>;
  using QStager = std::conditional_t<QCOL, ColumnStager<BQ, NW>, RowStager<BQ, NW>>;
  auto p_stager = [&] {
    if constexpr (PCOL) {
      return PStager(g.p, g.p_ld, p0, g.p_cols, wave, lane);
    } else {
      constexpr int kMine = PStager::kN * 8;   // rows of a wave
      const int row = wave * kMine;
      if constexpr (EPI == kGated) {
        // LDS rows of wave row wp: half of them gate's, half up's
        constexpr int kHalf = BP / WP / 2;
        static_assert(kHalf % kMine == 0, "a wave stages rows of one of them");
        const int first = p0 + row / (2 * kHalf) * kHalf + row % kHalf;
        return PStager(row / kHalf % 2 ? g.p2 : g.p, g.p_ld, first, g.np - first, g.kk, wave, lane);
      } else {
        return PStager(g.p, g.p_ld, p0 + row, g.np - p0 - row, g.kk, wave, lane);
      }
    }
  };
  auto q_stager = [&] {
    if constexpr (QCOL) {
      return QStager(g.q, g.q_ld, q0, g.q_cols, wave, lane);
    } else {
      const int row = wave * QStager::kN * 8;
      return QStager(g.q, g.q_ld, q0 + row, g.nq - q0 - row, g.kk, wave, lane);
    }
  };
  const PStager sp = p_stager();
  const QStager sq = q_stager();
  constexpr int kP = PStager::kN, kQ = QStager::kN;
  auto load_p = [&](uint16_t* lds, int k0, int i) {
    const bool live = k0 < g.kk;
    if constexpr (PCOL) {
      const bool second = k0 >= g.turn;
      sp.one(lds, second ? g.p2 : g.p, second ? k0 - g.turn : k0, g.p_end, live, i);
    } else {
      sp.one(lds, k0, live, i);
    }
  };
  auto load_q = [&](uint16_t* lds, int k0, int i) {
    const bool live = k0 < g.kk;
    if constexpr (QCOL)
      sq.one(lds, g.q, k0, g.q_end, live, i);
    else
      sq.one(lds, k0, live, i);
  };

  int at_p = PCOL ? lane_at_column<BP>(wp * (BP / WP), lane) : lane_at_row(wp * (BP / WP), lane);
  int at_q = QCOL ? lane_at_column<BQ>(wq * (BQ / WQ), lane) : lane_at_row(wq * (BQ / WQ), lane);
  // A wave's operands for half a stage: two 16-wide pieces of the summed index.
  struct Frags {
    b8 p[2][TP], q[2][TQ];
  };
  constexpr int kReads = 2 * (TP + TQ);
  auto read = [&](Frags& f, const uint16_t* ps, const uint16_t* qs, int half, int n) {
    const int u = n / (TP + TQ), i = n - u * (TP + TQ);
    if (i < TP) {
      if constexpr (PCOL) {
        const char* at = reinterpret_cast<const char*>(ps) + (at_p ^ (i << 6)) + (half * 32 + u * 16) * BP * 2;
        f.p[u][i] = transpose8(at, at + 4 * BP * 2);
      } else {
        f.p[u][i] = *reinterpret_cast<const b8*>(reinterpret_cast<const char*>(ps) + (at_p ^ (half * 64 + u * 32)) + i * 32 * kBk * 2);
      }
    } else {
      const int j = i - TP;
      if constexpr (QCOL) {
        const char* at = reinterpret_cast<const char*>(qs) + (at_q ^ (j << 6)) + (half * 32 + u * 16) * BQ * 2;
        f.q[u][j] = transpose8(at, at + 4 * BQ * 2);
      } else {
        f.q[u][j] = *reinterpret_cast<const b8*>(reinterpret_cast<const char*>(qs) + (at_q ^ (half * 64 + u * 32)) + j * 32 * kBk * 2);
      }
    }
  };

  f16 acc[TP][TQ] = {};
  Frags f0, f1;
  constexpr int kProducts = 2 * TP * TQ;
  // Half a stage: the products of `now`, and between them, evenly, the reads of
  // `then` and the loads of one operand (a wave issues in order: loads in a row hold
  // its products up).  The compiler keeps the groups apart.
  auto half = [&](const auto& load, auto n_loads, const Frags& now, Frags& then, const uint16_t* ps, const uint16_t* qs,
                  int which_half) {
    constexpr int kLoads = decltype(n_loads)::value;
    // Addresses are formed anew: kept over the loop for every slot they would
    // not fit the registers.
    asm volatile("" : "+v"(at_p), "+v"(at_q));
#pragma unroll
    for (int s = 0; s < kLoads; ++s) {
#pragma unroll
      for (int k = s * kProducts / kLoads; k < (s + 1) * kProducts / kLoads; ++k) {
        const int u = k / (TP * TQ), i = (k - u * TP * TQ) / TQ, j = k % TQ;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now.p[u][i], now.q[u][j], acc[i][j], 0, 0, 0);
      }
      load(s);
#pragma unroll
      for (int k = s * kReads / kLoads; k < (s + 1) * kReads / kLoads; ++k) read(then, ps, qs, which_half, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int k0 = 0;
  // One stage: P and Q in ps0 and qs0, the next stage's in ps1 and qs1; the stage
  // after that goes to ps2 and, once every wave has read this one, ps0.
  auto stage = [&](uint16_t* ps0, uint16_t* qs0, uint16_t* ps1, uint16_t* qs1, uint16_t* ps2) {
    half([&](int s) { load_p(ps2, k0 + 2 * kBk, s); }, std::integral_constant<int, kP>(), f0, f1, ps0, qs0, 1);
    // the next stage has arrived (all but ps2's loads), and this one is read
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(kP));
    wave_barrier();
    half([&](int s) { load_q(ps0, k0 + 2 * kBk, s); }, std::integral_constant<int, kQ>(), f1, f0, ps1, qs1, 0);
    return (k0 += kBk) < g.kk;
  };
#pragma unroll
  for (int i = 0; i < kP; ++i) load_p(slot0, 0, i);
#pragma unroll
  for (int i = 0; i < kQ; ++i) load_q(slot1, 0, i);
#pragma unroll
  for (int i = 0; i < kP; ++i) load_p(slot2, kBk, i);
#pragma unroll
  for (int i = 0; i < kQ; ++i) load_q(slot3, kBk, i);
  __builtin_amdgcn_s_waitcnt(wait_vm(kP + kQ));
  wave_barrier();
#pragma unroll
  for (int k = 0; k < kReads; ++k) read(f0, slot0, slot1, 0, k);
  while (stage(slot0, slot1, slot2, slot3, slot4) && stage(slot2, slot3, slot4, slot0, slot1) &&
         stage(slot4, slot0, slot1, slot2, slot3) && stage(slot1, slot2, slot3, slot4, slot0) &&
         stage(slot3, slot4, slot0, slot1, slot2)) {
  }
  __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));   // nothing is on its way into LDS any more

  // Results.  The lane's token (or row) and its neighbours along p.
  const int lq = lane & 31, lp = (lane >> 5) * 8;
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    const int q = q0 + wq * (BQ / WQ) + j * 32 + lq;
    if constexpr (EPI == kStore) {
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        float v[2][8];
        octets(acc[i][j], v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = p0 + wp * (BP / WP) + i * 32 + h * 16 + lp;
          if (q < g.nq && p < g.out_cols) store8(g.out + q * g.out_ld + p, v[h], g.out_vec, g.out_cols - p);
        }
      }
    } else if constexpr (EPI == kGated) {
#pragma unroll
      for (int i = 0; i < TP / 2; ++i) {
        float a[2][8], b[2][8], v[2][8];
        octets(acc[i][j], a);
        octets(acc[i + TP / 2][j], b);
        const int pb = p0 + wp * (BP / WP / 2) + i * 32;   // the block's first: a multiple of 32
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int n = 0; n < 8; ++n) v[h][n] = activate(a[h][n], args.act) * b[h][n];
          const int p = pb + h * 16 + lp;
          if (q < g.nq && p < g.out_cols) store8(g.out + q * g.out_ld + p, v[h], 1, 8);   // the workspace's: whole octets
        }
        if (args.save) {
          // 32 neighbours are one block: the lane's 16 and those of lane ^ 32
          auto keep = [&](const float (&x)[2][8], const Act8Rows& to) {
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const uint32_t m = __float_as_uint(x[h][n]) & 0x7FFFFFFFu;
                top = m > top ? m : top;
              }
            const uint32_t other = __shfl_xor(top, 32, 64);
            top = other > top ? other : top;
            const uint32_t byte = act8_scale_byte(top, args.format);
            const float inverse = act8_inverse(byte);
            if (q >= g.nq) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int p = pb + h * 16 + lp;
              const u32x2 w = {act8_codes(x[h][0], x[h][1], x[h][2], x[h][3], inverse, args.format),
                               act8_codes(x[h][4], x[h][5], x[h][6], x[h][7], inverse, args.format)};
              if (p < g.np) store_codes8(to.codes + static_cast<int64_t>(q) * g.np + p, w, g.np - p);
            }
            if (lane < 32 && pb < g.np) to.scales[static_cast<int64_t>(q) * args.blocks + (pb >> 5)] = static_cast<uint8_t>(byte);
          };
          keep(a, args.gate);
          keep(b, args.up);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        float dh[2][8];
        octets(acc[i][j], dh);
        const int pb = p0 + wp * (BP / WP) + i * 32;
        if (q >= g.nq || pb >= g.out_cols) continue;
        const bool some = pb < g.np;   // else: the pitch's zeros
        const int64_t at = static_cast<int64_t>(q) * args.blocks + (pb >> 5);
        const float sg = some ? act8_scale(args.gate.scales[at]) : 0.0f, su = some ? act8_scale(args.up.scales[at]) : 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = pb + h * 16 + lp;
          const u32x2 wg = load_codes8(args.gate.codes + static_cast<int64_t>(q) * g.np + p, g.np - p);
          const u32x2 wu = load_codes8(args.up.codes + static_cast<int64_t>(q) * g.np + p, g.np - p);
          float dg[8], du[8], hv[8];
#pragma unroll
          for (int n4 = 0; n4 < 2; ++n4) {
            float gv[4], uv[4];
            act8_values(wg[n4], sg, args.format, gv);
            act8_values(wu[n4], su, args.format, uv);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int k = n4 * 4 + n;
              float a, slope;
              activate_slope(gv[n], args.act, a, slope);
              // past the matrix's columns the sums are of something else
              const bool in_row = p + k < g.np;
              dg[k] = in_row ? dh[h][k] * uv[n] * slope : 0.0f;
              du[k] = in_row ? dh[h][k] * a : 0.0f;
              hv[k] = in_row ? a * uv[n] : 0.0f;
            }
          }
          if (p < g.out_cols) {   // the workspace's: whole octets
            store8(g.out + q * g.out_ld + p, dg, 1, 8);
            store8(args.du + q * g.out_ld + p, du, 1, 8);
            store8(args.h + q * args.h_ld + p, hv, 1, 8);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ operands that the products cannot take
// A matrix whose rows are not 16-byte aligned, or end inside a stage: copied to the
// workspace with a pitch of whole stages, zeros behind each row.
struct PackArgs {
  const uint16_t* from;
  int64_t ld;
  uint16_t* to;
  int64_t pitch;
  int64_t rows;
  int cols;
};
__global__ __launch_bounds__(256) void ffn_pack_kernel(PackArgs a) {
  const int64_t pieces = a.pitch / 8, n = a.rows * pieces;
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; k < n; k += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = k / pieces;
    const int c = static_cast<int>(k - r * pieces) * 8;
    const uint16_t* from = a.from + r * a.ld + c;
    u32x4 w = {};
    if (c + 8 <= a.cols) {
      __builtin_memcpy(&w, from, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < a.cols) w[q >> 1] |= static_cast<uint32_t>(from[q]) << ((q & 1) * 16);
    }
    *reinterpret_cast<u32x4*>(a.to + r * a.pitch + c) = w;
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

hipError_t pack(const uint16_t* from, int64_t ld, uint16_t* to, int64_t pitch, int64_t rows, int64_t cols, hipStream_t s) {
  const PackArgs a = {from, ld, to, pitch, rows, static_cast<int>(cols)};
  const int64_t n = rows * pitch / 8;
  const int64_t most = 4096;
  const int64_t grid = (n + 255) / 256;
  hipLaunchKernelGGL(ffn_pack_kernel, dim3(static_cast<unsigned>(grid < most ? grid : most)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int BP, int BQ, int WP, int WQ, bool PCOL, bool QCOL, Epilogue EPI>
hipError_t tiles(Products a, int n, hipStream_t s) {
  int64_t total = 0;
  for (int k = 0; k < 3; ++k) {
    a.first[k] = k < n ? static_cast<int>(total) : 0x7FFFFFFF;
    if (k >= n) continue;
    Product& g = a.of[k];
    const int own = EPI == kGated ? BP / 2 : BP;
    const int columns = g.out_cols > g.np ? g.out_cols : g.np;
    g.tiles_p = (columns + own - 1) / own;
    g.tiles_q = (g.nq + BQ - 1) / BQ;
    total += static_cast<int64_t>(g.tiles_p) * g.tiles_q;
  }
  hipLaunchKernelGGL((ffn_product_kernel<BP, BQ, WP, WQ, PCOL, QCOL, EPI>), dim3(static_cast<unsigned>(total)), dim3(WP * WQ * 64),
                     0, s, a);
  return hipGetLastError();
}

template <bool PCOL, bool QCOL, Epilogue EPI>
hipError_t product(const Products& a, int n, hipStream_t s) {
  int64_t large = 0;
  for (int k = 0; k < n; ++k) {
    const int64_t own = EPI == kGated ? 128 : 256;
    large += (a.of[k].np + own - 1) / own * ((a.of[k].nq + 255) / 256);
  }
  if (large >= 256) return tiles<256, 256, 2, 4, PCOL, QCOL, EPI>(a, n, s);
  return tiles<128, 128, 2, 2, PCOL, QCOL, EPI>(a, n, s);
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
  int64_t n = bytes(tokens * dp);                                   // x or dy
  if (backward)
    n += bytes(tokens * 2 * fp) + bytes(tokens * fp) + bytes(tokens * dp);
  else
    n += bytes(tokens * fp);
  if (unaligned || model % kPad || hidden % kPad) n += 2 * bytes(hidden * dp) + bytes(model * fp);
  return n;
}

bool ffn_weights_aligned(const FfnParams& p) {
  return aligned(p.w_gate, p.model) && aligned(p.w_up, p.model) && aligned(p.w_down, p.hidden);
}

hipError_t launch_ffn_forward(const FfnParams& p, hipStream_t s) {
  const int64_t t = p.tokens, d = p.model, f = p.hidden, dp = pad_up(d), fp = pad_up(f);
  Carver ws = {static_cast<char*>(p.workspace)};
  uint16_t* h = ws.take(t * fp);
  uint16_t* x_room = ws.take(t * dp);
  Matrix x = {p.x, p.x_row}, gate = {p.w_gate, d}, up = {p.w_up, d}, down = {p.w_down, f};
  if (!aligned(x.at, x.ld) || d % kPad) {
    ZERO_TRY(pack(x.at, x.ld, x_room, dp, t, d, s));
    x = {x_room, dp};
  }
  if (!ffn_weights_aligned(p) || d % kPad || f % kPad) {
    uint16_t* room[3] = {ws.take(f * dp), ws.take(f * dp), ws.take(d * fp)};
    ZERO_TRY(pack(gate.at, d, room[0], dp, f, d, s));
    ZERO_TRY(pack(up.at, d, room[1], dp, f, d, s));
    ZERO_TRY(pack(down.at, f, room[2], fp, d, f, s));
    gate = {room[0], dp};
    up = {room[1], dp};
    down = {room[2], fp};
  }
  if (p.save) {
    Act8Params a = {const_cast<uint16_t*>(p.x), p.x_row, t, d, p.ckpt.x_codes, p.ckpt.x_scales, p.ckpt.format, 0};
    ZERO_TRY(launch_act8_save(a, s));
  }
  Products a = {};
  a.gate = {p.ckpt.gate_codes, p.ckpt.gate_scales};
  a.up = {p.ckpt.up_codes, p.ckpt.up_scales};
  a.blocks = static_cast<int>((f + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK);
  a.format = p.ckpt.format;
  a.act = p.activation;
  a.save = p.save;
  Product& g = a.of[0];
  g.p = gate.at;
  g.p2 = up.at;
  g.p_ld = gate.ld;
  g.q = x.at;
  g.q_ld = x.ld;
  g.np = static_cast<int>(f);
  g.nq = static_cast<int>(t);
  g.kk = static_cast<int>(dp);
  g.out = h;
  g.out_ld = fp;
  g.out_cols = static_cast<int>(fp);
  g.out_vec = 1;
  ZERO_TRY((product<false, false, kGated>(a, 1, s)));
  Products b = {};
  Product& y = b.of[0];
  y.p = down.at;
  y.p_ld = down.ld;
  y.q = h;
  y.q_ld = fp;
  y.np = static_cast<int>(d);
  y.nq = static_cast<int>(t);
  y.kk = static_cast<int>(fp);
  y.out = p.y;
  y.out_ld = p.y_row;
  y.out_cols = static_cast<int>(d);
  y.out_vec = aligned(p.y, p.y_row);
  return product<false, false, kStore>(b, 1, s);
}

hipError_t launch_ffn_backward(const FfnParams& p, hipStream_t s) {
  const int64_t t = p.tokens, d = p.model, f = p.hidden, dp = pad_up(d), fp = pad_up(f);
  Carver ws = {static_cast<char*>(p.workspace)};
  uint16_t* dgu = ws.take(t * 2 * fp);
  uint16_t* h = ws.take(t * fp);
  uint16_t* x = ws.take(t * dp);
  uint16_t* dy_room = ws.take(t * dp);
  Matrix dy = {p.x, p.x_row}, gate = {p.w_gate, d}, up = {p.w_up, d}, down = {p.w_down, f};
  int dy_cols = static_cast<int>(d), w_cols = static_cast<int>(d), down_cols = static_cast<int>(f);
  if (!aligned(dy.at, dy.ld) || d % kPad) {
    ZERO_TRY(pack(dy.at, dy.ld, dy_room, dp, t, d, s));
    dy = {dy_room, dp};
    dy_cols = static_cast<int>(dp);
  }
  if (!ffn_weights_aligned(p) || d % kPad || f % kPad) {
    uint16_t* room[3] = {ws.take(f * dp), ws.take(f * dp), ws.take(d * fp)};
    ZERO_TRY(pack(gate.at, d, room[0], dp, f, d, s));
    ZERO_TRY(pack(up.at, d, room[1], dp, f, d, s));
    ZERO_TRY(pack(down.at, f, room[2], fp, d, f, s));
    gate = {room[0], dp};
    up = {room[1], dp};
    down = {room[2], fp};
    w_cols = static_cast<int>(dp);
    down_cols = static_cast<int>(fp);
  }
  Act8Params held = {x, dp, t, d, p.ckpt.x_codes, p.ckpt.x_scales, p.ckpt.format, 0};
  ZERO_TRY(launch_act8_load(held, s));
  // dh, and from it dg, du and h
  Products a = {};
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
  g.out_vec = 1;
  ZERO_TRY((product<true, false, kSlopes>(a, 1, s)));
  if (p.y) {   // dx
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
    y.out_vec = aligned(p.y, p.y_row);
    ZERO_TRY((product<true, false, kStore>(b, 1, s)));
  }
  Products c = {};
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
    w.out_vec = aligned(w.out, w.out_ld);
  }
  return product<true, true, kStore>(c, 3, s);
}

}  // namespace zero
