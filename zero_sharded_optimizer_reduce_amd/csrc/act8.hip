// gfx950 kernels of zero_act8_save and zero_act8_load: a matrix of activations in 8
// bits a value and a power of two per 32 neighbours of a row, and back.
//
// Both move data and are bound by HBM: 3.03 bytes a BF16 value.  A lane takes 8
// neighbours ("unit"): 16 bytes of BF16, 8 bytes of codes; the four lanes of a block
// find its largest magnitude with two exchanges.
// 16384 x 14336 BF16, passes in a row: saved and read back in 230 us, read back alone in 116 (6.1 TB/s).  Two
// units a lane, on their way together; least times of single launches: with one 124 and 122 us, with
// two 118 and 123, with four 128 and 122, with eight 135 and 126; storing past the caches brings
// two to 114 and 94 to 98, of which passes in a row keep the 116 (their median).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "act8.h"
#include "kernels.h"

#pragma clang fp contract(off)

namespace zero {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kUnit = 8;
constexpr int kEach = 2;                       // units of a lane
constexpr int kSpan = kThreads * kEach;        // units of a workgroup

// A matrix as units: row r has `per_row` of them, whole blocks of four.
struct Units {
  int64_t total;      // rows * per_row
  int64_t rows, cols;
  uint32_t per_row;
  uint32_t magic;     // ceil(2^32 / per_row)
};

// Where unit (workgroup's first + t) lies.  The workgroup's first is divided once; from
// there on, rows of over kSpan units are passed once at most, and for shorter ones
// the product with the reciprocal is exact (t < 2 kSpan: t * per_row < 2^32).
struct Place {
  int64_t row;
  uint32_t unit;
};
__device__ __forceinline__ Place place_of(const Units& u, int64_t row0, uint32_t unit0, uint32_t t) {
  const uint32_t at = unit0 + t;
  const uint32_t down = u.per_row > kSpan ? (at >= u.per_row ? 1u : 0u) : __umulhi(at, u.magic);
  return {row0 + down, at - down * u.per_row};
}

template <typename T>
__device__ __forceinline__ T load_any(const void* p) {   // at any address: the memory takes them
  T v;
  __builtin_memcpy(&v, p, sizeof v);
  return v;
}
// Past the caches: what is written is read much later.
__device__ __forceinline__ void stream16(void* p, u32x4 v) {
  typedef uint32_t any __attribute__((ext_vector_type(4), aligned(2)));
  __builtin_nontemporal_store(static_cast<any>(v), static_cast<any*>(p));
}
__device__ __forceinline__ void stream8(void* p, u32x2 v) {
  typedef uint32_t any __attribute__((ext_vector_type(2), aligned(1)));
  __builtin_nontemporal_store(static_cast<any>(v), static_cast<any*>(p));
}

// The unit's values, zeros past the row's end.
template <bool F32>
__device__ __forceinline__ void load_unit(const void* row, int64_t at, int64_t cols, float (&v)[kUnit]) {
  if (at + kUnit <= cols) {
    if constexpr (F32) {
      const float* p = static_cast<const float*>(row) + at;
      const u32x4 a = load_any<u32x4>(p), b = load_any<u32x4>(p + 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = __uint_as_float(a[q]);
        v[4 + q] = __uint_as_float(b[q]);
      }
    } else {
      const u32x4 w = load_any<u32x4>(static_cast<const uint16_t*>(row) + at);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < kUnit; ++q) {
    v[q] = 0.0f;
    if (at + q < cols) {
      if constexpr (F32)
        v[q] = static_cast<const float*>(row)[at + q];
      else
        v[q] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[at + q]) << 16);
    }
  }
}

struct SaveArgs {
  Units u;
  const void* x;
  int64_t x_row;
  uint8_t* codes;
  uint8_t* scales;
  int64_t blocks;     // of a row
  int format;
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void act8_save_kernel(SaveArgs a) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSpan;
  const int64_t row0 = first / a.u.per_row;
  const uint32_t unit0 = static_cast<uint32_t>(first - row0 * a.u.per_row);
  float v[kEach][kUnit];
  Place at[kEach];
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const uint32_t t = n * kThreads + threadIdx.x;
    at[n] = place_of(a.u, row0, unit0, t);
#pragma unroll
    for (int q = 0; q < kUnit; ++q) v[n][q] = 0.0f;
    if (first + t < a.u.total) {
      const char* row = static_cast<const char*>(a.x) + at[n].row * a.x_row * (F32 ? 4 : 2);
      load_unit<F32>(row, static_cast<int64_t>(at[n].unit) * kUnit, a.u.cols, v[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    uint32_t top = 0;   // magnitudes as whole numbers: NaN is above infinity
#pragma unroll
    for (int q = 0; q < kUnit; ++q) {
      const uint32_t m = __float_as_uint(v[n][q]) & 0x7FFFFFFFu;
      top = m > top ? m : top;
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      const uint32_t m = __shfl_xor(top, off, 64);
      top = m > top ? m : top;
    }
    const uint32_t t = n * kThreads + threadIdx.x;
    if (first + t >= a.u.total) continue;
    const uint32_t byte = act8_scale_byte(top, a.format);
    const float inverse = act8_inverse(byte);
    uint32_t words[2];
    act8_codes(v[n], inverse, a.format, words);
    const u32x2 w = {words[0], words[1]};
    const int64_t c = static_cast<int64_t>(at[n].unit) * kUnit;
    uint8_t* out = a.codes + at[n].row * a.u.cols + c;
    if (c + kUnit <= a.u.cols) {
      stream8(out, w);
    } else {
#pragma unroll
      for (int q = 0; q < kUnit; ++q)
        if (c + q < a.u.cols) out[q] = static_cast<uint8_t>(w[q >> 2] >> ((q & 3) * 8));
    }
    if ((at[n].unit & 3) == 0) a.scales[at[n].row * a.blocks + (at[n].unit >> 2)] = static_cast<uint8_t>(byte);
  }
}

struct LoadArgs {
  Units u;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t blocks;
  void* out;
  int64_t out_row;
  int format;
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void act8_load_kernel(LoadArgs a) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSpan;
  const int64_t row0 = first / a.u.per_row;
  const uint32_t unit0 = static_cast<uint32_t>(first - row0 * a.u.per_row);
  u32x2 w[kEach];
  uint32_t byte[kEach];
  Place at[kEach];
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const uint32_t t = n * kThreads + threadIdx.x;
    at[n] = place_of(a.u, row0, unit0, t);
    w[n] = u32x2{};
    byte[n] = 0;
    if (first + t >= a.u.total) continue;
    const int64_t c = static_cast<int64_t>(at[n].unit) * kUnit;
    if (c >= a.u.cols) continue;   // a whole unit past the row's end
    const uint8_t* in = a.codes + at[n].row * a.u.cols + c;
    byte[n] = a.scales[at[n].row * a.blocks + (at[n].unit >> 2)];
    if (c + kUnit <= a.u.cols) {
      w[n] = load_any<u32x2>(in);
    } else {
#pragma unroll
      for (int q = 0; q < kUnit; ++q)
        if (c + q < a.u.cols) w[n][q >> 2] |= static_cast<uint32_t>(in[q]) << ((q & 3) * 8);
    }
  }
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    const uint32_t t = n * kThreads + threadIdx.x;
    const int64_t c = static_cast<int64_t>(at[n].unit) * kUnit;
    if (first + t >= a.u.total || c >= a.u.cols) continue;
    const float scale = act8_scale(byte[n]);
    const uint32_t words[2] = {w[n].x, w[n].y};
    float v[kUnit];
    if (a.format == ZERO_ACT8_INT8)
      act8_numbers_int8(words, v);
    else
      act8_numbers_e4m3(words, v);
#pragma unroll
    for (int q = 0; q < kUnit; ++q) v[q] *= scale;   // exact
    if constexpr (F32) {
      float* out = static_cast<float*>(a.out) + at[n].row * a.out_row + c;
      if (c + kUnit <= a.u.cols) {
        stream16(out, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
        stream16(out + 4, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
      } else {
#pragma unroll
        for (int q = 0; q < kUnit; ++q)
          if (c + q < a.u.cols) out[q] = v[q];
      }
    } else {
      // whole numbers and e4m3 have less than BF16's 8 bits: rounded only below its normal values
      uint16_t* out = static_cast<uint16_t*>(a.out) + at[n].row * a.out_row + c;
      typedef __bf16 b8 __attribute__((ext_vector_type(8)));
      typedef float f8 __attribute__((ext_vector_type(8)));
      const b8 o = __builtin_convertvector((f8{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}), b8);
      if (c + kUnit <= a.u.cols) {
        stream16(out, __builtin_bit_cast(u32x4, o));
      } else {
#pragma unroll
        for (int q = 0; q < kUnit; ++q)
          if (c + q < a.u.cols) out[q] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[q]));
      }
    }
  }
}

// One after the other in memory and whole blocks: one row.
Units units_of(int64_t rows, int64_t cols, bool one_row) {
  Units u;
  if (one_row) {
    cols *= rows;
    rows = 1;
  }
  u.rows = rows;
  u.cols = cols;
  const int64_t per_row = (cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK * (ZERO_ACT8_BLOCK / kUnit);
  u.per_row = static_cast<uint32_t>(per_row);
  u.magic = static_cast<uint32_t>(((1ull << 32) + per_row - 1) / per_row);
  u.total = rows * per_row;
  return u;
}

}  // namespace

hipError_t launch_act8_save(const Act8Params& p, hipStream_t stream) {
  SaveArgs a;
  const bool one_row = p.row == p.cols && p.cols % ZERO_ACT8_BLOCK == 0 && p.rows * p.cols < ZERO_ACT8_MAX_COLS;
  a.u = units_of(p.rows, p.cols, one_row);
  a.x = p.values;
  a.x_row = p.row;
  a.codes = p.codes;
  a.scales = p.scales;
  a.blocks = (a.u.cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK;
  a.format = p.format;
  const dim3 grid(static_cast<unsigned>((a.u.total + kSpan - 1) / kSpan));
  if (p.f32)
    hipLaunchKernelGGL(act8_save_kernel<true>, grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(act8_save_kernel<false>, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_act8_load(const Act8Params& p, hipStream_t stream) {
  LoadArgs a;
  const bool one_row = p.row == p.cols && p.cols % ZERO_ACT8_BLOCK == 0 && p.rows * p.cols < ZERO_ACT8_MAX_COLS;
  a.u = units_of(p.rows, p.cols, one_row);
  a.codes = p.codes;
  a.scales = p.scales;
  a.blocks = (a.u.cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK;
  a.out = p.values;
  a.out_row = p.row;
  a.format = p.format;
  const dim3 grid(static_cast<unsigned>((a.u.total + kSpan - 1) / kSpan));
  if (p.f32)
    hipLaunchKernelGGL(act8_load_kernel<true>, grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(act8_load_kernel<false>, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace zero
