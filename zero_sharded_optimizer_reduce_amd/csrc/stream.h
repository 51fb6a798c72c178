// What the HBM-streaming kernels share (kernels.hip, muon.hip): vector types,
// BF16 conversions, non-temporal accesses, the tile's output stores, the
// weighted rank sum of one lane and the launch shape.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>

#include "../../include/zero.h"

#pragma clang fp contract(off)

namespace zero {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256;

// ------------------------------------------------------------------ helpers
// A BF16 value is the high half of a binary32, so widening is a shift (exact).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_at(const uint16_t* p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

// Round-to-nearest-even binary32 -> bfloat16 (gfx950 converts in hardware).
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  return static_cast<uint32_t>(to_bf16(lo)) | (static_cast<uint32_t>(to_bf16(hi)) << 16);
}

template <typename T>
__device__ __forceinline__ T ld_nt(const T* p) { return __builtin_nontemporal_load(p); }
template <typename T>
__device__ __forceinline__ void st_nt(T v, T* p) { __builtin_nontemporal_store(v, p); }

// Streamed output stores with a cache policy the compiler's builtin cannot
// set.  With SC1 a workgroup writes its tile through a buffer descriptor based
// at the tile's first element (workgroup-uniform, so the descriptor lives in
// scalar registers and every lane offset is below 4 KiB), with the store bits
// nt and sc1 (device scope); without it the plain non-temporal store is used.
// Same-box A/B on MI355X: with sc1 the update, the fused kernel (without the
// gradient output), the accumulate-mode reduce and the gather ran 1.0-3.6%
// faster; the plain reduce, the FP32-contribution reduce and the fused kernel
// storing the gradient ran 0.4-1.8% slower, so they keep the plain store
// (system scope, sc0|sc1, measured the same as sc1).
// The buffer forms are compiler intrinsics (not inline assembly), so the
// compiler schedules them and resolves their register hazards.
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
constexpr int kRawBufferFlags = 0x00020000;   // dword 3 of a raw buffer descriptor: 32-bit data format
constexpr int kStoreNtSc1 = 2 | 16;           // cache-policy operand: nt | sc1

template <typename T, bool SC1>
struct TileOut {
  T* global;                  // the tile's first element
  __amdgpu_buffer_rsrc_t rsrc;
  __device__ __forceinline__ TileOut(T* base, int64_t count) : global(base) {
    if constexpr (SC1)
      rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, static_cast<int>(count * static_cast<int64_t>(sizeof(T))),
                                               kRawBufferFlags);
  }
  // element j of the tile (0 <= j < count)
  __device__ __forceinline__ void store(T v, int j) const {
    if constexpr (!SC1) {
      __builtin_nontemporal_store(v, global + j);
    } else if constexpr (sizeof(T) == 16) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), rsrc, j * 16, 0, kStoreNtSc1);
    } else if constexpr (sizeof(T) == 8) {
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(i32x2, v), rsrc, j * 8, 0, kStoreNtSc1);
    } else {
      __builtin_nontemporal_store(v, global + j);
    }
  }
};

// Elements of the tile that starts `left` elements before the end of an array.
__device__ __forceinline__ int64_t tile_len(int64_t left, int bs) { return left < bs ? left : bs; }

// The 4 reduced values of one lane; x[r] holds rank r's 4 BF16 values.
template <int NMAX>
__device__ __forceinline__ f32x4 reduce4(const u32x2 (&x)[NMAX], int n, const float* w) {
  const float w0 = w[0];
  float a0 = w0 * bf16_lo(x[0].x), a1 = w0 * bf16_hi(x[0].x);
  float a2 = w0 * bf16_lo(x[0].y), a3 = w0 * bf16_hi(x[0].y);
#pragma unroll
  for (int r = 1; r < NMAX; ++r) {
    if (r < n) {
      const float wr = w[r];
      a0 = a0 + wr * bf16_lo(x[r].x);
      a1 = a1 + wr * bf16_hi(x[r].x);
      a2 = a2 + wr * bf16_lo(x[r].y);
      a3 = a3 + wr * bf16_hi(x[r].y);
    }
  }
  return f32x4{a0, a1, a2, a3};
}

template <int NMAX>
__device__ __forceinline__ f32x4 reduce4(const f32x4 (&x)[NMAX], int n, const float* w) {
  f32x4 a = w[0] * x[0];
#pragma unroll
  for (int r = 1; r < NMAX; ++r)
    if (r < n) a = a + w[r] * x[r];
  return a;
}

// -------------------------------------------------------------- launch shape
// Launch shape, chosen by measurement on MI355X: one tile per workgroup (the
// grid covers the whole array).  The dispatcher issues workgroups in index
// order, so the tiles in flight at any moment form a narrow moving window of
// each array, which keeps HBM row locality high; a persistent grid that
// sweeps the arrays in a grid-stride loop measured 5-15% slower on every
// kernel here.  The grid-stride loops stay so that a capped grid (the
// ZERO_BLOCKS_PER_CU tuning override, or arrays beyond kMaxGridX tiles) is
// still covered.
constexpr int64_t kMaxGridX = int64_t(1) << 24;

int blocks_per_cu() {
  static int v = [] {
    const char* s = getenv("ZERO_BLOCKS_PER_CU");
    int x = s ? atoi(s) : 0;
    return (x >= 1 && x <= 64) ? x : 0;
  }();
  return v;
}

// Compute units of the current device, cached per device (calls from several
// threads may fill a slot concurrently; they store the same value).
int device_cus() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int cus = cache[dev].load(std::memory_order_relaxed);
  if (cus == 0) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
      cus = 256;
    cache[dev].store(cus, std::memory_order_relaxed);
  }
  return cus;
}

// Blocks along x for `units` work items per owner, each block covering bs of
// them per loop iteration.
unsigned grid_x(int64_t units, int n_y, int bs = kBlock) {
  const int64_t per_iter = bs;
  int64_t need = (units + per_iter - 1) / per_iter;
  int64_t cap = kMaxGridX;
  if (blocks_per_cu() > 0) cap = static_cast<int64_t>(device_cus()) * blocks_per_cu() / (n_y > 0 ? n_y : 1);
  if (cap < 1) cap = 1;
  if (need > cap) need = cap;
  if (need < 1) need = 1;
  return static_cast<unsigned>(need);
}

}  // namespace
}  // namespace zero
