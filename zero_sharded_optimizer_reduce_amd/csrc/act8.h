// Activations in 8 bits (include/zero.h, zero_act8_save): device helpers shared by
// the checkpoint kernels (act8.hip) and the feed-forward products (ffn.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/zero.h"

namespace zero {
namespace {

constexpr uint32_t kAct8NaN = 255;   // the scale byte of a block that has none

// The scale byte (exponent + 127) of a block whose largest magnitude has the
// given bits: the least power of two, from 2^-126 on, with which it fits 127 or
// 448.  127 = 1.984375 * 2^6 and 448 = 1.75 * 2^8: the exponent field less 6 or 8,
// and one more where the fraction is above theirs, which the addition carries.
// Where it carries out of FP32's largest exponent the nearest code could stand for
// 2^128: no scale, as for an infinity or a NaN, which the same comparison finds.
__device__ __forceinline__ uint32_t act8_scale_byte(uint32_t top, int format) {
  const uint32_t k = (top + (format == ZERO_ACT8_INT8 ? 0x7FFFFFu - 0x7E0000u : 0x7FFFFFu - 0x600000u)) >> 23;
  const int e = static_cast<int>(k) - (format == ZERO_ACT8_INT8 ? 6 : 8);
  return k >= 255 ? kAct8NaN : e < 1 ? 1u : static_cast<uint32_t>(e);
}

// 2^-(byte - 127), exact: the byte of a block is at most 254 - 6.  0 for a block
// without a scale, whose codes then are zeros.
__device__ __forceinline__ float act8_inverse(uint32_t byte) {
  return byte == kAct8NaN ? 0.0f : __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ float act8_scale(uint32_t byte) {
  return __uint_as_float(byte == kAct8NaN ? 0x7FC00000u : byte ? byte << 23 : 0x00400000u);
}

// Four codes, lowest byte first.  Whole numbers: adding 1.5 * 2^23 rounds to the
// nearest even and leaves the two's complement in the low byte.
__device__ __forceinline__ uint32_t act8_int8(float a, float b, float c, float d) {
  constexpr float kRound = 12582912.0f;
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b + kRound), __float_as_uint(a + kRound), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d + kRound), __float_as_uint(c + kRound), 0x04000C0Cu);
  return lo | hi;
}
__device__ __forceinline__ uint32_t act8_e4m3(float a, float b, float c, float d) {
  uint32_t w = 0;
#ifdef __HIP_DEVICE_COMPILE__
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
#endif
  return w;
}

// N codes of N values (N a multiple of 4).  A block without a scale (inverse 0) has
// codes of 0 and reads back as NaN.
template <int N>
__device__ __forceinline__ void act8_codes(const float (&x)[N], float inverse, int format, uint32_t (&w)[N / 4]) {
  float v[N];
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = x[q] * inverse;
  if (format == ZERO_ACT8_INT8) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) w[q] = act8_int8(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) w[q] = act8_e4m3(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  }
#pragma unroll
  for (int q = 0; q < N / 4; ++q) w[q] = inverse == 0.0f ? 0u : w[q];
}

// What codes stand for before the scale: exact.
template <int N>
__device__ __forceinline__ void act8_numbers_int8(const uint32_t (&w)[N / 4], float (&v)[N]) {
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = static_cast<float>(static_cast<int8_t>(w[q / 4] >> (8 * (q & 3))));
}
template <int N>
__device__ __forceinline__ void act8_numbers_e4m3(const uint32_t (&w)[N / 4], float (&v)[N]) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[q]), false);
    const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[q]), true);
    v[4 * q] = lo.x;
    v[4 * q + 1] = lo.y;
    v[4 * q + 2] = hi.x;
    v[4 * q + 3] = hi.y;
  }
#endif
}

}  // namespace
}  // namespace zero
