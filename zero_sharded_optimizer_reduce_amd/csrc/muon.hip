// gfx950 streaming kernels of the Muon step: the momentum step of an owner's
// shard (alone, or fused with the reduce-scatter) and the owner update that
// applies the orthogonalised directions.  Like the kernels of kernels.hip they
// move each byte once and are bound by HBM: 14, 2N + 10 and 12 bytes per
// element against at most 2N + 6 binary32 operations.
//
// Floating point: contraction off, every multiply and add its own binary32
// rounding, in the order written at each kernel.
#include <hip/hip_runtime.h>

#include "kernels.h"
#include "stream.h"

#pragma clang fp contract(off)

namespace zero {
namespace {

// 4 BF16 values whose address is only 2-byte aligned: an owner's slice of a
// rank's contribution starts anywhere.  gfx950 reads them with one 8-byte
// load at any alignment, so the vector path needs no alignment of its inputs.
typedef u32x2 u32x2_any __attribute__((aligned(2)));
__device__ __forceinline__ u32x2 ld_nt_any(const u32x2_any* p) { return __builtin_nontemporal_load(p); }

// The momentum step of one element: m' = b*m + (1-b)*g, direction u = m', or
// with Nesterov's look-ahead u = (1-b)*g + b*m'.
__device__ __forceinline__ float momentum_elem(float& m, float g, const MuonScalars& s) {
  const float fresh = s.one_minus_momentum * g;
  m = s.momentum * m + fresh;
  return s.nesterov ? fresh + s.momentum * m : m;
}

__device__ __forceinline__ u32x2 momentum4(f32x4& m, f32x4 g, const MuonScalars& s) {
  float me[4] = {m.x, m.y, m.z, m.w};
  const float ge[4] = {g.x, g.y, g.z, g.w};
  float u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = momentum_elem(me[e], ge[e], s);
  m = f32x4{me[0], me[1], me[2], me[3]};
  return u32x2{to_bf16x2(u[0], u[1]), to_bf16x2(u[2], u[3])};
}

// ------------------------------------------------------------- momentum step
// 14 bytes per element: reads g and m, writes m and the BF16 direction.
template <bool SC, int BS>
__global__ __launch_bounds__(BS) void momentum_vec_kernel(MomentumParams a) {
  const int64_t nvec = a.n >> 2;
  f32x4* __restrict__ M = reinterpret_cast<f32x4*>(a.m);
  u32x2* __restrict__ U = reinterpret_cast<u32x2*>(a.u);
  const f32x4* __restrict__ G = reinterpret_cast<const f32x4*>(a.g);
  const float c = SC ? *a.gscale : 1.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * BS;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * BS; tile < nvec; tile += step) {
    const int64_t i = tile + threadIdx.x;
    if (i < nvec) {
      const int64_t len = tile_len(nvec - tile, BS);
      const TileOut<f32x4, true> oM(M + tile, len);
      const TileOut<u32x2, true> oU(U + tile, len);
      f32x4 g = ld_nt(G + i);
      f32x4 m = ld_nt(M + i);
      if (SC) g = g * c;
      const u32x2 u = momentum4(m, g, a.s);
      oM.store(m, threadIdx.x);
      oU.store(u, threadIdx.x);
    }
  }
  const int64_t tail = a.n - (nvec << 2);
  if (blockIdx.x == 0 && threadIdx.x < tail) {
    const int64_t i = (nvec << 2) + threadIdx.x;
    float m = a.m[i];
    const float u = momentum_elem(m, SC ? a.g[i] * c : a.g[i], a.s);
    a.m[i] = m;
    a.u[i] = to_bf16(u);
  }
}

// Element at a time, for FP32 pointers that are not 16-byte aligned.
template <bool SC>
__global__ __launch_bounds__(kBlock) void momentum_scalar_kernel(MomentumParams a) {
  const float c = SC ? *a.gscale : 1.0f;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < a.n;
       i += static_cast<int64_t>(gridDim.x) * kBlock) {
    float m = a.m[i];
    const float u = momentum_elem(m, SC ? a.g[i] * c : a.g[i], a.s);
    a.m[i] = m;
    a.u[i] = to_bf16(u);
  }
}

// ------------------------------------------------- reduce-scatter + momentum
// One owner: the reduced gradient of its slice is formed in registers in rank
// order (the reduce kernel's arithmetic; ACC: gacc + red), and the momentum
// step follows, so the gradient is never stored.  2N + 10 bytes per element
// (+4 with ACC) against 2N + 18 for the two calls.
template <int N, bool ACC>
__device__ __forceinline__ float reduce1(const ReduceMomentumParams& p, int n, int64_t i) {
  float g = p.w[0] * bf16_at(p.g[0], i);
  for (int r = 1; r < n; ++r) g = g + p.w[r] * bf16_at(p.g[r], i);
  return ACC ? p.gacc[i] + g : g;
}

template <int N, bool ACC, int BS>
__global__ __launch_bounds__(BS) void reduce_momentum_vec_kernel(ReduceMomentumParams p) {
  constexpr int NMAX = N > 0 ? N : ZERO_MAX_RANKS;
  const int n = N > 0 ? N : p.n_ranks;
  const int64_t nvec = p.n >> 2;
  f32x4* __restrict__ M = reinterpret_cast<f32x4*>(p.m);
  u32x2* __restrict__ U = reinterpret_cast<u32x2*>(p.u);
  const f32x4* __restrict__ GA = reinterpret_cast<const f32x4*>(p.gacc);
  const int64_t step = static_cast<int64_t>(gridDim.x) * BS;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * BS; tile < nvec; tile += step) {
    const int64_t i = tile + threadIdx.x;
    if (i < nvec) {
      const int64_t len = tile_len(nvec - tile, BS);
      const TileOut<f32x4, true> oM(M + tile, len);
      const TileOut<u32x2, true> oU(U + tile, len);
      u32x2 x[NMAX];
#pragma unroll
      for (int r = 0; r < NMAX; ++r)
        if (r < n) x[r] = ld_nt_any(reinterpret_cast<const u32x2_any*>(p.g[r]) + i);
      f32x4 m = ld_nt(M + i);
      f32x4 acc;
      if (ACC) acc = ld_nt(GA + i);
      f32x4 g = reduce4<NMAX>(x, n, p.w);
      if (ACC) g = acc + g;
      const u32x2 u = momentum4(m, g, p.s);
      oM.store(m, threadIdx.x);
      oU.store(u, threadIdx.x);
    }
  }
  const int64_t tail = p.n - (nvec << 2);
  if (blockIdx.x == 0 && threadIdx.x < tail) {
    const int64_t i = (nvec << 2) + threadIdx.x;
    float m = p.m[i];
    const float u = momentum_elem(m, reduce1<N, ACC>(p, n, i), p.s);
    p.m[i] = m;
    p.u[i] = to_bf16(u);
  }
}

template <bool ACC>
__global__ __launch_bounds__(kBlock) void reduce_momentum_scalar_kernel(ReduceMomentumParams p) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < p.n;
       i += static_cast<int64_t>(gridDim.x) * kBlock) {
    float m = p.m[i];
    const float u = momentum_elem(m, reduce1<0, ACC>(p, p.n_ranks, i), p.s);
    p.m[i] = m;
    p.u[i] = to_bf16(u);
  }
}

// -------------------------------------------------------------- owner update
// p' = p - lr*(o + wd*p), and the BF16 working weight: 12 bytes per element.
// The decay term is left out when wd is 0, as in the Adam update.
template <bool WD>
__device__ __forceinline__ float update_elem(float p, float o, float lr, float wd) {
  const float u = WD ? o + wd * p : o;
  return p - lr * u;
}

template <bool WD, int BS>
__global__ __launch_bounds__(BS) void muon_update_vec_kernel(MuonUpdateParams a) {
  const int64_t nvec = a.n >> 2;
  f32x4* __restrict__ P = reinterpret_cast<f32x4*>(a.p);
  u32x2* __restrict__ B = reinterpret_cast<u32x2*>(a.b);
  const u32x2_any* __restrict__ O = reinterpret_cast<const u32x2_any*>(a.o);
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * BS;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * BS; tile < nvec; tile += step) {
    const int64_t i = tile + threadIdx.x;
    if (i < nvec) {
      const int64_t len = tile_len(nvec - tile, BS);
      const TileOut<f32x4, true> oP(P + tile, len);
      const TileOut<u32x2, true> oB(B + tile, len);
      const u32x2 o = ld_nt_any(O + i);
      f32x4 p = ld_nt(P + i);
      p.x = update_elem<WD>(p.x, bf16_lo(o.x), lr, a.wd);
      p.y = update_elem<WD>(p.y, bf16_hi(o.x), lr, a.wd);
      p.z = update_elem<WD>(p.z, bf16_lo(o.y), lr, a.wd);
      p.w = update_elem<WD>(p.w, bf16_hi(o.y), lr, a.wd);
      oP.store(p, threadIdx.x);
      oB.store(u32x2{to_bf16x2(p.x, p.y), to_bf16x2(p.z, p.w)}, threadIdx.x);
    }
  }
  const int64_t tail = a.n - (nvec << 2);
  if (blockIdx.x == 0 && threadIdx.x < tail) {
    const int64_t i = (nvec << 2) + threadIdx.x;
    const float p = update_elem<WD>(a.p[i], bf16_at(a.o, i), lr, a.wd);
    a.p[i] = p;
    a.b[i] = to_bf16(p);
  }
}

template <bool WD>
__global__ __launch_bounds__(kBlock) void muon_update_scalar_kernel(MuonUpdateParams a) {
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < a.n;
       i += static_cast<int64_t>(gridDim.x) * kBlock) {
    const float p = update_elem<WD>(a.p[i], bf16_at(a.o, i), lr, a.wd);
    a.p[i] = p;
    a.b[i] = to_bf16(p);
  }
}

// -------------------------------------------------------------- launch shape
// 64 lanes of 4 elements: one wave, the fewest requests that leave together.
// Measured on shards of 54.5M elements (momentum, update) and 4 owners' 50.6M of
// 4 ranks (fused): workgroups of 64, 128, 256 take 116, 117, 122 us; 98.6, 99.3,
// 101.5 us; 563, 567, 567 us.
constexpr int kMomentumBlock = 64;
constexpr int kReduceMomentumBlock = 64;
constexpr int kMuonUpdateBlock = 64;

// Residency caps, as for the Adam update: the launches reserve this many bytes of
// LDS so that 160 KiB / bytes workgroups are resident per CU.  With 40 to 60 KB of
// loads on their way per CU the HBM keeps more row hits.  Measured without and with
// the cap: momentum 115.8 and 113.2 us (6.59, 6.74 TB/s), update 98.5 and 97.6 us
// (6.64, 6.70 TB/s; at 10 per CU 133 us); fused, TB/s with 1, 2, 4 and 8 ranks 6.62,
// 6.54, 6.48, 6.32 without and 6.68, 6.67, 6.68, 6.64 with (accumulating 6.63, 6.58,
// 6.41, 6.23 and 6.70, 6.74, 6.63, 6.63).  Other rank counts lose with any (without: 3
// ranks 6.65, 5 to 7 6.42 to 6.34, 9 to 16 6.22 to 6.05).
constexpr unsigned kMomentumResidencyLds = 8 * 1024;     // 20 workgroups
constexpr unsigned kMuonUpdateResidencyLds = 8 * 1024;
constexpr unsigned reduce_momentum_residency_lds(int n_ranks) {
  return n_ranks == 0 ? 0 : n_ranks == 1 ? 6 * 1024 : n_ranks == 2 ? 8 * 1024 : n_ranks == 4 ? 10 * 1024 : 16 * 1024;
}

template <bool SC>
hipError_t momentum_launch(const MomentumParams& a, bool vec, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((momentum_vec_kernel<SC, kMomentumBlock>), dim3(grid_x(a.n >> 2, 1, kMomentumBlock)),
                       dim3(kMomentumBlock), kMomentumResidencyLds, s, a);
  else
    hipLaunchKernelGGL((momentum_scalar_kernel<SC>), dim3(grid_x(a.n, 1)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int N, bool ACC>
hipError_t reduce_momentum_vec_launch(const ReduceMomentumParams& p, hipStream_t s) {
  hipLaunchKernelGGL((reduce_momentum_vec_kernel<N, ACC, kReduceMomentumBlock>),
                     dim3(grid_x(p.n >> 2, 1, kReduceMomentumBlock)), dim3(kReduceMomentumBlock),
                     reduce_momentum_residency_lds(N), s, p);
  return hipGetLastError();
}

template <bool ACC>
hipError_t reduce_momentum_dispatch(const ReduceMomentumParams& p, bool vec, hipStream_t s) {
  if (!vec) {
    hipLaunchKernelGGL((reduce_momentum_scalar_kernel<ACC>), dim3(grid_x(p.n, 1)), dim3(kBlock), 0, s, p);
    return hipGetLastError();
  }
  switch (p.n_ranks) {
    case 1: return reduce_momentum_vec_launch<1, ACC>(p, s);
    case 2: return reduce_momentum_vec_launch<2, ACC>(p, s);
    case 4: return reduce_momentum_vec_launch<4, ACC>(p, s);
    case 8: return reduce_momentum_vec_launch<8, ACC>(p, s);
    default: return reduce_momentum_vec_launch<0, ACC>(p, s);
  }
}

template <bool WD>
hipError_t muon_update_launch(const MuonUpdateParams& a, bool vec, hipStream_t s) {
  if (vec)
    hipLaunchKernelGGL((muon_update_vec_kernel<WD, kMuonUpdateBlock>), dim3(grid_x(a.n >> 2, 1, kMuonUpdateBlock)),
                       dim3(kMuonUpdateBlock), kMuonUpdateResidencyLds, s, a);
  else
    hipLaunchKernelGGL((muon_update_scalar_kernel<WD>), dim3(grid_x(a.n, 1)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_momentum(const MomentumParams& a, bool vec, hipStream_t s) {
  return a.gscale ? momentum_launch<true>(a, vec, s) : momentum_launch<false>(a, vec, s);
}

hipError_t launch_reduce_momentum(const ReduceMomentumParams& p, bool vec, hipStream_t s) {
  return p.gacc ? reduce_momentum_dispatch<true>(p, vec, s) : reduce_momentum_dispatch<false>(p, vec, s);
}

hipError_t launch_muon_update(const MuonUpdateParams& a, bool vec, hipStream_t s) {
  return a.wd != 0.0f ? muon_update_launch<true>(a, vec, s) : muon_update_launch<false>(a, vec, s);
}

}  // namespace zero
