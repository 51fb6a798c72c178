// Host-only driver for the Muon step's argument checks, built with g++ and the
// address/undefined-behaviour sanitizers (no HIP, no device): valid, boundary and
// extreme arguments, so that an overflow in a check itself is found.  Prints "ok".
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "../../zero_sharded_optimizer_reduce_amd/csrc/validate.h"

using namespace zero;

static int fails = 0;
#define EXPECT(cond)                                        \
  do {                                                      \
    if (!(cond)) {                                          \
      std::printf("FAILED line %d: %s\n", __LINE__, #cond); \
      ++fails;                                              \
    }                                                       \
  } while (0)

template <class T>
static T* P(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}

int main() {
  Err e;
  const float nan = std::numeric_limits<float>::quiet_NaN(), inf = std::numeric_limits<float>::infinity();
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 2, 3, 63, 4096, 262144, 262145, int64_t(1) << 31, int64_t(1) << 40,
                           int64_t(1) << 61, int64_t(1) << 62, INT64_MAX - 1, INT64_MAX};
  const zero_muon_hparams hp = {1e-3f, 0.95f, 0.1f, 1};
  for (float v : {nan, inf, -inf, -1.0f, 2.0f}) {
    zero_muon_hparams bad = hp;
    bad.momentum = v;
    EXPECT(check_muon_hparams(&bad, e) != ZERO_OK);
  }
  EXPECT(check_muon_hparams(&hp, e) == ZERO_OK && check_muon_hparams(nullptr, e) == ZERO_ERR_ARG);

  float *m = P<float>(0x100000), *g = P<float>(0x200000), *p = P<float>(0x300000);
  uint16_t *u = P<uint16_t>(0x400000), *b = P<uint16_t>(0x500000);
  EXPECT(check_muon_momentum(m, u, g, nullptr, 1000, &hp, e) == ZERO_OK);
  EXPECT(check_muon_shard(p, b, u, nullptr, 1000, &hp, e) == ZERO_OK);
  for (int64_t n : sizes) {
    const int a = check_muon_momentum(m, u, g, P<float>(0x600000), n, &hp, e);
    const int c = check_muon_shard(p, b, u, P<float>(0x600000), n, &hp, e);
    EXPECT((n >= 0 && n <= 262144) == (a == ZERO_OK));   // the buffers are 1 MiB apart: larger ones overlap or overflow
    EXPECT((n >= 0 && n <= 262144) == (c == ZERO_OK));
  }
  EXPECT(check_muon_momentum(m, u, g, m + 3, 1000, &hp, e) == ZERO_ERR_ARG);

  const uint16_t* x[ZERO_MAX_RANKS];
  float* ms[ZERO_MAX_RANKS];
  uint16_t* us[ZERO_MAX_RANKS];
  const float* acc[ZERO_MAX_RANKS];
  float w[ZERO_MAX_RANKS];
  for (int i = 0; i < ZERO_MAX_RANKS; ++i) {
    x[i] = P<uint16_t>(0x1000000 + 0x100000 * i);
    ms[i] = P<float>(0x3000000 + 0x100000 * i);
    us[i] = P<uint16_t>(0x5000000 + 0x100000 * i);
    acc[i] = P<float>(0x7000000 + 0x100000 * i);
    w[i] = 1.0f;
  }
  for (int n_ranks : {INT32_MIN, -1, 0, 1, ZERO_MAX_RANKS, ZERO_MAX_RANKS + 1, INT32_MAX})
    for (int n_shards : {INT32_MIN, 0, 1, 3, ZERO_MAX_RANKS, INT32_MAX})
      for (int64_t n : sizes) {
        const bool ok = n_ranks >= 1 && n_ranks <= ZERO_MAX_RANKS && n_shards >= 1 && n_shards <= ZERO_MAX_RANKS && n >= 0 &&
                        n % n_shards == 0 && n <= 262145;   // of 1 owner 4 bytes past 1 MiB, where nothing lies
        EXPECT(ok == (check_reduce_scatter_muon(x, w, n_ranks, n, n_shards, ms, us, acc, &hp, e) == ZERO_OK));
      }

  const float coefs[15] = {3.4445f, -4.7750f, 2.0315f, 3.4445f, -4.7750f, 2.0315f, 3.4445f, -4.7750f,
                           2.0315f, 3.4445f,  -4.7750f, 2.0315f, 3.4445f,  -4.7750f, 2.0315f};
  EXPECT(check_ns_coefs(coefs, 5, e) == ZERO_OK);
  for (int steps : {INT32_MIN, -1, 0, ZERO_NS_MAX_STEPS + 1, INT32_MAX}) EXPECT(check_ns_coefs(coefs, steps, e) != ZERO_OK);
  const float values[] = {nan, inf, -inf, 3.4e38f, -3.4e38f, 1e-45f, 0.0f, 1.0f, 17.0f};
  for (float a : values)
    for (float bb : values)
      for (float c : values) {
        const float one[3] = {a, bb, c};
        const int st = check_ns_coefs(one, 1, e);
        if (!std::isfinite(a) || !std::isfinite(bb) || !std::isfinite(c) || a > 16.0f) EXPECT(st != ZERO_OK);
      }

  for (int64_t mats : sizes)
    for (int64_t rows : sizes)
      for (int64_t cols : sizes) {
        const int st = check_ns_shape(mats, rows, cols, e);
        EXPECT((mats >= 0 && mats <= ZERO_NS_MAX_MATS && rows >= 0 && rows <= ZERO_NS_MAX_SIDE && cols >= 0 &&
                cols <= ZERO_NS_MAX_SIDE) == (st == ZERO_OK));
        for (int64_t row : sizes)
          for (int64_t mat : {INT64_MIN, int64_t(0), rows, int64_t(1) << 40, INT64_MAX}) {
            check_newton_schulz(P<void>(0x100000), ZERO_FP32, row, mat, u, cols, 0, mats, rows, cols, coefs, 5, 1.0f,
                                P<void>(0x800000), INT64_MAX, 256, e);
            check_newton_schulz(P<void>(0x100000), ZERO_BF16, cols, 0, u, row, mat, mats, rows, cols, coefs, 5, 1.0f,
                                P<void>(0x800000), INT64_MAX, 256, e);
          }
      }
  EXPECT(check_newton_schulz(P<void>(0x100000), ZERO_BF16, 64, 0, u, 64, 0, 1, 64, 64, coefs, 5, 1.0f, P<void>(0x800000),
                             4096, 4096, e) == ZERO_OK);
  EXPECT(check_newton_schulz(P<void>(0x100000), ZERO_BF16, 64, 0, u, 64, 0, 1, 64, 64, coefs, 5, nan, P<void>(0x800000),
                             4096, 4096, e) == ZERO_ERR_ARG);
  EXPECT(check_newton_schulz(P<void>(0x100000), ZERO_BF16, 64, 0, u, 64, 0, 1, 64, 64, coefs, 5, 1.0f, P<void>(0x800000),
                             4095, 4096, e) == ZERO_ERR_SIZE);
  EXPECT(check_newton_schulz(P<void>(0x100000), 7, 64, 0, u, 64, 0, 1, 64, 64, coefs, 5, 1.0f, P<void>(0x800000), 4096,
                             4096, e) == ZERO_ERR_ARG);
  if (fails) return 1;
  std::puts("ok");
  return 0;
}
