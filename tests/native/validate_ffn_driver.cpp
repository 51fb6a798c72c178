// Host-only driver for the checks of the 8-bit activations and the feed-forward block,
// built with g++ and the address/undefined-behaviour sanitizers (no HIP, no device): valid,
// boundary and extreme arguments, so that an overflow in a check itself is found.
// Prints "ok".
#include <cstdint>
#include <cstdio>
#include <initializer_list>

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
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 2, 31, 32, 33, 4096, 262144, 262145, int64_t(1) << 24, (int64_t(1) << 24) + 1,
                           int64_t(1) << 31, (int64_t(1) << 31) + 1, int64_t(1) << 35, int64_t(1) << 40, int64_t(1) << 61,
                           int64_t(1) << 62, INT64_MAX - 1, INT64_MAX};
  uint8_t *c = P<uint8_t>(uintptr_t(1) << 50), *k = P<uint8_t>(uintptr_t(1) << 54);
  void* v = P<void>(uintptr_t(1) << 44);
  for (int64_t rows : sizes)
    for (int64_t cols : sizes)
      for (int64_t row : sizes)
        for (int dtype : {ZERO_BF16, ZERO_FP32}) {
          const int st = check_act8("act8", v, dtype, row, rows, cols, ZERO_ACT8_E4M3, c, k, e);
          if (rows < 0 || cols < 0) {
            EXPECT(st == ZERO_ERR_ARG);
          } else if (rows == 0 || cols == 0) {
            EXPECT(st == ZERO_OK);
          } else {
            const bool few = cols <= ZERO_ACT8_MAX_COLS && rows <= ZERO_ACT8_MAX_VALUES / ((cols + 31) / 32 * 32);
            const bool stride = rows == 1 || (row >= cols && row <= ZERO_ACT8_MAX_COLS);
            EXPECT((few && stride) == (st == ZERO_OK) || st == ZERO_ERR_ARG);   // ARG: so far apart that they meet the codes
          }
        }
  EXPECT(check_act8("act8", v, 2, 32, 2, 32, 0, c, k, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", v, 0, 32, 2, 32, 2, c, k, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", nullptr, 0, 32, 2, 32, 0, c, k, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", v, 0, 32, 2, 32, 0, nullptr, k, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", v, 0, 32, 2, 32, 0, c, nullptr, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", nullptr, 0, 0, 0, 32, 0, nullptr, nullptr, e) == ZERO_OK);
  EXPECT(check_act8("act8", static_cast<char*>(v) + 1, 0, 32, 2, 32, 0, c, k, e) == ZERO_ERR_ALIGN);
  EXPECT(check_act8("act8", static_cast<char*>(v) + 2, 1, 32, 2, 32, 0, c, k, e) == ZERO_ERR_ALIGN);
  EXPECT(check_act8("act8", c - 8, 0, 32, 2, 32, 0, c, k, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", v, 0, 32, 2, 32, 0, c, c + 63, e) == ZERO_ERR_ARG);
  EXPECT(check_act8("act8", v, 0, 32, 2, 32, 0, c, c + 64, e) == ZERO_OK);

  for (int64_t t : sizes)
    for (int64_t d : sizes)
      for (int64_t h : sizes) {
        const int st = check_ffn_shape(t, d, h, e);
        const int64_t most = d > h ? d : h;
        const bool in = t >= 0 && d >= 1 && h >= 1 && t <= ZERO_FFN_MAX_TOKENS && most <= ZERO_FFN_MAX_SIDE &&
                        t <= ZERO_ACT8_MAX_VALUES / ((most + 31) / 32 * 32);
        EXPECT(in == (st == ZERO_OK));
      }

  struct Call {
    bool backward = false;
    uintptr_t in = 0x10000000, out = 0x20000000, wg = 0x30000000, wu = 0x31000000, wd = 0x32000000, dg = 0x40000000,
              du = 0x41000000, dd = 0x42000000, ws = 0x50000000, ck[6] = {0x60000000, 0x61000000, 0x62000000, 0x63000000, 0x64000000, 0x65000000};
    int64_t in_row = 64, out_row = 64, t = 10, d = 64, h = 96, bytes = 1000, need = 1000;
    int act = ZERO_FFN_SILU, format = ZERO_ACT8_INT8;
    bool saved = true;
    int go(Err& e) const {
      zero_ffn_checkpoint c = {P<uint8_t>(ck[0]), P<uint8_t>(ck[1]), P<uint8_t>(ck[2]), P<uint8_t>(ck[3]), P<uint8_t>(ck[4]), P<uint8_t>(ck[5]), format};
      return check_ffn(backward, P<uint16_t>(in), in_row, t, d, h, P<uint16_t>(wg), P<uint16_t>(wu), P<uint16_t>(wd), act,
                       P<uint16_t>(out), out_row, saved ? &c : nullptr, P<uint16_t>(dg), P<uint16_t>(du), P<uint16_t>(dd),
                       P<void>(ws), bytes, need, e);
    }
  };
  for (bool backward : {false, true}) {
    Call ok;
    ok.backward = backward;
    EXPECT(ok.go(e) == ZERO_OK);
    auto with = [&](auto change) {
      Call x = ok;
      change(x);
      return x.go(e);
    };
    EXPECT(with([](Call& x) { x.act = 3; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.format = -1; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.saved = false; }) == (backward ? ZERO_ERR_ARG : ZERO_OK));
    EXPECT(with([](Call& x) { x.in = 0; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.in += 1; }) == ZERO_ERR_ALIGN);
    EXPECT(with([](Call& x) { x.out = 0; }) == (backward ? ZERO_OK : ZERO_ERR_ARG));
    EXPECT(with([](Call& x) { x.out += 1; }) == ZERO_ERR_ALIGN);
    EXPECT(with([](Call& x) { x.wu = 0; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.wd += 1; }) == ZERO_ERR_ALIGN);
    EXPECT(with([](Call& x) { x.wd += 2; }) == ZERO_OK);
    EXPECT(with([](Call& x) { x.in_row = 63; }) == ZERO_ERR_SIZE);
    EXPECT(with([](Call& x) { x.out_row = INT64_MAX; }) == ZERO_ERR_SIZE);
    EXPECT(with([](Call& x) { x.in_row = ZERO_FFN_MAX_STRIDE + 1; }) == ZERO_ERR_SIZE);
    EXPECT(with([](Call& x) { x.in_row = -5, x.t = 1; }) == ZERO_OK);   // one row: no stride
    EXPECT(with([](Call& x) { x.ws = 0; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.ws += 128; }) == ZERO_ERR_ALIGN);
    EXPECT(with([](Call& x) { x.bytes = 999; }) == ZERO_ERR_SIZE);
    EXPECT(with([](Call& x) { x.out = x.in; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.out = x.wg + 64; }) == ZERO_ERR_ARG);
    EXPECT(with([](Call& x) { x.wu = x.wg; }) == ZERO_OK);   // both only read
    for (int i = 0; i < 6; ++i) {
      EXPECT(with([&](Call& x) { x.ck[i] = 0; }) == ZERO_ERR_ARG);
      EXPECT(with([&](Call& x) { x.ck[i] = x.out; }) == ZERO_ERR_ARG);
      EXPECT(with([&](Call& x) { x.ck[i] = x.in + 1; }) == (backward ? ZERO_OK : ZERO_ERR_ARG));
      EXPECT(with([&](Call& x) { x.ck[i] = x.ws + 5; }) == ZERO_ERR_ARG);
    }
    if (backward) {
      EXPECT(with([](Call& x) { x.dg = 0; }) == ZERO_ERR_ARG);
      EXPECT(with([](Call& x) { x.dd += 1; }) == ZERO_ERR_ALIGN);
      EXPECT(with([](Call& x) { x.du = x.dg + 2; }) == ZERO_ERR_ARG);
      EXPECT(with([](Call& x) { x.dd = x.wd; }) == ZERO_ERR_ARG);
      EXPECT(with([](Call& x) { x.t = 0, x.need = 0, x.in = x.out = x.wg = x.wu = x.wd = x.ws = 0; }) == ZERO_OK);
      EXPECT(with([](Call& x) { x.t = 0, x.need = 0, x.du = 0; }) == ZERO_ERR_ARG);
    } else {
      EXPECT(with([](Call& x) { x.t = 0, x.in = x.out = x.wg = x.ws = 0; }) == ZERO_OK);
    }
  }
  if (fails == 0) std::printf("ok\n");
  return fails != 0;
}
