// Host-only driver for the overlap check of the feed-forward calls' matrices, built with g++
// and the address/undefined-behaviour sanitizers (no HIP, no device): matrices with one row stride
// against a walk over all their elements.  Prints "ok".
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../../zero_sharded_optimizer_reduce_amd/csrc/validate.h"

using namespace zero;

template <class T>
static T* P(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}

static int call(bool backward, uintptr_t in, int64_t in_row, uintptr_t out, int64_t out_row, int64_t tokens, int64_t model, Err& e) {
  const uintptr_t far = uintptr_t(1) << 50;
  zero_ffn_checkpoint c;
  uint8_t** parts[6] = {&c.x_codes, &c.x_scales, &c.gate_codes, &c.gate_scales, &c.up_codes, &c.up_scales};
  for (int k = 0; k < 6; ++k) *parts[k] = P<uint8_t>(far + (uintptr_t(k) << 40));
  c.format = ZERO_ACT8_INT8;
  uint16_t* w[7];
  for (int k = 0; k < 7; ++k) w[k] = P<uint16_t>(far + (uintptr_t(k + 8) << 40));
  return check_ffn(backward, P<uint16_t>(in), in_row, tokens, model, 8, w[0], w[1], w[2], ZERO_FFN_RELU, P<uint16_t>(out), out_row, &c,
                   w[3], w[4], w[5], w[6], 256, 256, e);
}

int main() {
  Err e;
  int fails = 0;
  const uintptr_t base = 0x10000000;
  for (int64_t tokens = 1; tokens <= 3; ++tokens)
    for (int64_t model = 1; model <= 4; ++model)
      for (int64_t row = model; row <= 11; ++row)
        for (int64_t off = -3 * row - 5; off <= 3 * row + 5; ++off) {
          std::vector<char> used(200, 0);   // elements of the first, from 100 on
          bool shared = false;
          for (int64_t t = 0; t < tokens; ++t)
            for (int64_t j = 0; j < model; ++j) used[100 + t * row + j] = 1;
          for (int64_t t = 0; t < tokens; ++t)
            for (int64_t j = 0; j < model; ++j) {
              const int64_t at = 100 + off + t * row + j;
              shared = shared || (at >= 0 && at < 200 && used[at]);
            }
          for (bool backward : {false, true}) {
            const int st = call(backward, base, row, base + 2 * off, row, tokens, model, e);
            // never taken where an element is shared; refused without need only where a row of one runs into
            // the other's columns further on
            const int64_t column = (off % row + row) % row;
            const bool beside = column >= model && column + model <= row;
            if ((shared && st != ZERO_ERR_ARG) || (!shared && beside && st != ZERO_OK)) {
              std::printf("FAILED %d x %d row %d off %d: %d\n", (int)tokens, (int)model, (int)row, (int)off, st);
              ++fails;
            }
          }
        }
  // of different row strides: as ranges; far apart and at both ends of the strides
  if (call(false, base, 16, base + 16, 32, 5, 4, e) != ZERO_ERR_ARG) std::printf("FAILED strides\n"), ++fails;
  const int64_t most = ZERO_FFN_MAX_STRIDE, tokens = ZERO_FFN_MAX_TOKENS;
  if (call(true, base, most, base + 2 * (most - 64), most, tokens, 64, e) != ZERO_OK) std::printf("FAILED the longest\n"), ++fails;
  if (call(true, base, most, base + 2 * (most - 63), most, tokens, 64, e) != ZERO_ERR_ARG) std::printf("FAILED round the end\n"), ++fails;
  if (call(true, base + 2 * (most - 64), most, base, most, tokens, 64, e) != ZERO_OK) std::printf("FAILED the other way\n"), ++fails;
  if (fails == 0) std::printf("ok\n");
  return fails != 0;
}
