// The feed-forward calls' launches without a GPU: csrc/ffn.hip's host side with every
// launch written down instead of made.  Reads lines
//   f|b tokens model hidden unaligned saved|dx
// and prints for each the kernels in order, "name[its kind] workgroups", after
// checking that what a launch reads of and writes to the workspace lies inside the bytes that
// the call asks for, and that its workgroups cover its results.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

namespace routes {
template <class Args>
void note(const char* kernel, const char* where, dim3 grid, dim3 block, const Args& a);
}
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, args) routes::note(#kernel, __PRETTY_FUNCTION__, grid, block, args)
#define hipGetLastError() hipSuccess
#undef __global__
#define __global__ static __device__ __attribute__((unused))
#undef __launch_bounds__
#define __launch_bounds__(...)
#include "../../zero_sharded_optimizer_reduce_amd/csrc/ffn.hip"

namespace zero {
hipError_t launch_act8_save(const Act8Params& p, hipStream_t) {
  std::printf(" act8_save %lldx%lld;", (long long)p.rows, (long long)p.cols);
  return hipSuccess;
}
hipError_t launch_act8_load(const Act8Params& p, hipStream_t) {
  std::printf(" act8_load %lldx%lld;", (long long)p.rows, (long long)p.cols);
  return hipSuccess;
}
}  // namespace zero

namespace routes {
using namespace zero;

constexpr uintptr_t kRoom = uintptr_t(1) << 50;   // where the workspace lies
constexpr int64_t kFar = int64_t(1) << 44;        // beyond it other buffers
int64_t need = 0;

void fail(const char* what) {
  std::printf(" FAILED %s\n", what);
  std::exit(1);
}
// rows of `values` elements of `size` bytes, `ld` elements apart
void inside(const char* what, const void* p, int64_t rows, int64_t ld, int64_t values, int64_t size) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if (at < kRoom || at >= kRoom + kFar || rows < 1) return;
  if (static_cast<int64_t>(at - kRoom) + ((rows - 1) * ld + values) * size > need) fail(what);
}
int argument(const std::string& where, const char* name) {
  const size_t at = where.find(std::string(name) + " = ");
  return at == std::string::npos ? -1 : std::atoi(where.c_str() + at + std::strlen(name) + 3);
}
std::string rest(const std::string& where, const char* name) {
  const size_t at = where.find(std::string(name) + " = ");
  if (at == std::string::npos) return "";
  const size_t from = at + std::strlen(name) + 3;
  std::string value = where.substr(from, where.find_first_of(",]", from) - from);
  const size_t colon = value.rfind(':');
  return colon == std::string::npos ? value : value.substr(colon + 1);
}

void look(const std::string& kernel, const std::string& where, dim3 grid, dim3 block, const Products& a) {
  const bool few = kernel.find("few") != std::string::npos;
  const int64_t threads = block.x, side = (a.side + threads - 1) / threads;
  if (few) {
    const Product& g = a.of[0];
    std::printf(" few[%s,%d] %d;", rest(where, "GATED") == "true" ? "gated" : "plain", std::atoi(kernel.c_str() + kernel.find('<') + 1) * 16, a.tiles);
    if (grid.x != a.tiles + side || int64_t(a.tiles) * a.rows < g.np) fail("few: workgroups");
    inside("few: q", g.q, g.nq, g.q_ld, g.kk, 2);
    inside("few: out", g.out, g.nq, g.out_ld, g.np, 2);
    return;
  }
  const int bp = argument(where, "BP"), bq = argument(where, "BQ");
  const std::string epi = rest(where, "EPI");
  const bool pcol = rest(where, "PCOL") == "true", qcol = rest(where, "QCOL") == "true", part = epi == "kPartial";
  std::printf(" %s[%dx%d,%d,%s,%s%s%s] %u;", epi.c_str(), bp, bq, argument(where, "SLOTS"), pcol ? "columns" : "rows", qcol ? "columns" : "rows",
              a.quarters ? ",quarters" : "", a.spread ? ",spread" : "", a.tiles);
  if (grid.x != a.tiles + side || int64_t(grid.x) * threads >= int64_t(1) << 32) fail("tiles: workgroups");
  const int own = epi == "kGated" ? bp / 2 : bp;
  for (int k = 0; k < 3; ++k) {
    const Product& g = a.of[k];
    if (a.first[k] == 0x7FFFFFFF) continue;
    const int64_t across = int64_t(g.tiles_p) * own * (a.quarters ? 2 : 1), down = int64_t(g.tiles_q) * bq * (a.quarters ? 2 : 1);
    if (across < g.out_cols || across < g.np || down < g.nq) fail("tiles: results not covered");
    // operands
    if (pcol) {
      inside("p", g.p, g.p_end, g.p_ld, g.p_cols, 2);
      inside("p2", g.p2, g.p_end, g.p_ld, g.p_cols, 2);
    } else {
      inside("p", g.p, g.np, g.p_ld, g.kk, 2);
      inside("p2", g.p2, g.p2 ? g.np : 0, g.p_ld, g.kk, 2);
    }
    if (qcol) {
      inside("q", g.q, g.q_end, g.q_ld, g.q_cols, 2);
    } else {
      inside("q", g.q, g.nq, g.q_ld, g.kk, 2);
      if (g.kk % 64 || g.q_ld % 8 || reinterpret_cast<uintptr_t>(g.q) % 16) fail("q: whole stages of whole pieces");
    }
    if (!pcol && (g.kk % 64 || g.p_ld % 8 || reinterpret_cast<uintptr_t>(g.p) % 16)) fail("p: whole stages of whole pieces");
    if (pcol && (g.p_ld % 8 || reinterpret_cast<uintptr_t>(g.p) % 16)) fail("p: whole pieces");
    if (part) {
      if (int64_t(a.splits) * a.chunk < g.kk || int64_t(a.splits - 1) * a.chunk >= g.kk || a.chunk % 128) fail("parts do not cover the sum");
      if (int64_t(a.tiles) != int64_t(g.tiles_p) * g.tiles_q * a.splits) fail("parts: workgroups");
      if (a.pitch % 8 || a.pitch < g.np) fail("parts: pitch");
      inside("partial", a.partial, int64_t(a.splits) * g.nq, a.pitch, a.pitch, 4);
    } else {
      inside("out", g.out, g.nq, g.out_ld, g.out_cols, 2);
    }
    if (epi == "kSlopes") {
      inside("du", a.du, g.nq, g.out_ld, g.out_cols, 2);
      inside("h", a.h, g.nq, a.h_ld, g.out_cols, 2);
      inside("x", a.x.values, a.x.rows, a.x.row, a.x.cols, 2);
    }
  }
  if (a.begin == 0 && !a.quarters && !part) {
    int64_t all = 0;
    for (int k = 0; k < 3; ++k)
      if (a.first[k] != 0x7FFFFFFF) all += int64_t(a.of[k].tiles_p) * a.of[k].tiles_q;
    if (a.tiles > all) fail("more workgroups than tiles");
  }
  if (qcol && a.side) {
    std::printf(" join beside %d;", a.join.splits);
    if (side * threads < a.join.nq * (a.join.pitch / 8)) fail("join beside: workgroups");
    inside("join", a.join.partial, int64_t(a.join.splits) * a.join.nq, a.join.pitch, a.join.pitch, 4);
  }
}
void look(const std::string&, const std::string&, dim3 grid, dim3 block, const PackArgs& a) {
  std::printf(" pack %u;", grid.y);
  for (unsigned k = 0; k < grid.y; ++k) inside("packed", a.of[k].to, a.of[k].rows, a.of[k].pitch, a.of[k].pitch, 2);
}
void look(const std::string&, const std::string&, dim3 grid, dim3 block, const JoinArgs& a) {
  std::printf(" join %d;", a.splits);
  if (int64_t(grid.x) * block.x < a.nq * (a.pitch / 8)) fail("join: workgroups");
  inside("join", a.partial, int64_t(a.splits) * a.nq, a.pitch, a.pitch, 4);
}
template <class Args>
void note(const char* kernel, const char* where, dim3 grid, dim3 block, const Args& a) {
  look(kernel, where, grid, block, a);
}

template <class T>
T* other(int k) {   // a buffer outside the workspace
  return reinterpret_cast<T*>(kRoom + kFar * (k + 2));
}
}  // namespace routes

int main() {
  using namespace routes;
  char pass;
  long long tokens, model, hidden;
  int unaligned, extra;
  while (std::scanf(" %c %lld %lld %lld %d %d", &pass, &tokens, &model, &hidden, &unaligned, &extra) == 6) {
    FfnParams p;
    std::memset(&p, 0, sizeof p);
    p.x = other<uint16_t>(0);
    p.y = pass == 'f' || extra ? other<uint16_t>(1) : nullptr;
    p.x_row = p.y_row = model;
    p.tokens = tokens;
    p.model = model;
    p.hidden = hidden;
    p.w_gate = other<uint16_t>(2) + (unaligned ? 1 : 0);
    p.w_up = other<uint16_t>(3);
    p.w_down = other<uint16_t>(4);
    p.d_gate = other<uint16_t>(5);
    p.d_up = other<uint16_t>(6);
    p.d_down = other<uint16_t>(7);
    p.save = pass == 'f' && extra;
    p.workspace = reinterpret_cast<void*>(kRoom);
    need = ffn_workspace_bytes(tokens, model, hidden, pass == 'b', !ffn_weights_aligned(p));
    std::printf("%c %lld %lld %lld %d %d:", pass, tokens, model, hidden, unaligned, extra);
    if (pass == 'f' && tokens > 0 && launch_ffn_forward(p, nullptr) != hipSuccess) fail("forward");
    if (pass == 'b' && launch_ffn_backward(p, nullptr) != hipSuccess) fail("backward");
    std::printf("\n");
  }
  return 0;
}
