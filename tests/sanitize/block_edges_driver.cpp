// block_edges_driver.cpp -- the edges of the router's and the few-token experts' sizes: the grids of the most tokens
// against what a launch can have, and the spans of the largest banks (a stand-in device and recording launchers, no GPU).
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "../../include/w4a16.h"
#include "../../w4a16_int4_weight_linear_amd/csrc/moe_topk_plan.hpp"
#include "block_recording_launchers.hpp"

static int g_checks = 0, g_fail = 0;
static void expect(bool ok, const char* what, int line) {
  ++g_checks;
  if (!ok) {
    ++g_fail;
    std::fprintf(stderr, "FAILED line %d: %s\n", line, what);
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)

// Every token has its lanes, a launch's threads along an axis fit 32 bits, and at most a row of grids' rounding is idle.
static void topk_grid(int tokens, int experts, int topk) {
  using namespace w4a16::topk_plan;
  const int lanes = lanes_of(tokens, experts, topk);
  const Grid g = grid_of(tokens, lanes);
  const int64_t per = kThreads / lanes, blocks = (int64_t)g.x * g.y;
  EXPECT((int64_t)g.x * kThreads < (int64_t)1 << 32);
  EXPECT(g.y >= 1 && g.y <= 65535);
  EXPECT(blocks * per >= tokens && (blocks - g.y) * per < tokens);
  EXPECT((g.y == 1) == ((tokens + per - 1) / per <= kGridRow));
}

static void topk_grids() {
  using namespace w4a16::topk_plan;
  for (int experts : {1, 17, 256, 257, 1024})
    for (int topk : {1, 16, 17, 64})
      if (topk <= experts)
        for (int tokens : {1, 3, 4, 5, 2047, 2048, 2049, 1 << 20, (1 << 25) - 1, 1 << 25, (1 << 26) - 5, (1 << 26) - 4, (1 << 26) - 3,
                           (1 << 26) - 2, kTokens})
          topk_grid(tokens, experts, topk);
  EXPECT(grid_of(kTokens, 64).y == 2 && grid_of(kTokens - 3, 64).y == 1 && grid_of(kTokens, 16).y == 1);
}

// Banks of very many experts: scales of 32 x 32 at group 32 are 128 (gate/up) and 64 bytes (down) an expert.  Never dereferenced.
template <typename T> static T* address(int64_t a) { return reinterpret_cast<T*>((uintptr_t)a); }
static w4a16_status ffn(int32_t experts, int64_t out) {
  g_ans.moe = 1 << 20;
  const int64_t t = (int64_t)1 << 40;      // apart from one another
  return w4a16_moe_ffn(address<const uint16_t>(1 << 20), address<const int32_t>(2 << 20), address<const float>(3 << 20),
                       address<const uint32_t>(16 * t), address<const uint16_t>(t), address<const uint32_t>(32 * t),
                       address<const uint16_t>(4 * t), nullptr, address<uint16_t>(out), 2, 2, experts, 32, 32, 32,
                       address<void>(8 << 20), 1 << 20, nullptr);
}
static void large_banks() {
  const int64_t t = (int64_t)1 << 40;
  for (int64_t experts : {(int64_t)1 << 29, ((int64_t)1 << 29) + 7, (int64_t)1 << 30, ((int64_t)1 << 31) - 1}) {
    const int32_t e = (int32_t)experts;
    EXPECT(ffn(e, 64 * t) == W4A16_OK);
    EXPECT(ffn(e, t + 128 * experts - 16) == W4A16_ERR_OVERLAP && ffn(e, t + 128 * experts) == W4A16_OK);
    EXPECT(ffn(e, 4 * t + 64 * experts - 16) == W4A16_ERR_OVERLAP && ffn(e, 4 * t + 64 * experts) == W4A16_OK);
    EXPECT(ffn(e, 16 * t + 1024 * experts - 16) == W4A16_ERR_OVERLAP && ffn(e, 32 * t + 512 * experts - 16) == W4A16_ERR_OVERLAP);
  }
}

int main() {
  topk_grids();
  large_banks();
  if (g_fail) {
    std::fprintf(stderr, "block edges driver: %d of %d checks failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("block edges driver: ok (%d checks)\n", g_checks);
  return 0;
}
