// block_edges_driver.cpp -- the edges of the router's and the few-token experts' sizes: the grids of the most tokens
// against what a launch can have (no GPU).
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "../../w4a16_int4_weight_linear_amd/csrc/moe_topk_plan.hpp"

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

int main() {
  topk_grids();
  if (g_fail) {
    std::fprintf(stderr, "block edges driver: %d of %d checks failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("block edges driver: ok (%d checks)\n", g_checks);
  return 0;
}
