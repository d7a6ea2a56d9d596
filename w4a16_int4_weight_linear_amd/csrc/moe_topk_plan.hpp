// moe_topk_plan.hpp -- how the router's kernels lay tokens over lanes and workgroups (plain C++, swept on the host).
#pragma once

#include <stdint.h>

namespace w4a16 {
namespace topk_plan {

constexpr int kThreads = 256;
constexpr int kExperts = 1024, kSlots = 64;        // most experts, most slots
constexpr int kTokens = (1 << 26) - 1;             // most tokens

// Lanes of a token: a DPP row for up to 256 experts and 16 slots, else a wave; and a wave per token
// where there are few tokens (a round's chain of instructions is shorter).  A wave against a row, 256 experts, 8
// slots, fp32: 64 tokens 4.9 / 5.2 us, 1024 tokens 4.9 / 5.3, 2048 tokens 5.0 / 5.4, 4096 tokens 6.1 / 5.6, 16384 tokens
// 14.5 / 9.7.
constexpr int kWaveTokens = 2048;
inline int lanes_of(int tokens, int experts, int topk) {
  return topk <= 16 && experts <= 256 && tokens > kWaveTokens ? 16 : 64;
}

// The grid: a launch has fewer than 2^32 threads along an axis, counted in whole workgroups, so past kGridRow
// workgroups there are several rows of them (a wave per token reaches 2^24 workgroups of 256 threads).  Workgroup
// y * gridDim.x + x; those past the last token have nothing to do.
constexpr int64_t kGridRow = ((int64_t)1 << 32) / kThreads - 1;
struct Grid {
  unsigned x, y;
};
inline Grid grid_of(int tokens, int lanes) {
  const int64_t per = kThreads / lanes, blocks = (tokens + per - 1) / per, rows = (blocks + kGridRow - 1) / kGridRow;
  return {(unsigned)((blocks + rows - 1) / rows), (unsigned)rows};
}

}  // namespace topk_plan
}  // namespace w4a16
