// gemm_t_skinny_plan.hpp -- the work split of the weight-streaming product with the weights' other
// side (gemm_t_skinny.hip): plain C++, so that a host without a GPU can check it.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kernels.hpp"

#ifdef __HIPCC__
#define W4A16_HD __host__ __device__
#else
#define W4A16_HD
#endif

namespace w4a16 {
namespace skinny_t {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 32;                       // n per unit
constexpr int CW = 256;                         // columns per strip

struct SkinnyPlan {
  int strips, splits, units, range;             // strips of CW columns, ranges of n, units of 32 n, n per range
  uint32_t lds;
  bool fused;                                   // the strips' last workgroups add the ranges' sums
};

// Rows (ranges x rows of d, 1 KB each) that a strip's last workgroup adds at most.  Measured, last
// workgroup against second kernel, device time in us (graph replays over 1 GB of weights in turn):
// 1 row 5120 -> 17408 (3 rows) 16.7 / 17.5, 1 row 1024 -> 1024 (4) 5.4 / 6.0, 1 row through a 1024 x
// 2048 pair (4) 6.8 / 7.6, 1 row 2048 -> 2048 (8) 6.3 / 6.7, 4 rows 5120 -> 17408 (12) 17.5 / 17.9, 1 row
// 17408 -> 5120 (12) 15.7 / 15.6, 4 rows 1024 -> 1024 (16) 6.0 / 6.4, 1 row 4096 -> 4096 (16) 9.4 / 7.2,
// 1 row 16384 -> 4096 (16) 13.9 / 12.8, 8 rows 1024 -> 1024 (32) 7.2 / 6.9, 4 rows 17408 -> 5120 (48)
// 17.0 / 16.9, 19 rows through the pair (76) 12.1 / 10.5, 16 rows 17408 -> 5120 (192) 21.5 / 18.7.  The
// second launch also takes 2.3 us of the host's time per call, which bounds small calls made one after
// another (through the binding 7.8 us with one launch, 10.1 with two); in a graph twelve and more
// ranges of one row lose up to 2 us by the rule.
constexpr int kJoinRows = 16;

// Floats of one wave's sums (whole quads of rows of d, a block of 16 rows at a time: 128 KB of LDS).
W4A16_HD constexpr int red_stride(int m) { return (m < 16 ? (m + 3) / 4 * 4 : 16) * CW; }

constexpr size_t kMaxSums = (size_t)256 << 20;   // bytes of the ranges' sums, at most

inline int blocks_of(int m) { return m <= 16 ? 1 : 2; }

inline SkinnyPlan skinny_plan(int m, int n, int k, const DeviceInfo& dev) {
  SkinnyPlan p;
  p.strips = (k + CW - 1) / CW;
  p.units = (n + kUnit - 1) / kUnit;
  const int slots = dev.num_cu;
  int splits = slots / p.strips;
  if (splits > (p.units + kWaves - 1) / kWaves) splits = (p.units + kWaves - 1) / kWaves;
  if (splits < 1) splits = 1;
  p.range = ((p.units + splits - 1) / splits) * kUnit;
  p.splits = (n + p.range - 1) / p.range;
  p.fused = p.splits > 1 && p.splits * m <= kJoinRows && p.strips <= kCounters;
  p.lds = (uint32_t)(kWaves * red_stride(m) * 4);
  return p;
}

inline size_t sums_bytes(const SkinnyPlan& p, int m, int k) {
  return p.splits > 1 ? (size_t)p.splits * m * k * 4 : 0;
}

// Whether the kernel takes the plan: its LDS, and the ranges' sums within 32-bit offsets.
inline bool plan_fits(const SkinnyPlan& p, int m, int k, const DeviceInfo& dev) {
  return p.lds + 8192 <= dev.max_lds && sums_bytes(p, m, k) <= kMaxSums;
}

}  // namespace skinny_t
}  // namespace w4a16
