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

// Rows (ranges x rows of d, 1 KB each) that a strip's last workgroup adds at most.  Measured,
// last workgroup against second kernel, device time: 1 row 1024 -> 1024 (4 rows) 6.8 / 7.4 us,
// 1 row through a 1024 x 2048 pair (4) 9.1 / 9.6, 1 row 17408 -> 5120 (25) 19.0 / 18.3, 19 rows
// through the pair (76) 14.3 / 12.3, 16 rows 17408 -> 5120 (400) 27.3 / 21.3; the second launch
// also takes 2.3 us of the host's time per call, which is what bounds the small ones.
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
