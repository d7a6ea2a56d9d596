// split_plan.hpp -- the work split of output tiles over persistent workgroups: host code that
// plans it and the functions by which kernels read the plan (plain C++, so that a host without
// a GPU can check them against each other).
//
// Work split.  T output tiles, I steps each along the sum, W persistent workgroups
// (a multiple of the 8 XCDs; workgroup g runs on XCD g % 8):
// * data-parallel rounds: the first floor(T / W) * W tiles are computed whole, W at a
//   time; in each round the workgroups of an XCD take consecutive tiles of the tile
//   order, so they share rows and columns in the XCD's L2;
// * the leftover tiles are dealt to the XCDs in contiguous ranges, and an XCD's
//   (tile, step) iterations are split evenly over nsk of its workgroups, which compute
//   them first and store fp32 partial tiles.  A workgroup's range is no longer than
//   one tile, so it touches at most two tiles (slots 2 g and 2 g + 1);
// * where splitting the leftover tiles would save fewer steps than joining them costs, nothing
//   is split: they are a last round that not every workgroup has a tile in, and no second
//   kernel runs.
#pragma once

#include <stdint.h>

#include "kernels.hpp"

#ifdef __HIPCC__
#define W4A16_HD __host__ __device__
#else
#define W4A16_HD
#endif

namespace w4a16 {

constexpr int kXCD = 8;
constexpr int kGroupM = 4;                  // tile rows per group of the tile order

struct SplitPlan {
  int tiles_m, tiles_n, iters;              // iters: steps per tile
  int wgs, rounds, sk_tiles, nsk;           // nsk: stream-K workgroups per XCD
};

// What splitting costs a kernel: steps per segment, at least; and a join, in the time of steps:
// join_steps for the second kernel, and one more for every parts_per_step partial tiles.
struct SplitCost {
  int min_steps, join_steps, parts_per_step;
};

inline SplitPlan split_plan(int tiles_m, int tiles_n, int iters, const SplitCost& cost, const DeviceInfo& dev) {
  SplitPlan p;
  p.tiles_m = tiles_m;
  p.tiles_n = tiles_n;
  p.iters = iters;
  int per_xcd = dev.num_cu / kXCD;
  if (per_xcd < 1) per_xcd = 1;
  if (per_xcd > 32) per_xcd = 32;           // (32-bit iteration counts, see sk_begin)
  p.wgs = per_xcd * kXCD;
  const long long tiles = (long long)tiles_m * tiles_n;
  p.rounds = (int)(tiles / p.wgs);
  p.sk_tiles = (int)(tiles - (long long)p.rounds * p.wgs);
  // stream-K workgroups per XCD, from the busiest XCD's ceil(R / 8) tiles;
  // at least one per tile, so no range is longer than a tile
  const int cnt_max = (p.sk_tiles + kXCD - 1) / kXCD;
  long long nsk = (long long)cnt_max * iters / cost.min_steps;
  if (nsk < cnt_max) nsk = cnt_max;
  if (nsk > per_xcd) nsk = per_xcd;
  // no empty ranges on an XCD with fewer leftover tiles (a join takes every workgroup between
  // a tile's first and last contributor); for one step per tile a range may then be two tiles
  const long long least = (long long)(p.sk_tiles >= kXCD ? p.sk_tiles / kXCD : 1) * iters;
  if (nsk > least) nsk = least;
  p.nsk = p.sk_tiles ? (int)nsk : 0;
  if (p.sk_tiles == 0) return p;
  const long long saved = iters - ((long long)cnt_max * iters + nsk - 1) / nsk;
  const long long parts = nsk * (p.sk_tiles < kXCD ? p.sk_tiles : kXCD);
  if (saved <= cost.join_steps + parts / cost.parts_per_step) {
    if (tiles < p.wgs) p.wgs = (int)(tiles + kXCD - 1) / kXCD * kXCD;
    p.rounds = (int)((tiles + p.wgs - 1) / p.wgs);
    p.sk_tiles = p.nsk = 0;
  }
  return p;
}

// Places for partial tiles: two for each workgroup that may have split tiles (l < nsk of every XCD).
inline size_t split_slots(const SplitPlan& p) { return 2 * (size_t)p.nsk * kXCD; }

W4A16_HD inline int xcd_begin(int xcd, int count) {
  const int q = count / kXCD, r = count % kXCD;
  return xcd * q + (xcd < r ? xcd : r);
}

// Tile order: groups of kGroupM tile rows; inside a group, column by column.
W4A16_HD inline void tile_coords(int tau, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per_group = kGroupM * tiles_n;
  const int grp = tau / per_group;
  const int first_m = grp * kGroupM;
  const int gsize = tiles_m - first_m < kGroupM ? tiles_m - first_m : kGroupM;
  const int r = tau - grp * per_group;
  tm = first_m + r % gsize;
  tn = r / gsize;
}

// One work item: steps [a, b) of the tile whose first output row and column are r0 and c0.
struct TileItem {
  int a, b, r0, c0;
};

// Iterations [sk_begin(l), sk_begin(l + 1)) of an XCD with `cnt` leftover tiles belong to its
// workgroup l.  32 bits hold the product: at most 32 leftover tiles and 32 workgroups per
// XCD, and fewer than 2^21 steps (a packed weight tensor stays below 2 GiB).
W4A16_HD inline uint32_t sk_begin(const SplitPlan& p, int cnt, int l) {
  return (uint32_t)cnt * (uint32_t)p.iters * (uint32_t)l / (uint32_t)p.nsk;
}

// The items of workgroup `wg`: its stream-K segments (n_seg of them: 0, 1 or 2), then one whole tile per round.
struct WorkRange {
  int wg, xcd, lwg, sk_lo, n_seg, j_first;
  int s, e;
  W4A16_HD inline WorkRange(const SplitPlan& p, int wg_) : wg(wg_) {
    xcd = wg % kXCD;
    lwg = wg / kXCD;
    sk_lo = xcd_begin(xcd, p.sk_tiles);
    const int cnt = xcd_begin(xcd + 1, p.sk_tiles) - sk_lo;
    const bool in = lwg < p.nsk && cnt > 0;
    s = in ? (int)sk_begin(p, cnt, lwg) : 0;
    e = in ? (int)sk_begin(p, cnt, lwg + 1) : 0;
    j_first = s / p.iters;
    n_seg = e > s ? (e > (j_first + 1) * p.iters ? 2 : 1) : 0;
  }
  // items of this workgroup (the last round may be a partial one)
  W4A16_HD inline int count(const SplitPlan& p) const {
    const int last = (p.rounds - 1) * p.wgs + xcd * (p.wgs / kXCD) + lwg;
    return n_seg + p.rounds - (p.rounds > 0 && last >= p.tiles_m * p.tiles_n ? 1 : 0);
  }
  W4A16_HD inline TileItem item(const SplitPlan& p, int i, int tile_rows, int tile_cols) const {
    TileItem it;
    int tau;
    if (i < n_seg) {
      const int lo = (j_first + i) * p.iters;
      it.a = (s > lo ? s : lo) - lo;
      it.b = (e < lo + p.iters ? e : lo + p.iters) - lo;
      tau = p.rounds * p.wgs + sk_lo + j_first + i;
    } else {
      it.a = 0;
      it.b = p.iters;
      tau = (i - n_seg) * p.wgs + xcd * (p.wgs / kXCD) + lwg;
    }
    int tm, tn;
    tile_coords(tau, p.tiles_m, p.tiles_n, tm, tn);
    it.r0 = tm * tile_rows;
    it.c0 = tn * tile_cols;
    return it;
  }
};

// The workgroups [first, last] of an XCD that hold parts of leftover tile `tile` (0 .. sk_tiles - 1), in order.
struct Contributors {
  int xcd, first, last;
  bool first_cut;            // the first one's range began in the tile before
  W4A16_HD inline Contributors(const SplitPlan& p, int tile) {
    const int q = p.sk_tiles / kXCD, r = p.sk_tiles % kXCD;
    xcd = tile < r * (q + 1) ? tile / (q + 1) : r + (tile - r * (q + 1)) / (q > 0 ? q : 1);
    const int sk_lo = xcd_begin(xcd, p.sk_tiles);
    const int cnt = xcd_begin(xcd + 1, p.sk_tiles) - sk_lo;
    const uint32_t total = (uint32_t)cnt * (uint32_t)p.iters, lo = (uint32_t)(tile - sk_lo) * (uint32_t)p.iters;
    // the largest l with floor(total l / nsk) <= i, i.e. l < (i + 1) nsk / total
    first = (int)(((lo + 1) * (uint32_t)p.nsk - 1) / total);
    last = (int)(((lo + (uint32_t)p.iters) * (uint32_t)p.nsk - 1) / total);
    first_cut = sk_begin(p, cnt, first) < lo;
  }
  // partial slot of contributor l: its second segment if its range began in the tile before
  W4A16_HD inline int slot(int l) const { return 2 * (l * kXCD + xcd) + (l == first && first_cut ? 1 : 0); }
};

}  // namespace w4a16
