// plan_driver.cpp -- sweeps the work splits of the tiled kernels and of the weight-streaming
// product with the weights' other side on the host: every step of every tile is done once, the
// parts of a split tile lie where the joining kernel looks for them, and 32-bit products hold
// what 64 bits would.  Built under AddressSanitizer and UndefinedBehaviorSanitizer; no GPU.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <random>
#include <vector>

#include "../../w4a16_int4_weight_linear_amd/csrc/gemm_t_skinny_plan.hpp"
#include "../../w4a16_int4_weight_linear_amd/csrc/split_plan.hpp"

using namespace w4a16;

static long g_plans = 0;
static char g_what[200];
#define EXPECT(c)                                                                 \
  do {                                                                            \
    if (!(c)) {                                                                   \
      std::fprintf(stderr, "FAILED line %d: %s (%s)\n", __LINE__, #c, g_what);    \
      std::exit(1);                                                               \
    }                                                                             \
  } while (0)

static DeviceInfo device(int cus) {
  DeviceInfo d;
  d.num_cu = cus;
  d.max_lds = 160 * 1024;
  return d;
}

// every (tile, step) once, by whom, and the parts' places
static void walk(int tiles_m, int tiles_n, int iters, const SplitCost& cost, int cus) {
  std::snprintf(g_what, sizeof g_what, "%d x %d tiles of %d steps, cost %d %d %d, %d CUs", tiles_m, tiles_n, iters,
                cost.min_steps, cost.join_steps, cost.parts_per_step, cus);
  const SplitPlan p = split_plan(tiles_m, tiles_n, iters, cost, device(cus));
  ++g_plans;
  const int tiles = tiles_m * tiles_n;
  EXPECT(p.wgs >= kXCD && p.wgs % kXCD == 0 && p.nsk * kXCD <= p.wgs && (p.nsk > 0) == (p.sk_tiles > 0));
  EXPECT(split_slots(p) == (p.sk_tiles ? (size_t)16 * p.nsk : 0));
  const int rows = 16, cols = 32;
  std::vector<int> next(tiles, 0), owner(tiles, -1);
  struct Part { int tile, a, b, slot; };
  std::vector<Part> parts;
  for (int wg = 0; wg < p.wgs; ++wg) {
    const WorkRange wr(p, wg);
    EXPECT(wr.n_seg >= 0 && wr.n_seg <= 2);
    for (int i = 0; i < wr.count(p); ++i) {
      const TileItem it = wr.item(p, i, rows, cols);
      EXPECT(it.a >= 0 && it.a < it.b && it.b <= iters);
      EXPECT(it.r0 % rows == 0 && it.r0 / rows < tiles_m && it.c0 % cols == 0 && it.c0 / cols < tiles_n);
      const int tile = it.r0 / rows * tiles_n + it.c0 / cols;
      if (i < wr.n_seg) {
        parts.push_back({tile, it.a, it.b, 2 * wg + i});
        EXPECT((size_t)(2 * wg + i) < split_slots(p));
      } else {
        EXPECT(it.a == 0 && it.b == iters && owner[tile] < 0);
        owner[tile] = wg;
        next[tile] = iters;
      }
    }
  }
  // the joining kernel's view of each split tile
  std::vector<char> seen(parts.size(), 0);
  for (int t = 0; t < p.sk_tiles; ++t) {
    int tm, tn;
    tile_coords(p.rounds * p.wgs + t, tiles_m, tiles_n, tm, tn);
    const int tile = tm * tiles_n + tn;
    const Contributors cs(p, t);
    EXPECT(cs.xcd >= 0 && cs.xcd < kXCD && cs.first >= 0 && cs.first <= cs.last && cs.last < p.nsk);
    for (int l = cs.first; l <= cs.last; ++l) {
      bool found = false;
      for (size_t i = 0; i < parts.size(); ++i)
        if (parts[i].slot == cs.slot(l)) {
          EXPECT(!found && !seen[i] && parts[i].tile == tile && parts[i].a == next[tile]);
          found = true;
          seen[i] = 1;
          next[tile] = parts[i].b;
        }
      EXPECT(found);
    }
  }
  for (char s : seen) EXPECT(s);
  for (int t = 0; t < tiles; ++t) EXPECT(next[t] == iters);
}

// the 32-bit positions against 64 bits, for sums too long to walk
static void positions(int tiles, int iters, const SplitCost& cost, int cus) {
  std::snprintf(g_what, sizeof g_what, "%d tiles of %d steps, %d CUs", tiles, iters, cus);
  const SplitPlan p = split_plan(tiles, 1, iters, cost, device(cus));
  ++g_plans;
  for (int t = 0; t < p.sk_tiles; ++t) {
    const Contributors cs(p, t);
    const int lo = xcd_begin(cs.xcd, p.sk_tiles), cnt = xcd_begin(cs.xcd + 1, p.sk_tiles) - lo;
    auto begin = [&](int l) { return (int64_t)cnt * iters * l / p.nsk; };
    for (int l = 0; l <= p.nsk; ++l) EXPECT((int64_t)sk_begin(p, cnt, l) == begin(l));
    const int64_t a = (int64_t)(t - lo) * iters, b = a + iters;
    int first = p.nsk, last = -1;
    for (int l = 0; l < p.nsk; ++l)
      if (begin(l) < b && begin(l + 1) > a) {
        first = l < first ? l : first;
        last = l;
      }
    EXPECT(cs.first == first && cs.last == last && cs.first_cut == (begin(first) < a));
    for (int l = 0; l < p.nsk; ++l) {
      const WorkRange wr(p, l * kXCD + cs.xcd);
      EXPECT(wr.s == begin(l) && wr.e == begin(l + 1) && wr.n_seg >= 1 && wr.n_seg <= 2);
    }
  }
}

static void skinny(int m, int64_t n64, int64_t k64, int cus) {
  using namespace skinny_t;
  const int n = (int)n64, k = (int)k64;
  std::snprintf(g_what, sizeof g_what, "skinny m %d n %d k %d, %d CUs", m, n, k, cus);
  const DeviceInfo dev = device(cus);
  const SkinnyPlan p = skinny_plan(m, n, k, dev);
  ++g_plans;
  EXPECT(p.strips >= 1 && (int64_t)p.strips * CW >= k && (int64_t)(p.strips - 1) * CW < k);
  EXPECT(p.splits >= 1 && p.range % kUnit == 0 && p.range >= kUnit);
  EXPECT((int64_t)p.splits * p.range >= n && (int64_t)(p.splits - 1) * p.range < n);     // no empty range
  EXPECT(p.splits == 1 || (int64_t)p.strips * p.splits <= cus);
  EXPECT(!p.fused || (p.splits * m <= kJoinRows && p.strips <= kCounters && p.splits > 1));
  EXPECT(p.lds >= (uint32_t)kWaves * ((m < 16 ? m : 16) * CW * 4) && p.lds <= 128 * 1024);
  if (!plan_fits(p, m, k, dev)) return;
  // offsets of the ranges' sums: the last float of the last range, in 32 bits
  if (p.splits > 1)
    EXPECT(((int64_t)p.splits * m * k - 1) * 4 < (int64_t)1 << 31 && sums_bytes(p, m, k) == (size_t)p.splits * m * k * 4);
}

int main() {
  // the kernels' own costs, and ones that split always or hardly ever
  const SplitCost costs[] = {{4, 4, 14}, {4, 7, 1 << 20}, {3, 3, 28}, {1, -1, 1 << 20}, {1, 0, 1}, {7, 0, 1 << 20}};
  for (int cus : {256, 304, 128, 40, 8, 1})
    for (const SplitCost& c : costs) {
      for (int tm = 1; tm <= 9; ++tm)
        for (int tn : {1, 2, 3, 5, 8, 20, 33, 68})
          for (int iters : {1, 2, 3, 4, 5, 7, 8, 13, 32, 33}) walk(tm, tn, iters, c, cus);
    }
  std::mt19937 rng(3);
  auto any = [&](int lo, int hi) { return lo + (int)(rng() % (uint32_t)(hi - lo + 1)); };
  for (int i = 0; i < 3000; ++i) walk(any(1, 40), any(1, 40), any(1, 300), costs[any(0, 5)], any(0, 3) ? 256 : any(1, 304));
  // long sums: fewer than 2^21 steps, up to 32 leftover tiles per XCD
  for (int tiles : {1, 7, 8, 9, 100, 255, 256, 257, 511})
    for (int iters : {1000, 65535, (1 << 20) + 3, (1 << 21) - 1})
      for (const SplitCost& c : costs) positions(tiles, iters, c, 256);
  // ... and one tile of up to 2^23 (a product with few outputs and the longest sums)
  for (const SplitCost& c : costs) positions(1, 1 << 23, c, 256);

  for (int m = 1; m <= kSkinnyTRows; ++m)
    for (int cus : {256, 304, 64, 1}) {
      for (int64_t n : {1, 2, 31, 32, 33, 255, 256, 257, 1000, 2003, 5120, 17408, 34816})
        for (int64_t k : {32, 64, 224, 256, 288, 1024, 2080, 5120, 17408, 70016}) skinny(m, n, k, cus);
      // weights, d and y near their limit of 2 GiB
      for (int64_t k : {(int64_t)32, (int64_t)1024, (int64_t)1 << 20, ((int64_t)1 << 30) / m / 32 * 32}) {
        int64_t n = (((int64_t)1 << 31) - 1) / (k / 2);
        const int64_t most = (((int64_t)1 << 30) - 8) / m;
        n = n < most ? n : most;
        if (n >= 1 && 2 * m * k < (int64_t)1 << 31) skinny(m, n, k, cus);
      }
    }
  std::printf("plan driver: ok (%ld plans)\n", g_plans);
  return 0;
}
