// dscales.hip -- gradient of the group scales of the int4 weights on gfx950 (fp16 MFMA):
// ds[n, j] = sum_{k in group j} q[n, k] * (sum_m d[m, n] x[m, k]).
//
// y = x . W^T with W[n, k] = s[n, j] q[n, k] is linear in the scales, so the scales'
// gradient is the weight gradient dW = d^T . x, weighted by the codes and summed over
// each group.  dW itself (n x k fp32, 356 MB for the dense up projection) never leaves
// the registers: a group of 128 shrinks it by that factor.
//
// * dW is a dense product whose sum runs over the rows of both inputs, so both
//   operands come from row-major tiles through the 16-bit LDS transpose read
//   (ds_read_b64_tr_b16: a 4 x 16 block per sixteen lanes, lane j gets column j).
//   Tiles of 256 n x 256 k, steps of 32 rows m, eight wavefronts of 128 x 64 (4 x 2
//   blocks of v_mfma_f32_32x32x16_f16); no VALU work in the loop.
// * A tile row is 512 bytes; its 16-byte chunk c is stored at c ^ 4 (row % 4), which
//   puts the four rows of a transpose read on distinct banks.
// * Epilogue: an accumulator holds one column k of sixteen rows n per lane, so one
//   ds_read_b64_tr_b4 of the packed tile brings a lane exactly its sixteen codes.
//   acc * code is summed over the 32 lanes of a block by halving (each exchange sums
//   two rows and keeps one per lane: 2.4 operations per accumulator instead of 10),
//   which leaves lane l rows 2 l and 2 l + 1 of the wave's 64 per half.
// * Leftover tiles are split along m as in split_plan.hpp; a part is 256 x groups fp32
//   (2 or 8 KB), and a second kernel adds the parts in order (adding them in the last
//   contributor instead measured 6 us slower at 133 rows: its stores, its arrival and its
//   loads each pay the device-scope latency in turn).  Sums are fp32 throughout, products
//   of fp16 pairs exact; results do not depend on timing.
// * Measured (MI355X; boxes differ): 2048 rows, 17408 x 5120 314-325 us = 1.12-1.16 PFLOP/s (8192 rows 1235
//   us), the rate of a large dense library product: bound by the matrix cores at the clock their
//   power leaves (MFMAs busy 60% of the time at 1.77 GHz); 133 rows, 1001 x 1120 11.4 us with the
//   padding, one step's latency after another.
#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "tile_gemm.hpp"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int BN = 256, BC = 256, BR = 32;      // weight rows, weight columns, rows m per step
constexpr int kSub = BR / 16;
constexpr int kMB = 4, kNB = 2;                  // 32 x 32 blocks per wave
constexpr int kTileBytes = BR * 512;             // one operand's tile of a step
constexpr int kStage = 2 * kTileBytes;
// A join takes the time of seven steps, whatever the parts (2 or 8 KB each).  Whole against split
// tiles, device time, 1024 x 1024: 64 rows (2 steps) 7.3 / 9.4 us, 160 (5) 8.7 / 10.9, 256 (8)
// 10.1 / 10.8, 384 (12) 12.0 / 11.4, 512 (16) 13.7 / 11.8; 133 rows 1001 x 1120 11.4 / 16.3.
constexpr SplitCost kCost = {4, 7, 1 << 20};
constexpr int kStepLoads = 4;                    // vector loads of a wave per step

__device__ inline void schedule_substep() {
#pragma unroll
  for (int i = 0; i < kMB * kNB; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);             // LDS reads
    if (i < kStepLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // global load
    __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);             // VALU
  }
  __builtin_amdgcn_sched_barrier(0);
}

// Barrier inside a step: every LDS access of this wave is complete, and of its vector memory
// accesses all but (at most) the newest kStepLoads, one step's loads.
__device__ inline void step_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(kStepLoads | (7 << 4));       // vmcnt(kStepLoads) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// a + b of two values over lane pairs: lanes whose `bit` is clear keep a, the others b.
template <int CTRL>
__device__ inline float halve(float a, float b, bool bit) {
  const float keep = bit ? b : a, send = bit ? a : b;
  return keep + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, send), CTRL, 0xf, 0xf,
                                                                      false));
}

template <int G>
__global__ void __launch_bounds__(kThreads)
dscales_kernel(const uint16_t* __restrict__ d, const uint16_t* __restrict__ x, const uint32_t* __restrict__ packed,
               float* __restrict__ ds, int M, int N, int K, uint32_t dpitch, SplitPlan plan,
               float* __restrict__ partials) {
  constexpr int kGroups = BC / G;                // groups per tile (2 or 8)
  __shared__ __attribute__((aligned(16))) uint8_t stage0[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t stage1[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t stage2[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t codes[BN * BC / 2];
  __shared__ float sums[4][BN];                  // g 128: the halves of a group, by column quarter
  auto stage = [&](int st) -> uint8_t* { return st == 0 ? stage0 : (st == 1 ? stage1 : stage2); };

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int h = lane >> 5, li = lane & 31, p16 = lane & 15, half = (lane >> 4) & 1;

  const uint32_t wrow = (uint32_t)K >> 1, xpitch = (uint32_t)K * 2u;
  const int spr = K / G;
  const __amdgpu_buffer_rsrc_t dres = make_rsrc(d, (uint32_t)M * dpitch);
  const __amdgpu_buffer_rsrc_t xres = make_rsrc(x, (uint32_t)M * xpitch);
  const __amdgpu_buffer_rsrc_t wres = make_rsrc(packed, (uint32_t)N * wrow);

  // ---- loads: load j of wave w fills rows 2 w + 16 j, + 1 (lane i: row + i / 32, stored chunk i % 32)
  const int l_row = 2 * wave + h;                                      // + 16 j
  const int l_chunk = li ^ (4 * (l_row & 3));
  // ---- transpose reads: quad q of sub-step s, block b: rows 16 s + 8 h + 4 q + p16 / 4, columns
  // base + 32 b + 16 half + 4 (p16 % 4) .. + 3.  (row % 4) = p16 / 4, so the swizzle is the lane's.
  const uint32_t r_lane = (uint32_t)(8 * h + (p16 >> 2)) * 512u;
  auto r_col = [&](int base, int b) -> uint32_t {
    const int byte = (base + 32 * b + 16 * half + 4 * (p16 & 3)) * 2;
    return (uint32_t)(((byte >> 4) ^ (4 * (p16 >> 2))) << 4) + (uint32_t)(byte & 15);
  };
  uint32_t a_r[kMB], b_r[kNB];
#pragma unroll
  for (int i = 0; i < kMB; ++i) a_r[i] = r_lane + r_col(128 * wm, i);
#pragma unroll
  for (int nb = 0; nb < kNB; ++nb) b_r[nb] = (uint32_t)kTileBytes + r_lane + r_col(64 * wn, nb);

  // ---- codes: packed row n of 128 bytes, chunk c at c ^ (n % 8); a transpose read names the
  // sixteen rows n of a lane's accumulators, r = p16: 8 (r / 4) + 4 h + r % 4.
  const int c_row = tid >> 3, c_chunk = (tid & 7) ^ (c_row & 7);        // rows c_row + 64 j
  const int c_n = 128 * wm + 8 * (p16 >> 2) + 4 * h + (p16 & 3);        // + 32 i

  const WorkRange wr(plan, blockIdx.x);
  const int n_items = wr.count(plan);

  // Part p of step r of an item into stage st: d (p = 0, 1), x (p = 2, 3).  Rows past M, and
  // steps past the item's last, go outside the buffers (no memory access, zeros); chunks past
  // a row's end only feed outputs that are not stored.
  auto load_part = [&](const TileItem& it, int r, int st, int p) {
    const int row = l_row + 16 * (p & 1);
    const bool in = r < it.b - it.a;
    const int kt = in ? it.a + r : it.a;
    const bool ok = in && kt * BR + row < M;
    uint8_t* dst = stage(st) + (p < 2 ? 0 : kTileBytes) + (2 * wave + 16 * (p & 1)) * 512;
    if (p < 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(dres, W4A16_LDS(dst), 16,
                                               ok ? (uint32_t)row * dpitch + (uint32_t)l_chunk * 16u : kOutOfRange,
                                               (uint32_t)kt * BR * dpitch + (uint32_t)it.r0 * 2u, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xres, W4A16_LDS(dst), 16,
                                               ok ? (uint32_t)row * xpitch + (uint32_t)l_chunk * 16u : kOutOfRange,
                                               (uint32_t)kt * BR * xpitch + (uint32_t)it.c0 * 2u, 0, 0);
  };
  auto load_step = [&](const TileItem& it, int r, int st) {
#pragma unroll
    for (int p = 0; p < 4; ++p) load_part(it, r, st, p);
  };
  auto load_codes = [&](const TileItem& it) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = it.r0 + 64 * j + c_row;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wres, W4A16_LDS(codes + (64 * j + 8 * wave) * 128), 16,
          n < N ? (uint32_t)n * wrow + (uint32_t)(it.c0 >> 1) + (uint32_t)c_chunk * 16u : kOutOfRange, 0, 0, 0);
    }
  };

  typedef short i16x4 __attribute__((ext_vector_type(4)));
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  auto read8 = [&](const uint8_t* p) -> f16x8 {          // rows 0 .. 3 and 4 .. 7 of one column
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p + 4 * 512));
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read_ops = [&](int st, int s, f16x8 (&a)[kMB], f16x8 (&b)[kNB]) {
    const uint8_t* base = stage(st) + s * 16 * 512;
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) b[nb] = read8(base + b_r[nb]);
#pragma unroll
    for (int i = 0; i < kMB; ++i) a[i] = read8(base + a_r[i]);
  };

  TileItem cur{};
  if (n_items > 0) {
    cur = wr.item(plan, 0, BN, BC);
    for (int r = 0; r < 3; ++r) load_step(cur, r, r);
  }
  for (int item = 0; item < n_items; ++item) {
    const bool dp = item >= wr.n_seg;
    const int nsteps = cur.b - cur.a;
    f32x16 acc[kMB][kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) acc[i][nb] = f32x16{};
    f16x8 aop[2][kMB], bop[2][kNB];
    lds_barrier();
    load_codes(cur);
    read_ops(0, 0, aop[0], bop[0]);

    // One step r (stage r % 3 == U).  Its second sub-step's operands are read in the first; the
    // barrier between them frees the stage, which takes the loads of step r + 3, and publishes
    // step r + 1, whose loads were issued two steps ago.
    auto step = [&](auto u_tag, int r) {
      constexpr int U = decltype(u_tag)::value;
      constexpr int st_cur = U, st_nxt = (U + 1) % 3;
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        if (s + 1 < kSub) {
          read_ops(st_cur, s + 1, aop[(s + 1) & 1], bop[(s + 1) & 1]);
        } else {
          step_barrier();
          read_ops(st_nxt, 0, aop[(s + 1) & 1], bop[(s + 1) & 1]);
          load_step(cur, r + 3, st_cur);
        }
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb)
            acc[i][nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(aop[s & 1][i], bop[s & 1][nb], acc[i][nb], 0, 0, 0);
        schedule_substep();
      }
    };
    for (int r = 0;;) {
      step(std::integral_constant<int, 0>{}, r);
      if (++r == nsteps) break;
      step(std::integral_constant<int, 1>{}, r);
      if (++r == nsteps) break;
      step(std::integral_constant<int, 2>{}, r);
      if (++r == nsteps) break;
    }
    lds_barrier();               // every wave's codes have arrived (the only loads left to wait for)
    const TileItem done = cur;
    if (item + 1 < n_items) {
      cur = wr.item(plan, item + 1, BN, BC);
      // (every stage is free: needed reads end before a step's barrier, and a wave's loads into
      // one place land in order)
      for (int r = 0; r < 3; ++r) load_step(cur, r, r);
    }

    // ---- codes, then the sum over the 32 columns of each block.  v[b][16 i + r]: accumulator r
    // of block (i, b); for g 128 the two column blocks belong to one group and are added at once.
    constexpr int kB = G == 128 ? 1 : kNB;
    float v[kB][64];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        const int n = c_n + 32 * i;
        const i32x2 w = __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) i32x2*)(
            codes + n * 128 + (((2 * wn + nb) ^ (n & 7)) << 4) + 8 * half));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const uint32_t u = (uint32_t)(r < 8 ? w.x : w.y) ^ 0x88888888u;      // two's complement codes
          const float q = (float)((int32_t)(u << (28 - 4 * (r & 7))) >> 28);
          float& t = v[kB == 1 ? 0 : nb][16 * i + r];
          t = (kB == 1 && nb) ? __builtin_fmaf(q, acc[i][nb][r], t) : q * acc[i][nb][r];
        }
      }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      float* t = v[b];
      // lanes 16 apart: after the swap the two registers hold the halves of value j (lanes
      // 0-15 of each 32) and of value j + 32 (lanes 16-31)
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        // (four exchanges between the wait states that the first and the last one need)
        float a0 = t[j], a1 = t[j + 1], a2 = t[j + 2], a3 = t[j + 3];
        float c0 = t[j + 32], c1 = t[j + 33], c2 = t[j + 34], c3 = t[j + 35];
        asm volatile(
            "s_nop 1\n\tv_permlane16_swap_b32 %0, %4\n\tv_permlane16_swap_b32 %1, %5\n\t"
            "v_permlane16_swap_b32 %2, %6\n\tv_permlane16_swap_b32 %3, %7\n\ts_nop 1"
            : "+v"(a0), "+v"(a1), "+v"(a2), "+v"(a3), "+v"(c0), "+v"(c1), "+v"(c2), "+v"(c3));
        t[j] = a0 + c0;
        t[j + 1] = a1 + c1;
        t[j + 2] = a2 + c2;
        t[j + 3] = a3 + c3;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) t[j] = halve<0x128>(t[j], t[j + 16], lane & 8);   // row_ror:8
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = halve<0x141>(t[j], t[j + 8], lane & 4);     // row_half_mirror
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = halve<0x4E>(t[j], t[j + 4], lane & 2);      // quad_perm [2,3,0,1]
#pragma unroll
      for (int j = 0; j < 2; ++j) t[j] = halve<0xB1>(t[j], t[j + 2], lane & 1);      // quad_perm [1,0,3,2]
    }
    // lane li of half h now has values 2 li, 2 li + 1: row 32 (v / 16) + 8 (v % 16 / 4) + 4 h + v % 4
    const int val = 2 * li;
    const int n_loc = 128 * wm + 32 * (val >> 4) + 8 * ((val & 15) >> 2) + 4 * h + (val & 3);
    // dp: rows n of ds at column c0 / G + group; else the segment's slot, [256][kGroups]
    float* slot = dp ? nullptr : partials + (size_t)(2 * blockIdx.x + item) * (BN * kGroups);
    auto put = [&](int n, int g, float s) {
      if (!dp) slot[n * kGroups + g] = s;
      else if (done.r0 + n < N && done.c0 / G + g < spr) ds[(size_t)(done.r0 + n) * spr + done.c0 / G + g] = s;
    };
    if constexpr (G == 128) {
      sums[wn][n_loc] = v[0][0];
      sums[wn][n_loc + 1] = v[0][1];
      lds_barrier();
      const int n = tid >> 1, g = tid & 1;
      put(n, g, sums[2 * g][n] + sums[2 * g + 1][n]);
      lds_barrier();           // before the next item's sums
    } else {
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        put(n_loc, 2 * wn + b, v[b][0]);
        put(n_loc + 1, 2 * wn + b, v[b][1]);
      }
    }
  }
}

// Adds the parts of each split tile in contributor order: one thread per (row, group).
__global__ void __launch_bounds__(256)
dscales_join_kernel(const float* __restrict__ partials, float* __restrict__ ds, int N, int spr, int groups,
                    SplitPlan plan) {
  const int tile = blockIdx.x / groups, c = (blockIdx.x % groups) * 256 + threadIdx.x;
  const Contributors cs(plan, tile);
  float s = 0.f;
  for (int l = cs.first; l <= cs.last; ++l) s += partials[(size_t)cs.slot(l) * (BN * groups) + c];
  int tm, tn;
  tile_coords(plan.rounds * plan.wgs + tile, plan.tiles_m, plan.tiles_n, tm, tn);
  const int n = tm * BN + c / groups, g = tn * groups + c % groups;
  if (n < N && g < spr) ds[(size_t)n * spr + g] = s;
}

SplitPlan plan_of(int m, int n, int k, const DeviceInfo& dev) {
  return split_plan((n + BN - 1) / BN, (k + BC - 1) / BC, (m + BR - 1) / BR, kCost, dev);
}

}  // namespace

size_t dscales_workspace_bytes(int m, int n, int k, int group, const DeviceInfo& dev) {
  const SplitPlan p = plan_of(m, n, k, dev);
  const size_t bytes = padded_bytes(m, n) + split_slots(p) * BN * (BC / group) * 4;
  return bytes ? kCounterBytes + bytes : 0;
}

hipError_t launch_dscales(const uint16_t* d, const uint16_t* x, const uint32_t* packed, float* ds, int m, int n, int k,
                          int group, void* workspace, const DeviceInfo& dev, hipStream_t stream) {
  const SplitPlan p = plan_of(m, n, k, dev);
  uint8_t* ws = workspace ? behind_counters(workspace) : nullptr;
  uint32_t pitch = (uint32_t)n * 2u;
  if (n % 8) {
    const hipError_t e = launch_pad_rows(d, reinterpret_cast<uint16_t*>(ws), m, n, stream);
    if (e != hipSuccess) return e;
    d = reinterpret_cast<uint16_t*>(ws);
    pitch = (uint32_t)((n + 7) / 8 * 8) * 2u;
    ws += padded_bytes(m, n);
  }
  float* partials = p.sk_tiles ? reinterpret_cast<float*>(ws) : nullptr;
  const hipError_t e = launch_kernel(group == 128 ? dscales_kernel<128> : dscales_kernel<32>, dim3(p.wgs),
                                     dim3(kThreads), 0, stream, d, x, packed, ds, m, n, k, pitch, p, partials);
  if (e != hipSuccess || p.sk_tiles == 0) return e;
  const int groups = BC / group;
  return launch_kernel(dscales_join_kernel, dim3((unsigned)(p.sk_tiles * groups)), dim3(256), 0, stream, partials, ds,
                       n, k / group, groups, p);
}

}  // namespace w4a16
