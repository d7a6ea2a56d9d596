// gemm_t.hip -- the product with the other side of the int4 weights, tiled for many rows:
// y[m, k] = sum_n d[m, n] * s[n, k / g] * q[n, k] on gfx950 (fp16 MFMA).
//
// This is the input gradient of the W4A16 layer (d = dy), and of the gate/up pair
// of a SwiGLU feed-forward (d = the pair's gradient).  The weights keep the one
// packed layout of the forward product, eight codes per word along k, so here the
// words run along an output dimension and the sum crosses them.
//
// * Operands: an MFMA operand lane needs eight consecutive n of one column k.  The
//   LDS transpose read (ds_read_b64_tr_b4) turns a 16 x 16 block of nibbles around
//   on the way to the registers: lane i of sixteen names row n_i, and lane j gets
//   nibble j of all sixteen rows.  Its rows are named in the order 0 2 4 6 1 3 5 7,
//   so that nibbles p and p + 4 of a result word are neighbours in n: one AND-OR
//   per pair makes fp16 1024 + u or 64 + u of them, one packed subtraction the code
//   and one packed multiplication by the two rows' scales the operand q s, rounded
//   once to fp16 (the operand precision of the forward GEMM): 13 VALU per 8 weights.
// * Scales differ along the sum here, so a K step's scales are staged in LDS
//   [group][n] and read eight at a time (one broadcast 16-byte read per sub-step).
// * Tiles: 256 x 256 outputs, steps of 64 n, eight wavefronts of 128 x 64 (4 x 2
//   blocks of v_mfma_f32_32x32x16_f16): each dequantised fragment feeds four MFMAs
//   and each activation fragment two, so a sub-step of 8 MFMAs (256 cycles) takes 26
//   VALU and 5.5 LDS reads of 16 bytes per lane.
// * Gradient rows and packed weights reach a three-stage LDS ring straight from
//   memory, two steps ahead; 16-byte chunks are XOR-swizzled so the operand reads
//   spread over the banks.
// * Work split: whole tiles in data-parallel rounds, the leftover tiles split along
//   n (stream-K).  Partial tiles go to the workspace and a second, small kernel adds
//   them in contributor order: no workgroup waits for another, so calls on several
//   streams cannot hold each other up, and the workspace holds no state.
// * Measured (MI355X; boxes differ): 4096 rows 17408 -> 5120 599-636 us with its join (1.15-1.22 PFLOP/s;
//   the best dense fp16 library product measured beside it reached 1.16); 512 rows 109-120 us; 300
//   rows 2003 -> 2080 25 us: padded rows 5, tiles 15, join 6.  Bound at many rows by power: MFMAs busy 69%
//   of the time at 1.6 GHz (with scales of one bit, i.e. operands of few, the same code takes 6% less
//   time); at few hundred rows by the steps' latency and the partial tiles' way through memory.
//   A product whose tiles are all split (160 tiles: the backward pass at 2048 rows) reads 3.7 GB instead of
//   0.84, as the workgroups of an XCD are at different places of the sum and share nothing in its L2.
// * Measured slower: loads three steps ahead with a barrier inside the step (3%), no
//   scheduling groups (1-2%), segments of fewer than four steps (kCost).
#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "tile_gemm.hpp"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int BM = 256, BC = 256, BR = 64;     // output rows, output columns, n per step
constexpr int kSub = BR / 16;                   // MFMA sub-steps per step
constexpr int kMB = 4, kNB = 2;                 // 32 x 32 blocks per wave
constexpr int kABytes = BM * BR * 2;            // gradient tile: 256 rows of 128 bytes
constexpr int kBBytes = BR * BC / 2;            // packed weight tile: 64 rows of 128 bytes
constexpr size_t kPartialBytes = (size_t)BM * BC * 4;
// Steps per stream-K segment, at least.  8 / 5 / 4 / 3 steps: 128 x 1024 x 1024 13.2 / 12.0 /
// 10.9 / 11.4 us, 300 x 2000 x 2080 22.6 / 23.1 / 22.5 / 26 us; larger products unchanged.
// A join: four steps, and one per 14 partial tiles (256 KB each, written and read).  Whole against
// split tiles, device time: 64 x 320 -> 1024 (5 steps) 8.3 / 9.9 us, 64 x 512 -> 1024 (8) 10.4 / 9.3 (but
// 2.4 us more of the host's time), 64 x 768 -> 1024 (12) 13.2 / 9.4, 300 x 1024 -> 2080 (16) 24.2 / 18.2;
// 2048 rows, 160 tiles: 512 -> 5120 (8) 18.1 / 43.8, 1024 -> 5120 (16) 30.7 / 51.4.
constexpr SplitCost kCost = {4, 4, 14};

// The operand values q s of eight n of one column: word w holds the codes of n0 n2
// n4 n6 n1 n3 n5 n7, sc their scales in the order n0 .. n7.
__device__ inline f16x8 dequant_transposed(uint32_t w, const u32x4& sc, uint32_t m_lo, uint32_t m_hi, uint32_t e_lo,
                                           uint32_t e_hi) {
  const uint32_t w8 = w >> 8;
  const uint32_t t[4] = {(w & m_lo) | e_lo, (w & m_hi) | e_hi, (w8 & m_lo) | e_lo, (w8 & m_hi) | e_hi};
  const f16x2 b_lo = {(_Float16)-1032.f, (_Float16)-1032.f}, b_hi = {(_Float16)-72.f, (_Float16)-72.f};
  // whole vectors are cast (a bit cast of one vector element takes the first)
  const f16x8 s8 = __builtin_bit_cast(f16x8, sc);
  f16x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 v = (__builtin_bit_cast(f16x2, t[i]) + (i & 1 ? b_hi : b_lo)) * f16x2{s8[2 * i], s8[2 * i + 1]};
    r[2 * i] = v[0];
    r[2 * i + 1] = v[1];
  }
  return r;
}

__device__ inline void schedule_substep() {
#pragma unroll
  for (int i = 0; i < kMB * kNB; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);             // LDS read
    if (i < 6) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // global load
    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);             // VALU
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int G>
__global__ void __launch_bounds__(kThreads)
gemm_t_kernel(const uint16_t* __restrict__ d, const uint32_t* __restrict__ packed, const uint16_t* __restrict__ scales,
              uint16_t* __restrict__ y, int M, int N, int K, uint32_t dpitch, SplitPlan plan,
              float* __restrict__ partials) {
  constexpr int kGroups = BC / G;                 // scale groups per tile (2 or 8)
  constexpr int kSBytes = kGroups * BR * 2;
  constexpr int kStage = kABytes + kBBytes + kSBytes;
  static_assert(3 * kStage <= 160 * 1024, "LDS use exceeds 160 KB");
  __shared__ __attribute__((aligned(16))) uint8_t stage0[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t stage1[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t stage2[kStage];
  auto stage = [&](int st) -> uint8_t* { return st == 0 ? stage0 : (st == 1 ? stage1 : stage2); };

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;        // 128-row half, 64-column quarter
  const int h = lane >> 5, li = lane & 31;

  const uint32_t wrow = (uint32_t)K >> 1;
  const uint32_t spr = (uint32_t)K / (uint32_t)G;
  const __amdgpu_buffer_rsrc_t dres = make_rsrc(d, (uint32_t)M * dpitch);
  const __amdgpu_buffer_rsrc_t wres = make_rsrc(packed, (uint32_t)N * wrow);
  const __amdgpu_buffer_rsrc_t sres = make_rsrc(scales, (uint32_t)N * spr * 2u);

  // ---- gradient tile: row r of 128 bytes, 16-byte chunk c (8 n) stored at c ^ (r / 2 % 8): the
  // sixteen lanes of a read phase cover 256 bytes (two rows share a place, in either 128-byte half).
  // Load j of wave w fills rows 64 j + 8 w .. + 7 (lane i: row + i / 8, stored chunk i % 8).
  const int a_row = tid >> 3;                                        // + 64 j
  const int a_chunk = (tid & 7) ^ ((a_row >> 1) & 7);
  // per item: the byte offset of the thread's chunk in each of its four rows, outside the
  // buffer for rows past M (the step's offset, at most a row, goes into the scalar offset)
  uint32_t a_v[4];
  auto set_rows = [&](int r0) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      a_v[p] = r0 + 64 * p + a_row < M ? (uint32_t)(r0 + 64 * p + a_row) * dpitch + (uint32_t)a_chunk * 16u : kOutOfRange;
  };
  // Operand reads: sub-step s takes chunk 4 h + s (n = 32 h + 8 s .. + 7) of row 128 wm + 32 i + li.
  uint32_t a_r[kSub];
#pragma unroll
  for (int s = 0; s < kSub; ++s)
    a_r[s] = (uint32_t)(128 * wm + li) * 128u + (uint32_t)(((4 * h + s) ^ ((li >> 1) & 7)) << 4);

  // ---- packed tile: row n of 128 bytes, chunk c (32 columns) stored at c ^ ((n / 2) % 8), so
  // that the sixteen rows of a transpose read fall on distinct banks (two rows share a chunk
  // place and differ in the row's 128-byte half).  Wave w loads rows 8 w .. 8 w + 7.
  const int b_row = tid >> 3;
  const int b_chunk = (tid & 7) ^ ((b_row >> 1) & 7);
  const uint32_t b_v = (uint32_t)b_row * wrow + (uint32_t)b_chunk * 16u;
  // Transpose reads: read t covers sub-steps 2 t, 2 t + 1, i.e. rows 32 h + 16 t .. + 15; the
  // lane's sixteenth names row 8 (p / 8) + (0 2 4 6 1 3 5 7)[p % 8], p = lane % 16; columns
  // 64 wn + 32 nb + 16 (lane / 16 % 2) .. + 15 are half a chunk.
  const int p16 = lane & 15;
  const int b_n = 32 * h + 8 * (p16 >> 3) + 2 * (p16 & 3) + ((p16 >> 2) & 1);
  uint32_t b_r[2][kNB];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) {
      const int n = b_n + 16 * t;
      b_r[t][nb] = (uint32_t)kABytes + (uint32_t)n * 128u + (uint32_t)(((2 * wn + nb) ^ ((n >> 1) & 7)) << 4) +
                   8u * (uint32_t)((lane >> 4) & 1);
    }

  // ---- scales of a step: [group][64 n] fp16; thread t < 64 kGroups loads group t % kGroups of
  // row t / kGroups and stores it a step later.
  const bool s_live = tid < BR * kGroups;
  const int s_n = tid / kGroups, s_g = tid % kGroups;
  const uint32_t s_v = (uint32_t)s_n * spr * 2u + (uint32_t)s_g * 2u;
  const uint32_t s_w = (uint32_t)(kABytes + kBBytes) + (uint32_t)(s_g * BR + s_n) * 2u;
  // reads: the group of the wave's columns (g 128: one; g 32: one per block)
  auto s_r = [&](int nb, int s) -> uint32_t {
    const int g = G == 128 ? (wn >> 1) : 2 * wn + nb;
    return (uint32_t)(kABytes + kBBytes) + (uint32_t)(g * BR + 32 * h + 8 * s) * 2u;
  };
  constexpr int kSV = G == 128 ? 1 : kNB;         // scale reads per sub-step

  const uint32_t m_lo = __builtin_amdgcn_readfirstlane(0x000F000Fu), m_hi = __builtin_amdgcn_readfirstlane(0x00F000F0u);
  uint32_t e_lo = 0x64006400u, e_hi = 0x54005400u;     // fp16 1024 and 64, both halves
  asm volatile("" : "+v"(e_lo), "+v"(e_hi));

  const WorkRange wr(plan, blockIdx.x);
  const int n_items = wr.count(plan);

  // Part p of step kt of the tile at (m0, c0) into stage st: gradients (p < 4), weights (p = 4).
  // Chunks past N are sent outside the buffer (zeros), rows of weights past N lie outside it.
  auto load_part = [&](const TileItem& it, int kt, int st, int p) {
    uint8_t* base = stage(st);
    if (p < 4) {
      const bool ok = kt * BR + a_chunk * 8 < N;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(dres, W4A16_LDS(base + (64 * p + 8 * wave) * 128), 16,
                                               ok ? a_v[p] : kOutOfRange, (uint32_t)kt * (BR * 2), 0, 0);
    } else {
      const bool ok = kt * BR + b_row < N;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, W4A16_LDS(base + kABytes + 8 * wave * 128), 16,
                                               ok ? b_v : kOutOfRange,
                                               (uint32_t)kt * BR * wrow + (uint32_t)(it.c0 >> 1), 0, 0);
    }
  };
  auto load_scale = [&](const TileItem& it, int kt) -> uint16_t {
    const bool ok = s_live && kt * BR + s_n < N && it.c0 / G + s_g < (int)spr;
    return __builtin_amdgcn_raw_buffer_load_b16(
        sres, ok ? s_v + (uint32_t)kt * BR * spr * 2u + (uint32_t)(it.c0 / G) * 2u : kOutOfRange, 0, 0);
  };
  auto store_scale = [&](int st, uint16_t v) {
    if (s_live) *reinterpret_cast<uint16_t*>(stage(st) + s_w) = v;
  };
  auto clamp_of = [&](const TileItem& it, int r) { return it.a + (r < it.b - it.a ? r : it.b - it.a - 1); };
  // What an item needs before its first step: steps 0 and 1 whole, and the scales of step 2 on their way.
  uint16_t sreg[3];
  auto prologue_loads = [&](const TileItem& it) {
    set_rows(it.r0);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      for (int p = 0; p < 5; ++p) load_part(it, clamp_of(it, r), r, p);
      sreg[r] = load_scale(it, clamp_of(it, r));
    }
    sreg[2] = load_scale(it, clamp_of(it, 2));
  };
  auto read_a = [&](int st, int s, u32x4 (&dst)[kMB]) {
#pragma unroll
    for (int i = 0; i < kMB; ++i) dst[i] = *reinterpret_cast<const u32x4*>(stage(st) + a_r[s] + i * 32 * 128);
  };
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  auto read_w = [&](int st, int t, i32x2 (&dst)[kNB]) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
      dst[nb] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
          (__attribute__((address_space(3))) i32x2*)(stage(st) + b_r[t][nb]));
  };
  auto read_s = [&](int st, int s, u32x4 (&dst)[kSV]) {
#pragma unroll
    for (int v = 0; v < kSV; ++v) dst[v] = *reinterpret_cast<const u32x4*>(stage(st) + s_r(v, s));
  };
  auto dequant = [&](const i32x2 (&w)[kNB], int half, const u32x4 (&sc)[kSV], f16x8 (&dst)[kNB]) {
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb)
      dst[nb] = dequant_transposed((uint32_t)(half ? w[nb].y : w[nb].x), sc[kSV == 1 ? 0 : nb], m_lo, m_hi, e_lo, e_hi);
  };

  TileItem cur{};
  if (n_items > 0) {
    cur = wr.item(plan, 0, BM, BC);
    prologue_loads(cur);
  }
  for (int item = 0; item < n_items; ++item) {
    const bool dp = item >= wr.n_seg;
    const int nsteps = cur.b - cur.a;
    // 32-row blocks of this wave with rows below M.  A wave without any (the second half of a
    // last tile) only loads its share: its SIMD's other wave has the matrix core to itself.
    const int live = min(kMB, (M - cur.r0 - 128 * wm + 31) >> 5);
    if (live <= 0) {
      store_scale(0, sreg[0]);
      store_scale(1, sreg[1]);
      lds_barrier();
      auto idle_step = [&](int st, int r) {
        store_scale(st, sreg[2]);
        sreg[2] = load_scale(cur, clamp_of(cur, r + 3));
        for (int p = 0; p < 5; ++p) load_part(cur, clamp_of(cur, r + 2), st, p);
        lds_barrier();
      };
      for (int r = 0;;) {
        idle_step(2, r);
        if (++r == nsteps) break;
        idle_step(0, r);
        if (++r == nsteps) break;
        idle_step(1, r);
        if (++r == nsteps) break;
      }
      if (item + 1 < n_items) {
        cur = wr.item(plan, item + 1, BM, BC);
        prologue_loads(cur);
      }
      continue;
    }

    f32x16 acc[kMB][kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) acc[i][nb] = f32x16{};

    // Registers carried across sub-steps: operands of this and the next one, the packed
    // words of two sub-steps (halves of a transpose read) twice, scales of two sub-steps.
    u32x4 aop[2][kMB];
    i32x2 wv[2][kNB];
    u32x4 sv[2][kSV];
    f16x8 bop[2][kNB];

    store_scale(0, sreg[0]);
    store_scale(1, sreg[1]);
    lds_barrier();
    read_a(0, 0, aop[0]);
    read_w(0, 0, wv[0]);
    read_s(0, 0, sv[0]);
    read_s(0, 1, sv[1]);
    dequant(wv[0], 0, sv[0], bop[0]);

    // One step r (stage r % 3 == U): loads step r + 2 into the stage step r - 1 used; the
    // barrier at its end publishes it.
    auto step = [&](auto u_tag, int r) {
      constexpr int U = decltype(u_tag)::value;
      constexpr int st_cur = U, st_nxt = (U + 1) % 3, st_ld = (U + 2) % 3;
      store_scale(st_ld, sreg[2]);
      sreg[2] = load_scale(cur, clamp_of(cur, r + 3));
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        // (all of them in the first sub-step: the barrier at the step's end waits for them)
        if (s == 0)
          for (int p = 0; p < 5; ++p) load_part(cur, clamp_of(cur, r + 2), st_ld, p);
        // operands of sub-step s + 1, scales of s + 2, words of the pair after next
        if (s + 1 < kSub) read_a(st_cur, s + 1, aop[(s + 1) & 1]);
        else read_a(st_nxt, 0, aop[(s + 1) & 1]);
        if (s == 0) read_w(st_cur, 1, wv[1]);
        if (s == 2) read_w(st_nxt, 0, wv[0]);
        dequant(wv[((s + 1) >> 1) & 1], (s + 1) & 1, sv[(s + 1) & 1], bop[(s + 1) & 1]);
        if (s + 2 < kSub) read_s(st_cur, s + 2, sv[s & 1]);
        else read_s(st_nxt, s + 2 - kSub, sv[s & 1]);
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb)
            acc[i][nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, aop[s & 1][i]),
                                                                bop[s & 1][nb], acc[i][nb], 0, 0, 0);
        schedule_substep();
      }
      lds_barrier();
    };
    for (int r = 0;;) {
      step(std::integral_constant<int, 0>{}, r);
      if (++r == nsteps) break;
      step(std::integral_constant<int, 1>{}, r);
      if (++r == nsteps) break;
      step(std::integral_constant<int, 2>{}, r);
      if (++r == nsteps) break;
    }

    // The next item's first loads, before this one's results are written (stages 0 and 1 are free).
    const TileItem done = cur;
    if (item + 1 < n_items) {
      cur = wr.item(plan, item + 1, BM, BC);
      prologue_loads(cur);
    }

    if (dp) {
      // Through LDS (stage 2): 32 rows x 64 columns per wave and pass, row pitch 144 bytes,
      // then 16-byte stores, eight lanes per 128-byte row piece.  K is a multiple of 32, so a
      // piece of 8 columns is whole or absent and 16-byte aligned.
      constexpr int kPitch = 64 * 2 + 16;
      static_assert(8 * 32 * kPitch <= kStage, "epilogue slabs exceed stage 2");
      uint8_t* ep = stage2 + wave * 32 * kPitch;
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            *reinterpret_cast<uint16_t*>(ep + (8 * (r >> 2) + 4 * h + (r & 3)) * kPitch + (32 * nb + li) * 2) =
                float_to_half_bits(acc[i][nb][r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 8 * j + (lane >> 3), c = lane & 7;
          const u32x4 v = *reinterpret_cast<const u32x4*>(ep + row * kPitch + c * 16);
          const int m = done.r0 + 128 * wm + 32 * i + row, k = done.c0 + 64 * wn + 8 * c;
          if (m < M && k < K) *reinterpret_cast<u32x4*>(y + (size_t)m * K + k) = v;
        }
      }
    } else {
      // fp32 partial tile of segment `item`: 16-byte quad q of block blk of thread t at
      // ((4 blk + q) 512 + t) 16, so every store covers 1 KB contiguously
      uint8_t* slot = reinterpret_cast<uint8_t*>(partials) + (size_t)(2 * blockIdx.x + item) * kPartialBytes;
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
        if (i >= live) break;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = {acc[i][nb][4 * q], acc[i][nb][4 * q + 1], acc[i][nb][4 * q + 2], acc[i][nb][4 * q + 3]};
            *reinterpret_cast<f32x4*>(slot + (size_t)(((i * kNB + nb) * 4 + q) * kThreads + tid) * 16) = v;
          }
      }
    }
  }
}

// Adds the partial tiles of each stream-K tile in contributor order and writes fp16: one thread
// per 16-byte quad (four rows of a column).
constexpr int kQuads = kMB * kNB * 4 * kThreads;
__global__ void __launch_bounds__(256)
gemm_t_join_kernel(const float* __restrict__ partials, uint16_t* __restrict__ y, int M, int K, SplitPlan plan) {
  const int tile = blockIdx.x / (kQuads / 256), c = (blockIdx.x % (kQuads / 256)) * 256 + threadIdx.x;
  int tm, tn;
  tile_coords(plan.rounds * plan.wgs + tile, plan.tiles_m, plan.tiles_n, tm, tn);
  const int t = c % kThreads, bq = c / kThreads, blk = bq >> 2, q = bq & 3;
  const int wave = t >> 6, h = (t >> 5) & 1, li = t & 31;
  const int k = tn * BC + 64 * (wave & 3) + 32 * (blk % kNB) + li;
  const int m0 = tm * BM + 128 * (wave >> 2) + 32 * (blk / kNB) + 8 * q + 4 * h;
  if (k >= K || m0 >= M) return;
  const Contributors cs(plan, tile);
  const uint8_t* base = reinterpret_cast<const uint8_t*>(partials) + (size_t)c * 16;
  f32x4 v = f32x4{};
  for (int l = cs.first; l <= cs.last; l += 4) {       // four loads in flight
    f32x4 p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      p[u] = *reinterpret_cast<const f32x4*>(base + (size_t)cs.slot(min(l + u, cs.last)) * kPartialBytes);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (l + u <= cs.last) v += p[u];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (m0 + r < M) y[(size_t)(m0 + r) * K + k] = float_to_half_bits(v[r]);
}

// d [m, n] copied with the row pitch padded to 8 elements (zeros), for an n that is no multiple of
// 8: a thread makes one 16-byte chunk.  Against one element per thread and a grid row per row of d,
// whole calls: 4096 x 17407 -> 5120 666 / 731 us, 300 x 2003 -> 2080 25.1 / 25.8, 64 x 401 -> 416 11.8 / 11.6.
__global__ void __launch_bounds__(256)
pad_rows_kernel(const uint16_t* __restrict__ d, uint16_t* __restrict__ out, uint32_t n, uint32_t per, uint32_t chunks) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint32_t row = i / per, c = (i - row * per) * 8;       // per: chunks of a padded row
  const uint16_t* src = d + (size_t)row * n;
  uint16_t t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = src[c + e < n ? c + e : n - 1];
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    v[e >> 1] = (c + e < n ? t[e] : 0u) | (c + e + 1 < n ? (uint32_t)t[e + 1] << 16 : 0u);
  *reinterpret_cast<u32x4*>(out + (size_t)i * 8) = v;
}

SplitPlan plan_of(int m, int n, int k, const DeviceInfo& dev) {
  return split_plan((m + BM - 1) / BM, (k + BC - 1) / BC, (n + BR - 1) / BR, kCost, dev);
}

}  // namespace

size_t gemm_t_workspace_bytes(int m, int n, int k, const DeviceInfo& dev) {
  const SplitPlan p = plan_of(m, n, k, dev);
  const size_t bytes = padded_bytes(m, n) + split_slots(p) * kPartialBytes;
  return bytes ? kCounterBytes + bytes : 0;
}

hipError_t launch_pad_rows(const uint16_t* d, uint16_t* out, int m, int n, hipStream_t stream) {
  const uint32_t per = (uint32_t)(n + 7) / 8, chunks = (uint32_t)m * per;      // (fewer than 2^27)
  return launch_kernel(pad_rows_kernel, dim3((chunks + 255) / 256), dim3(256), 0, stream, d, out, (uint32_t)n, per,
                       chunks);
}

uint16_t* gemm_t_padded(int n, void* workspace) {
  return n % 8 ? reinterpret_cast<uint16_t*>(behind_counters(workspace)) : nullptr;
}

hipError_t launch_gemm_t(const uint16_t* d, const uint32_t* packed, const uint16_t* scales, uint16_t* y, int m, int n,
                         int k, int group, void* workspace, const DeviceInfo& dev, hipStream_t stream) {
  const SplitPlan p = plan_of(m, n, k, dev);
  uint8_t* ws = workspace ? behind_counters(workspace) : nullptr;
  uint32_t pitch = (uint32_t)n * 2u;
  if (n % 8) {
    if (d) {
      const hipError_t e = launch_pad_rows(d, reinterpret_cast<uint16_t*>(ws), m, n, stream);
      if (e != hipSuccess) return e;
    }
    d = reinterpret_cast<uint16_t*>(ws);
    pitch = (uint32_t)((n + 7) / 8 * 8) * 2u;
    ws += padded_bytes(m, n);
  }
  float* partials = p.sk_tiles ? reinterpret_cast<float*>(ws) : nullptr;
  hipError_t e = launch_kernel(group == 128 ? gemm_t_kernel<128> : gemm_t_kernel<32>, dim3(p.wgs), dim3(kThreads), 0,
                               stream, d, packed, scales, y, m, n, k, pitch, p, partials);
  if (e != hipSuccess || p.sk_tiles == 0) return e;
  return launch_kernel(gemm_t_join_kernel, dim3((unsigned)p.sk_tiles * (kQuads / 256)), dim3(256), 0, stream,
                       partials, y, m, k, p);
}

}  // namespace w4a16
