// gemm_t_skinny.hip -- the product with the other side of the int4 weights for few rows
// (weight-streaming): y[m, k] = sum_n d[m, n] * s[n, k / g] * q[n, k], m <= 32.
//
// With few rows the product is one pass over the packed weights, bound by HBM (0.53 bytes
// per 2 m operations).  The packed words run along k, the output side, so every
// word holds eight output columns of one n:
//
// * A workgroup owns a strip of 256 columns and a range of n; its eight waves take the
//   range's units of 32 n in turn, each for the whole strip.  Lane (lq, li) of a unit loads
//   two words of each of the rows 8 lq .. 8 lq + 7: sixteen lanes read 128 contiguous
//   bytes of a row, a whole line.
// * Two words of neighbouring n give their nibble pairs by one byte permute per four
//   columns; an AND-OR makes fp16 1024 + u or 64 + u of a pair, a packed subtraction the
//   code and a packed multiplication by the two rows' scales the operand q s (rounded
//   once, as in the GEMM; exact weights, by a second MFMA on what the rounding leaves of a scale in two
//   parts, would take 17.4 against 15.8 us at 1 row 17408 -> 5120, 22.4 / 20.9 at 16 rows 5120 -> 17408
//   and 5.8 / 5.4 at 1 row 1024 -> 1024, for an error of 2.1e-4 instead of 2.7e-4).  Eight n of a column are exactly a lane's slice of
//   v_mfma_f32_16x16x32_f16, so a unit is 16 such operands, each used by the one or two
//   blocks of sixteen rows of d.
// * A wave loads what a unit needs, weights, operands of d (already in MFMA layout) and
//   scales, straight to registers; only the scales cross lanes, through 128
//   or 512 bytes of LDS of the wave's own.  No workgroup barrier precedes the sums: staging d
//   and the scales per workgroup instead kept the first unit waiting until 3.5 us after the
//   start (4.3 us to its end, of 8.6; 32 rows 17408 -> 5120: 35.4 us against 22.6).  Rows of d
//   go to MFMA rows (r, lq) -> 4 lq + r, so that up to four rows of d occupy one accumulator
//   register per column.
// * The waves' sums are added in wave order in LDS; the ranges' sums of a strip by
//   its last workgroup, in range order (one launch; no workgroup waits for another), or,
//   where that workgroup would have more than kJoinRows rows to add, by a second kernel on
//   the whole device.  Results do not depend on timing.
// * Measured (MI355X, device time in graph replays over 1 GB of weights in turn, i.e. from HBM): 1
//   row 17408 -> 5120 (46 MB) 15.6-16.0 us = 2.9 TB/s, 16 rows 5120 -> 17408 20.9-21.2 us with its
//   join, 1 row 1024 -> 1024 5.4 us.  Bound by latency: with no loads at all the first takes 8.7 us
//   (launch, start, six units of arithmetic, joins), without the offset and scale arithmetic 13.9,
//   without the sums over the waves 14.9; a wave loads its next unit only when it has used the last.
// * Measured slower: a ring of units through LDS-direct loads (0.3-1.7 us), workgroups of 256 or
//   1024 threads, 33-64 rows here instead of on the tiles (74 against 46 us, 17408 -> 5120).
#include "arrive.hpp"
#include "device.hpp"
#include "gemm_t_skinny_plan.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "swiglu_grad.hpp"

namespace w4a16 {
namespace {

using namespace skinny_t;

constexpr int kWords = CW / 128;                // words per lane and row
constexpr int kF = CW / 16;                     // operands (columns) per lane and unit

// Units per wave up to which every strip makes the pairs' gradient for itself (GRAD); past that
// the elementwise kernel runs first, as its one pass costs less than the strips' repeated work.
// Device time, within the product against in front of it: 19 rows, 1024 x 2048 pair (1 unit per
// wave) 10.4 / 11.4 us, 1 row, 16384 x 2048 (2 x 8192; 2 units) 11.4 / 12.5, 1 row 32768 x 2048
// (4) 15.3 / 15.7, 32 rows 24576 x 2048 (3) 20.6 / 21.5, 1 row 34816 x 5120 (12) 30.3 / 27.5, 32
// rows 47.1 / 39.4; it also saves 2.7 us of the host's time per call.
constexpr int kGradUnits = 4;
// The same for the gradient of a linear layer's activation and bias (Slope); for rows off eight elements 1.
// What it adds to the product against the kernel in front of it: 19 rows, 1024 x 2048 (1 unit) 2.4 / 4.8 us,
// 1 row 2048 x 16384 (2) 2.4 / 4.7, 32 rows 4.1 / 4.8, 32 rows 5120 x 5120 (2) 4.2 / 4.8, 1 row 2048 x 32768 (4)
// 4.6 / 4.7, 1 row 5120 x 17408 (3) 7.3 / 4.8, 32 rows 14.4 / 4.8; odd rows: 19 rows 1120 x 1001 (1) 3.8 / 4.7,
// 32 rows 5120 x 5119 (2) 7.6 / 4.9.
constexpr int kSlopeUnits = 2;

// The same four columns of two neighbouring n.
__device__ inline uint32_t pair_perm(uint32_t w0, uint32_t w1, bool hi) {
  return __builtin_amdgcn_perm(w1, w0, hi ? 0x07060302u : 0x05040100u);
}

// VEC: rows of d are 16-byte aligned (N a multiple of 8); otherwise eight elements come as the five
// dwords that hold them (as eight 2-byte loads: 1 row 17407 -> 5120 17.4 against 16.5 us, 32 rows
// 5119 -> 17408 40.6 against 34.0; the last element's dword is read and checked by itself).
// GRAD (with VEC): d is the gradient of SiLU(g) u at the pairs gate_up [M, N]: `d` holds that of
// the products h [M, N / 2], every wave makes its operands of d from the two, and the first
// strip's workgroups write them to dgate_up.  One launch less than with the elementwise
// kernel in front; see kGradUnits.
// Slope (not GRAD): d is the gradient of act(z), gate_up holds z [M, N] and dgate_up receives d act'(z), which
// is the operand (both null: without an activation); the first strip also writes the column sums of its
// unrounded values, the bias's gradient: a wave has all rows of its n.
struct SlopeArgs {
  int act;
  float* dbias;            // or null
};
template <int G, int MB, bool VEC, bool GRAD, typename... Slope>
__global__ void __launch_bounds__(kThreads, 2)   // (two waves per SIMD: one workgroup per CU)
gemm_t_skinny_kernel(const uint16_t* __restrict__ d, const uint32_t* __restrict__ packed,
                     const uint16_t* __restrict__ scales, uint16_t* __restrict__ y, int M, int N, int K,
                     SkinnyPlan plan, float* __restrict__ partials, uint32_t* __restrict__ counters,
                     const uint16_t* __restrict__ gate_up, uint16_t* __restrict__ dgate_up, Slope... slope) {
  constexpr bool kSlope = sizeof...(Slope) > 0;
  static_assert(VEC || !GRAD, "pairs are read eight elements at a time");
  constexpr int kGroups = CW / G;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ __attribute__((aligned(16))) uint8_t scale_tile[kWaves * kGroups * kUnit * 2];
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lq = lane >> 4, li = lane & 15;

  const int strip = blockIdx.x % plan.strips, split = blockIdx.x / plan.strips;
  const int c0 = strip * CW;
  const int n_lo = split * plan.range;
  const int n_cnt = min(plan.range, N - n_lo);                 // at least 1
  const int units = (n_cnt + kUnit - 1) / kUnit;

  const uint32_t wrow = (uint32_t)K >> 1;
  const int spr = K / G;
  const __amdgpu_buffer_rsrc_t wres = make_rsrc(packed, (uint32_t)N * wrow);

  // ---- loads of unit u, all straight to registers: its rows n = n_lo + 32 u + 8 lq + j of the
  // weights, the lane's operand of d (row 4 (li % 4) + li / 4 of each block, eight n; zeros past
  // N; rows past M feed nothing) and the unit's scales, kS per lane.  Past the wave's last unit
  // every offset lies outside the buffers (no memory access).
  constexpr int kS = kGroups / 2;               // lane: row lane / 2, groups kS (lane % 2) ..
  // (to a whole dword: the last element may share one with what follows, which is cleared)
  const __amdgpu_buffer_rsrc_t dres = make_rsrc(GRAD ? gate_up : d, ((uint32_t)M * (uint32_t)N * 2u + 3u) & ~3u);
  const __amdgpu_buffer_rsrc_t hres = make_rsrc(d, GRAD ? (uint32_t)M * (uint32_t)N : 0u);
  const __amdgpu_buffer_rsrc_t sres = make_rsrc(scales, (uint32_t)N * (uint32_t)spr * 2u);
  const uint32_t w_v = (uint32_t)(8 * lq) * wrow + (uint32_t)(4 * kWords * li);
  const int x_row = (li & 3) * 4 + (li >> 2);
  const int s_n = lane >> 1, s_g = kS * (lane & 1);
  struct Unit {
    uint32_t w[8][kWords];
    u32x4 x[MB];
    u32x2 dh[GRAD ? MB : 1];
    uint32_t x4[VEC ? 1 : MB];
    u32x4 z[kSlope ? MB : 1];
    uint32_t z4[kSlope && !VEC ? MB : 1];
    uint16_t s[kS];
  };
  const __amdgpu_buffer_rsrc_t zres =
      make_rsrc(gate_up, kSlope && gate_up ? ((uint32_t)M * (uint32_t)N * 2u + 3u) & ~3u : 0u);
  auto load_unit = [&](int u, Unit& t) {
    const bool live = u < units;                                // wave-uniform
    const int n0 = n_lo + kUnit * u;
#pragma unroll
    for (int g = 0; g < kS; ++g) {
      const int n = n0 + s_n, gg = c0 / G + s_g + g;
      t.s[g] = __builtin_amdgcn_raw_buffer_load_b16(
          sres, live && n < N && gg < spr ? ((uint32_t)n * (uint32_t)spr + (uint32_t)gg) * 2u : kOutOfRange, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int r = x_row + 16 * b, n = n0 + 8 * lq;
      const bool ok = live && r < M;
      const uint32_t at = ((uint32_t)r * (uint32_t)N + (uint32_t)n) * 2u;
      if constexpr (GRAD)
        t.dh[b] = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(hres, ok && n < N ? at >> 1 : kOutOfRange, 0, 0));
      if constexpr (VEC) {
        t.x[b] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(dres, ok && n < N ? at : kOutOfRange, 0, 0));
        if constexpr (kSlope)
          t.z[b] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(zres, ok && n < N ? at : kOutOfRange, 0, 0));
      } else {
        // the dwords that hold the eight elements, from one down to a multiple of four bytes, turned in
        // use_unit; elements past N (the next row's) are cleared there
        const uint32_t from = ok && n < N ? at & ~3u : kOutOfRange;
        uint32_t e[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) e[j] = __builtin_amdgcn_raw_buffer_load_b32(dres, from, 4 * j, 0);
        t.x[b] = u32x4{e[0], e[1], e[2], e[3]};
        t.x4[b] = e[4];
        if constexpr (kSlope) {
#pragma unroll
          for (int j = 0; j < 5; ++j) e[j] = __builtin_amdgcn_raw_buffer_load_b32(zres, from, 4 * j, 0);
          t.z[b] = u32x4{e[0], e[1], e[2], e[3]};
          t.z4[b] = e[4];
        }
      }
    }
    const uint32_t off = live ? w_v : kOutOfRange;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t so = live ? (uint32_t)(n0 + j) * wrow + (uint32_t)(c0 >> 1) : 0u;
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(wres, off, so, kStream));
      t.w[j][0] = v[0];
      t.w[j][1] = v[1];
    }
  };

  f32x4 acc[MB][kF];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int f = 0; f < kF; ++f) acc[b][f] = f32x4{};

  const uint32_t m_lo = __builtin_amdgcn_readfirstlane(0x000F000Fu), m_hi = __builtin_amdgcn_readfirstlane(0x00F000F0u);
  uint32_t e_lo = 0x64006400u, e_hi = 0x54005400u;     // fp16 1024 and 64, both halves
  asm volatile("" : "+v"(e_lo), "+v"(e_hi));
  const f16x2 b_lo = {(_Float16)-1032.f, (_Float16)-1032.f}, b_hi = {(_Float16)-72.f, (_Float16)-72.f};

  // the wave's scales of a unit, turned to [group][32 n] (a wave's LDS accesses stay in order)
  uint8_t* ss = scale_tile + wave * (kGroups * kUnit * 2);
  uint8_t* s_w = ss + (s_g * kUnit + s_n) * 2;
  const uint8_t* s_r = ss + ((kF * li) / G) * kUnit * 2 + 16 * lq;

  auto use_unit = [&](const Unit& t, int u) {
    const auto& w = t.w;
#pragma unroll
    for (int g = 0; g < kS; ++g) *reinterpret_cast<uint16_t*>(s_w + g * kUnit * 2) = t.s[g];
    const f16x8 sc = *reinterpret_cast<const f16x8*>(s_r);
    f16x8 xv[MB];
    float sums[8] = {};                          // (Slope) over the lane's rows
    // the eight elements of block b's row, turned and cleared past N where they came as dwords
    auto eight = [&](const u32x4& x, uint32_t x4, int b) {
      u32x4 v = x;
      if constexpr (!VEC) {
        const int n = n_lo + kUnit * u + 8 * lq, left = N - n;
        const uint32_t turn = ((uint32_t)(x_row + 16 * b) * (uint32_t)N & 1u) * 16u;      // n is even
        const uint32_t from[5] = {x.x, x.y, x.z, x.w, x4};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t e = __builtin_amdgcn_alignbit(from[j + 1], from[j], turn);
          v[j] = left >= 2 * j + 2 ? e : (left == 2 * j + 1 ? e & 0xFFFFu : 0u);
        }
      }
      return __builtin_bit_cast(f16x8, v);
    };
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      xv[b] = eight(t.x[b], t.x4[VEC ? 0 : b], b);
      auto times = [&](const SlopeArgs& a) {
        const f16x8 z16 = eight(t.z[kSlope ? b : 0], t.z4[kSlope && !VEC ? b : 0], b);
        float d[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] = (float)xv[b][e];
          z[e] = (float)z16[e];
        }
        times_slope(a.act, z, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xv[b][e] = (_Float16)d[e];
          sums[e] += d[e];
        }
        const int r = x_row + 16 * b, n = n_lo + kUnit * u + 8 * lq;
        if (strip == 0 && dgate_up && r < M && n < N) store_eight<VEC>(dgate_up + (size_t)r * N + n, N - n, xv[b]);
      };
      (times(slope), ...);
      if constexpr (GRAD) {
        const f16x8 z = xv[b];
        using f16x4 = _Float16 __attribute__((ext_vector_type(4)));
        const f16x4 dh = __builtin_bit_cast(f16x4, t.dh[b]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f16x2 r = grad_pair(z[2 * e], z[2 * e + 1], dh[e]);
          xv[b][2 * e] = r[0];
          xv[b][2 * e + 1] = r[1];
        }
        const int r = x_row + 16 * b, n = n_lo + kUnit * u + 8 * lq;
        if (strip == 0 && r < M && n < N) *reinterpret_cast<f16x8*>(dgate_up + (size_t)r * N + n) = xv[b];
      }
    }
    auto add_rows = [&](const SlopeArgs& a) {
      if (strip != 0 || !a.dbias) return;
      // over the sixteen lanes of a row of n (each has other rows of d); lane e < 8 stores element e
      float mine = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = dpp_add<0xB1>(sums[e]);    // quad_perm [1,0,3,2]
        v = dpp_add<0x4E>(v);                // quad_perm [2,3,0,1]
        v = dpp_add<0x124>(v);               // row_ror:4
        v = dpp_add<0x128>(v);               // row_ror:8
        mine = li == e ? v : mine;
      }
      const int n = n_lo + kUnit * u + 8 * lq + li;
      if (li < 8 && n < N) a.dbias[n] = mine;
    };
    (add_rows(slope), ...);
#pragma unroll
    for (int wd = 0; wd < kWords; ++wd)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t p[4], p8[4];
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {
          p[jp] = pair_perm(w[2 * jp][wd], w[2 * jp + 1][wd], hh);
          p8[jp] = p[jp] >> 8;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f16x8 op;
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {
            const uint32_t src = c < 2 ? p[jp] : p8[jp];
            const uint32_t v16 = (c & 1) ? ((src & m_hi) | e_hi) : ((src & m_lo) | e_lo);
            const f16x2 v = (__builtin_bit_cast(f16x2, v16) + ((c & 1) ? b_hi : b_lo)) * f16x2{sc[2 * jp], sc[2 * jp + 1]};
            op[2 * jp] = v[0];
            op[2 * jp + 1] = v[1];
          }
          const int f = 8 * wd + 4 * hh + c;
#pragma unroll
          for (int b = 0; b < MB; ++b)
            acc[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[b], op, acc[b][f], 0, 0, 0);
        }
      }
  };

  // One unit per wave at a time.  (Two, three or four in registers mean as many copies of the
  // unit's 2 KB of code, which every launch fetches anew: 1 row 1024 -> 1024 6.2 / 7.3 / 8.6 us
  // against 5.4 us, 17408 -> 5120 16.1 / 16.9 / 19.0 against 15.8.)
  Unit t;
  load_unit(wave, t);
#pragma unroll 1
  for (int u = wave; u < units; u += kWaves) {
    use_unit(t, u);
    load_unit(u + kWaves, t);
  }

  // ---- sums over the waves, 16 rows of d at a time: buffer [wave][16 rows][256 columns]
  // fp32, columns 16 li + f; 16-byte chunk j of a lane's columns at j ^ (li / 2 % 4) (bank
  // spread).  Accumulator r of lane (lq, li) is row 4 r + lq of its block.
  const __amdgpu_buffer_rsrc_t pres =
      make_rsrc(partials, plan.splits > 1 ? (uint32_t)plan.splits * (uint32_t)(M * K) * 4u : 0u);
  float* red = reinterpret_cast<float*>(smem);
  const int wstride = red_stride(M);
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int row0 = 16 * b;
    if (row0 >= M) break;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (row0 + 4 * r >= M) break;
#pragma unroll
      for (int j = 0; j < kF / 4; ++j) {
        const f32x4 v = {acc[b][4 * j][r], acc[b][4 * j + 1][r], acc[b][4 * j + 2][r],
                         acc[b][4 * j + 3][r]};
        *reinterpret_cast<f32x4*>(red + wave * wstride + (4 * r + lq) * CW + kF * li + 4 * (j ^ ((li >> 1) & 3))) = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int o = tid; o < 16 * CW / 2; o += kThreads) {
      const int q = o / (CW / 2), c = (o % (CW / 2)) * 2;
      if (row0 + q >= M) break;
      const int l = c / kF, f = c % kF;
      const float* src = red + q * CW + kF * l + 4 * ((f >> 2) ^ ((l >> 1) & 3)) + (f & 3);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(src + w * wstride);
        s0 += v.x;
        s1 += v.y;
      }
      const int m = row0 + q, k = c0 + c;
      if (m < M && k < K) {
        if (plan.splits == 1)
          *reinterpret_cast<uint32_t*>(y + (size_t)m * K + k) =
              (uint32_t)float_to_half_bits(s0) | ((uint32_t)float_to_half_bits(s1) << 16);
        else
          __builtin_amdgcn_raw_buffer_store_b64(
              u32x2{__builtin_bit_cast(uint32_t, s0), __builtin_bit_cast(uint32_t, s1)}, pres,
              (uint32_t)(m * K + k) * 4u, (uint32_t)split * (uint32_t)(M * K) * 4u, kDeviceScope);
      }
    }
  }

  // ---- ranges of n: the strip's last workgroup adds the ranges' sums in range order ----
  if (plan.splits == 1 || !plan.fused || !arrive_last(counters + strip, (uint32_t)plan.splits, &arrived)) return;
  const int cols = min(CW, K - c0) / 2;                        // column pairs of the strip
  for (int o = tid; o < M * (CW / 2); o += kThreads) {
    const int m = o / (CW / 2), c = o % (CW / 2);
    if (c >= cols) continue;
    const uint32_t at = (uint32_t)(m * K + c0 + 2 * c) * 4u;
    float s0 = 0.f, s1 = 0.f;
    for (int p0 = 0; p0 < plan.splits; p0 += 8) {              // eight loads in flight
      u32x2 v[8];
#pragma unroll
      for (int p = 0; p < 8; ++p)
        v[p] = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                       pres, at, (uint32_t)min(p0 + p, plan.splits - 1) * (uint32_t)(M * K) * 4u, kDeviceScope));
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p0 + p < plan.splits) {
          const uint32_t lo = v[p][0], hi = v[p][1];
          s0 += __builtin_bit_cast(float, lo);
          s1 += __builtin_bit_cast(float, hi);
        }
    }
    *reinterpret_cast<uint32_t*>(y + (size_t)m * K + c0 + 2 * c) =
        (uint32_t)float_to_half_bits(s0) | ((uint32_t)float_to_half_bits(s1) << 16);
  }
}

// y = the ranges' sums [splits][m k] added in order: two outputs per thread, sixteen loads in flight.
__global__ void __launch_bounds__(64)
gemm_t_skinny_join_kernel(const float* __restrict__ partials, uint16_t* __restrict__ y, int count, int splits) {
  const int i = (blockIdx.x * 64 + threadIdx.x) * 2;           // count is a multiple of 32
  if (i >= count) return;
  float s0 = 0.f, s1 = 0.f;
  for (int p0 = 0; p0 < splits; p0 += 16) {
    float2 v[16];
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      const int q = p0 + p < splits ? p0 + p : p0;
      v[p] = *reinterpret_cast<const float2*>(partials + (size_t)q * count + i);
    }
#pragma unroll
    for (int p = 0; p < 16; ++p)
      if (p0 + p < splits) {
        s0 += v[p].x;
        s1 += v[p].y;
      }
  }
  *reinterpret_cast<uint32_t*>(y + i) = (uint32_t)float_to_half_bits(s0) | ((uint32_t)float_to_half_bits(s1) << 16);
}

template <int G>
auto kernel_of(int m, int n, bool grad) {
  const bool one = blocks_of(m) == 1;
  if (grad) return one ? gemm_t_skinny_kernel<G, 1, true, true> : gemm_t_skinny_kernel<G, 2, true, true>;
  if (n % 8 == 0) return one ? gemm_t_skinny_kernel<G, 1, true, false> : gemm_t_skinny_kernel<G, 2, true, false>;
  return one ? gemm_t_skinny_kernel<G, 1, false, false> : gemm_t_skinny_kernel<G, 2, false, false>;
}
template <int G>
auto kernel_of(int m, int n, bool, const SlopeArgs&) {
  const bool one = blocks_of(m) == 1;
  if (n % 8 == 0)
    return one ? gemm_t_skinny_kernel<G, 1, true, false, SlopeArgs> : gemm_t_skinny_kernel<G, 2, true, false, SlopeArgs>;
  return one ? gemm_t_skinny_kernel<G, 1, false, false, SlopeArgs> : gemm_t_skinny_kernel<G, 2, false, false, SlopeArgs>;
}

// With gate_up: d is the gradient of h, and the pairs' gradient is written to dgate_up; with slope: see SlopeArgs.
template <typename... Slope>
hipError_t launch_any(const uint16_t* d, const uint16_t* gate_up, uint16_t* dgate_up, const uint32_t* packed,
                      const uint16_t* scales, uint16_t* y, int m, int n, int k, int group, void* workspace,
                      const DeviceInfo& dev, hipStream_t stream, const Slope&... slope) {
  const SkinnyPlan p = skinny_plan(m, n, k, dev);
  float* partials = p.splits > 1 ? reinterpret_cast<float*>(behind_counters(workspace)) : nullptr;
  uint32_t* counters = static_cast<uint32_t*>(workspace);
  auto kern = group == 128 ? kernel_of<128>(m, n, gate_up, slope...) : kernel_of<32>(m, n, gate_up, slope...);
  const hipError_t e = launch_kernel(kern, dim3((unsigned)(p.strips * p.splits)), dim3(kThreads), p.lds, stream, d,
                                     packed, scales, y, m, n, k, p, partials, counters, gate_up, dgate_up, slope...);
  if (e != hipSuccess || p.splits == 1 || p.fused) return e;
  const int count = m * k;
  return launch_kernel(gemm_t_skinny_join_kernel, dim3((unsigned)((count / 2 + 63) / 64)), dim3(64), 0, stream,
                       partials, y, count, p.splits);
}

}  // namespace

size_t gemm_t_skinny_workspace_bytes(int m, int n, int k, int group, const DeviceInfo& dev) {
  const size_t sums = sums_bytes(skinny_plan(m, n, k, dev), m, k);
  return sums ? kCounterBytes + sums : 0;
}

bool gemm_t_skinny_fits(int m, int n, int k, int group, const DeviceInfo& dev) {
  return m <= kSkinnyTRows && plan_fits(skinny_plan(m, n, k, dev), m, k, dev);
}

hipError_t launch_gemm_t_skinny(const uint16_t* d, const uint32_t* packed, const uint16_t* scales, uint16_t* y, int m,
                                int n, int k, int group, void* workspace, const DeviceInfo& dev, hipStream_t stream) {
  return launch_any(d, nullptr, nullptr, packed, scales, y, m, n, k, group, workspace, dev, stream);
}

bool swiglu_backward_skinny_fits(int m, int n, int k, int group, const DeviceInfo& dev) {
  return n % 8 == 0 && gemm_t_skinny_fits(m, n, k, group, dev) &&
         skinny_plan(m, n, k, dev).range <= kGradUnits * kWaves * kUnit;
}

hipError_t launch_swiglu_backward_skinny(const uint16_t* dh, const uint16_t* gate_up, uint16_t* dgate_up,
                                         const uint32_t* packed, const uint16_t* scales, uint16_t* dx, int m, int n,
                                         int k, int group, void* workspace, const DeviceInfo& dev, hipStream_t stream) {
  return launch_any(dh, gate_up, dgate_up, packed, scales, dx, m, n, k, group, workspace, dev, stream);
}

bool linear_backward_skinny_fits(int m, int n, int k, int group, const DeviceInfo& dev) {
  return gemm_t_skinny_fits(m, n, k, group, dev) &&
         skinny_plan(m, n, k, dev).range <= (n % 8 == 0 ? kSlopeUnits : 1) * kWaves * kUnit;
}

hipError_t launch_linear_backward_skinny(const uint16_t* dy, const uint16_t* pre, uint16_t* dpre, float* dbias,
                                         const uint32_t* packed, const uint16_t* scales, uint16_t* dx, int m, int n,
                                         int k, int group, int act, void* workspace, const DeviceInfo& dev,
                                         hipStream_t stream) {
  return launch_any(dy, pre, dpre, packed, scales, dx, m, n, k, group, workspace, dev, stream, SlopeArgs{act, dbias});
}

}  // namespace w4a16
