// moe_ffn.hip -- the routed experts' feed-forward for a few tokens, in two or three kernels on gfx950.
//
//     y[t] = residual[t] + sum_s w[t, s] * W2[e] h(t, s),   e = ids[t, s],
//     h(t, s) = SiLU(g) u,   (g, u) = W1[e] x[t]
//
// With up to 512 (token, slot) pairs nearly every expert that is used is used once or twice, so
// the layer is a stream of the used experts' weights: 1.77 MB each at 2048 x 512, g32.
//
// * Few pairs (kDirectPairs): two kernels, each pair by itself.  Gate/up: a workgroup per (pair, 32 weight
//   rows).  Down and combine: a workgroup per 8 output columns, a wave per pair; the pairs' results meet
//   in LDS and the router's weights add them in slot order with the residual.
// * More pairs: three kernels.  In both products the workgroups walk over (block of up to four pairs of one
//   expert, band of weight rows), so an expert's weights are read once for every four of its pairs; each workgroup
//   of the first sorts the pairs into blocks itself (group_pairs), the second reads the lists.  A third kernel adds a
//   token's results with the router's weights.
// No atomics on results and no order that depends on timing: a token's output has the same bits in any batch
// of the same kind.
//
// All products run on v_mfma_f32_4x4x4_16b_f16: block b of 16 is four weight rows (B columns) at 32 k of their
// own (one 16-byte load per lane: 4 rows x 256 contiguous bytes), times four activation rows (A).  A
// lane's 32 k lie in one scale group, so the codes enter as the integers u - 8 (exact in fp16) and
// the scale is applied to the fp32 result: weights are exact.  The MFMA wants neighbouring lanes on
// different weight rows; loaded so, every four lanes touch four cache lines.  So weights and scales are loaded
// with sixteen lanes side by side on a row and the lanes are permuted afterwards (spread_rows).
//
// The grouped products take one workgroup's loads at a time and hide them behind three others on the CU
// (64 VGPRs, four workgroups of 512 threads); with the next piece in registers instead and fewer of them 64
// tokens took 62 + 37 us instead of 56 + 38 (as they were then).  Weight loads bypass the caches' retention (kStream):
// the first product 66 instead of 104 us, both as they were then.
//
// Measured (MI355X, operands from memory, medians; 2048 x 512, group 32, 256 experts, 8 slots a token): 1 token 5.4 + 4.9 us
// (launch and one trip to memory each), 8 tokens 15.4 + 10.6, 16 tokens 25.3 + 17.8 + 4.8, 32 tokens 37.7 + 24.0 + 4.8, 64
// tokens 51.2 + 32.0 + 4.8 us (31.2 to 36.5 by which experts are used): 391 MB of their weights at 4.4-4.7 TB/s over both
// products, against 4.9 of a large copy.  What is left is the fixed part (launch, sorting the pairs, the last work items)
// and the third kernel.
//
// h goes between the kernels as two fp16 parts, h 2^-8 = hi + lo 2^-11: off by at most 2^-23 |h|, or by 2^-28 where that
// is more (|h| below 2^-5: lo is subnormal there), for |h| up to 2^24.  Rounded once to fp16 it would add as much error
// again as the rounding of y; 2^-28 is an eighth of what fp16 is off by in its smallest numbers.
#include <type_traits>

#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "mfma_operands.hpp"
#include "tile_gemm.hpp"

namespace w4a16 {
namespace {

constexpr int kStepK = 512;                      // k of one step: 16 chunks of 32
constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kBlock = 4;                        // pairs of a block: the A rows
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
static_assert(kThreads >= kMoeFfnPairs && kThreads >= 8 * kMoeFfnTokens, "one pair, and one output, per thread");

constexpr float kHScale = 0x1p-8f, kLoScale = 0x1p11f;

// The pairs in blocks of up to four of one expert each.
struct Blocks {
  int expert[kMoeFfnPairs];                      // of block b
  uint16_t size[kMoeFfnPairs];                   // its pairs: 1 .. 4,
  uint16_t pair[kMoeFfnPairs * kBlock];          // pair[4 b + i]
  int total, unused[3];
};
static_assert(sizeof(Blocks) % 16 == 0 && sizeof(Blocks) / 16 <= kThreads, "copied in one go, 16 bytes per thread");
// What sorting them needs: an expert's place (open addressing) has
struct Places {
  unsigned long long count[2 * kMoeFfnPairs];    // its pairs in each wave, a byte each
  uint32_t key[2 * kMoeFfnPairs];                // the expert (kFree: none); then its first block among those of the wave
                                                 // that has its first pair (low half), and that wave
  uint32_t wave_blocks[kWaves];                  // blocks whose expert's first pair is in this wave
};
constexpr uint32_t kFree = 0xFFFFFFFFu;
constexpr int kPlaceBits = 10;
static_assert(2 * kMoeFfnPairs == 1 << kPlaceBits, "places");

// Sum over a wave's lanes up to and with this one (DPP: shifts within rows, then whole rows).
__device__ inline uint32_t wave_scan(uint32_t v) {
  auto add = [&](auto ctrl, auto rows) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});      // row_shr:1, 2, 4, 8
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});      // row_bcast:15 to rows 1 and 3
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});      // row_bcast:31 to rows 2 and 3
  return v;
}

// Sorts the pairs; returns the number of blocks.  Blocks and their pairs are in the pairs' order, the same in
// every workgroup (which share the blocks out), whatever order the atomics take.  Pairs whose id is no expert are in
// no block.  All waves do this at once, so its instructions count (the first form, a loop over the lanes for a pair's
// rank and counters in 64-bit atomics, cost 600 a wave, as much as a third of the weights' arithmetic).
__device__ inline int group_pairs(Blocks& s, Places& q, const int32_t* __restrict__ ids, int pairs, int experts) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = tid < pairs ? ids[tid] : -1;
  const bool known = e >= 0 && e < experts;
#pragma unroll
  for (int i = 0; i < 2 * kMoeFfnPairs; i += kThreads) {
    q.key[tid + i] = kFree;
    q.count[tid + i] = 0;
  }
  __syncthreads();
  uint32_t at = 0;
  if (known) {
    // (512 pairs at most in 1024 places: a free one is found)
    const uint32_t want = (uint32_t)e;
    at = (want * 0x9E3779B1u) >> (32 - kPlaceBits);
    for (uint32_t k = atomicCAS(&q.key[at], kFree, want); k != kFree && k != want; k = atomicCAS(&q.key[at], kFree, want))
      at = (at + 1) & (2 * kMoeFfnPairs - 1);
  }
  unsigned long long same = __ballot(known);                // the wave's pairs of this expert
#pragma unroll
  for (int b = 0; b < kPlaceBits; ++b) {
    const int bit = (int)(at << (31 - b)) >> 31;            // 0 or -1
    same &= ~(__ballot(bit != 0) ^ (unsigned long long)(long long)bit);
  }
  uint32_t rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
  if (known && rank == 0) reinterpret_cast<uint8_t*>(&q.count[at])[wave] = (uint8_t)__popcll(same);
  __syncthreads();
  const unsigned long long counts = known ? q.count[at] : 0ull, ahead = counts & ((1ull << (8 * wave)) - 1);
  auto bytes = [](unsigned long long v) {
    return __builtin_amdgcn_sad_u8((uint32_t)(v >> 32), 0, __builtin_amdgcn_sad_u8((uint32_t)v, 0, 0));
  };
  const uint32_t count = bytes(counts);
  rank += bytes(ahead);
  const uint32_t mine = known && rank == 0 ? (count + kBlock - 1) / kBlock : 0u;      // blocks of the expert
  const uint32_t upto = wave_scan(mine);
  if (lane == 63) q.wave_blocks[wave] = upto;
  if (mine) q.key[at] = (upto - mine) | (uint32_t)wave << 16;
  __syncthreads();
  const uint32_t place = known ? q.key[at] : 0u;
  uint32_t before = place & 0xFFFFu, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint32_t n = q.wave_blocks[w];
    before += (uint32_t)w < place >> 16 ? n : 0u;
    total += n;
  }
  if (known) {
    const uint32_t b = before + rank / kBlock;
    s.pair[kBlock * b + rank % kBlock] = (uint16_t)tid;
    if (rank % kBlock == 0) {
      s.expert[b] = e;
      s.size[b] = (uint16_t)min((uint32_t)kBlock, count - rank);
    }
  }
  if (tid == 0) s.total = (int)total;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane((int)total);
}

// The eight codes of a packed word as fp16 integers u - 8, in the order of permute_a: a nibble
// under the exponent of 1024 (mantissa bits 0-3) or of 64 (bits 4-7), less 1032 or 72.  Masks (scalar) and
// exponents (vector) are held in registers, so each pair is one v_and_or_b32 and one packed addition.
struct Decoder {
  uint32_t m_lo, m_hi, e_lo, e_hi;
  __device__ inline Decoder() {
    m_lo = __builtin_amdgcn_readfirstlane(0x000F000Fu);
    m_hi = __builtin_amdgcn_readfirstlane(0x00F000F0u);
    e_lo = 0x64006400u;
    e_hi = 0x54005400u;
    asm volatile("" : "+v"(e_lo), "+v"(e_hi));
  }
  __device__ inline void operator()(uint32_t q, f16x4& a, f16x4& b) const {
    const uint32_t q8 = q >> 8;
    const f16x2 c1 = {(_Float16)-1032.f, (_Float16)-1032.f}, c2 = {(_Float16)-72.f, (_Float16)-72.f};
    const f16x2 p0 = __builtin_bit_cast(f16x2, (q & m_lo) | e_lo) + c1;      // (0, 4)
    const f16x2 p1 = __builtin_bit_cast(f16x2, (q8 & m_lo) | e_lo) + c1;     // (2, 6)
    const f16x2 p2 = __builtin_bit_cast(f16x2, (q & m_hi) | e_hi) + c2;      // (1, 5)
    const f16x2 p3 = __builtin_bit_cast(f16x2, (q8 & m_hi) | e_hi) + c2;     // (3, 7)
    a = f16x4{p0[0], p0[1], p1[0], p1[1]};
    b = f16x4{p2[0], p2[1], p3[0], p3[1]};
  }
};

// Four activation rows times a lane's four weight rows over a word's eight k: a[q] is set q of the rows' activations in
// permute_a's order (two sets: the codes are decoded once).
template <int SETS>
__device__ inline void word_product(const Decoder& decode, uint32_t word, const u32x4 (&a)[SETS], f32x4 (&t)[SETS]) {
  f16x4 b0, b1;
  decode(word, b0, b1);
#pragma unroll
  for (int q = 0; q < SETS; ++q) {
    t[q] = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, u32x2{a[q].x, a[q].y}), b0, t[q], 0, 0, 0);
    t[q] = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, u32x2{a[q].z, a[q].w}), b1, t[q], 0, 0, 0);
  }
}
// ... over the lane's chunk of 32 k.
__device__ inline f32x4 chunk_product(const Decoder& decode, const u32x4& wv, const u32x4 (&a)[4]) {
  f32x4 t[1] = {f32x4{}};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const u32x4 aw[1] = {a[w]};
    word_product(decode, wv[w], aw, t);
  }
  return t[0];
}

// From the lane that loaded it (row l / 16, chunk l % 16) to the one that multiplies it (row l % 4, chunk l / 4).
__device__ inline uint32_t spread_rows(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute(((lane & 3) << 6) + (lane & ~3), (int)v);
}
__device__ inline u32x4 spread_rows(const u32x4& v, int lane) {
  return u32x4{spread_rows(v.x, lane), spread_rows(v.y, lane), spread_rows(v.z, lane), spread_rows(v.w, lane)};
}

// Four values' sums over the sixteen chunks (lanes 4 c + column): a lane gets that of value
// sum_index(lane).  Two lane swaps halve the lanes of a value while two values share a register, then
// two DPP steps finish (8 before 4: the sums then have a period of 8 lanes, so every lane adds the
// same two).  All four are added in the same order, so a pair's result has the same bits whichever
// A row serves it.  The swaps are inline assembly because both registers are outputs (the compiler's
// builtins lose one of them); the s_nop give the wait states around them.
__device__ inline int sum_index(int lane) { return ((lane >> 3) & 2) | (lane >> 5); }
__device__ inline float chunk_sums(f32x4 v) {
  float a = v[0], b = v[1], c = v[2], d = v[3];
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\tv_permlane32_swap_b32 %2, %3\n\ts_nop 1"
               : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
  float s = a + b, t = c + d;                    // lanes 0-31: values 0 and 2, 32-63: 1 and 3
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\ts_nop 1" : "+v"(s), "+v"(t));
  s += t;                                        // rows of sixteen lanes: values 0, 2, 1, 3
  s = dpp_add<0x128>(s);                         // row_ror:8
  return dpp_add<0x124>(s);                      // row_ror:4
}

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A load's offset, or one outside every buffer.  (The empty asm keeps the choice a value: as a branch
// around the load, every other load would be waited for where the branch joins.)
__device__ inline uint32_t offset_if(bool in, uint32_t off) {
  uint32_t v = in ? off : kOutOfRange;
  asm("" : "+v"(v));
  return v;
}

// A value as the two parts of h.
__device__ inline void split_h(float v, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)v;
  hi = __builtin_bit_cast(uint16_t, h);
  // (past fp16's range the upper part says it alone)
  lo = __builtin_fabsf((float)h) <= 65504.0f ? float_to_half_bits((v - (float)h) * kLoScale) : (uint16_t)0;
}
__device__ inline float silu_product(float gate, float up) {
  return gate * __builtin_amdgcn_rcpf(1.0f + __expf(-gate)) * up;
}
// The lane's neighbour in the weight rows: the up row of an even lane's gate row.
__device__ inline float next_row(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, false));
}
// Place of element k of an h row in its step, in the order of the A loads: word, chunk, row of `rows`, permute_a's order.
__device__ inline uint32_t h_place(uint32_t k, uint32_t rows, uint32_t row) {
  const uint32_t c = k % kStepK / 32, w = k % 32 / 8, j = k % 8;
  return ((w * 16 + c) * rows + row) * 8 + (((j & 1) << 2) | (j & 2) | (j >> 2));
}
__host__ __device__ inline int h_steps(int inter) { return (inter + kStepK - 1) / kStepK; }

// ---- few pairs: each by itself ----
// Up to this many: two launches and no sorting.  Direct against grouped: 32 pairs of experts that are nearly all
// different 9.4 + 6.7 against 10.9 + 6.9 + 4.8 us, 64 pairs 15.3 + 10.3 against 17.2 + 10.9 + 4.9; of twelve experts 32 pairs 9.1
// + 6.7 against 7.7 + 5.2 + 4.9, 64 pairs 14.0 + 9.7 against 9.3 + 5.7 + 4.9: there the grouped form is faster by a sixth,
// at different experts slower by a quarter, and the host, which chooses, does not see the ids.  Also what
// moe_down_direct_kernel holds: an id per lane, a result per pair in LDS.
constexpr int kDirectPairs = 64;
constexpr int kBandRows = 4 * kWaves;            // gate/up rows of a workgroup: four per wave
constexpr int kXSteps = 4;                       // steps of a staged piece of x
constexpr int kXK = kXSteps * kStepK;            // 2048 k
constexpr uint32_t kDirectStep = 2 * kStepK * 2; // bytes of a pair's h per step: upper and lower parts

// h: [pair][step] blocks of kDirectStep bytes (h_place, two rows).
template <int G>
__global__ void __launch_bounds__(kThreads)
moe_gate_up_direct_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids,
                          const uint32_t* __restrict__ packed, const uint16_t* __restrict__ scales,
                          uint16_t* __restrict__ h, int topk, int experts, int rows, int K) {
  __shared__ __attribute__((aligned(16))) uint8_t xs[2][2 * kXK];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int c = lane >> 2, p = blockIdx.y, r0 = blockIdx.x * kBandRows;
  const int e = ids[p];
  if (e < 0 || e >= experts) return;
  const uint32_t row_w = (uint32_t)K >> 1, spr = (uint32_t)K / G;
  const size_t first = (size_t)e * rows + r0;
  const uint32_t lrow = (uint32_t)(wave * 4 + (lane >> 4)), lchunk = (uint32_t)(lane & 15);
  const uint32_t w_off = lrow * row_w + 16u * lchunk, s_off = (lrow * spr + 32u * lchunk / G) * 2u;
  const uint16_t* xp = x + (size_t)(p / topk) * K;
  const Decoder decode;
  float acc = 0.0f;
  for (int k0 = 0, buf = 0; k0 < K; k0 += kXK, buf ^= 1) {
    // the first four waves stage the piece's 4 KB, 16 bytes a thread
    const __amdgpu_buffer_rsrc_t xres = make_rsrc(xp + k0, (uint32_t)(K - k0) * 2u);
    u32x4 xv = u32x4{};
    if (wave < 4) xv = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xres, 16u * threadIdx.x, 0, 0));
    const __amdgpu_buffer_rsrc_t wres = make_rsrc(reinterpret_cast<const uint8_t*>(packed) + first * row_w + k0 / 2,
                                                  (uint32_t)(rows - r0) * row_w - (uint32_t)k0 / 2);
    const __amdgpu_buffer_rsrc_t sres =
        make_rsrc(scales + first * spr + k0 / G, ((uint32_t)(rows - r0) * spr - (uint32_t)k0 / G) * 2u);
    u32x4 wv[kXSteps];
    uint32_t sc[kXSteps];
#pragma unroll
    for (int s = 0; s < kXSteps; ++s) {
      const bool in = (uint32_t)(k0 + s * kStepK) + 32u * lchunk < (uint32_t)K;     // (else: the next row's)
      wv[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                            wres, offset_if(in, w_off) + (uint32_t)(kStepK / 2) * s, 0, kStream));
      sc[s] = __builtin_amdgcn_raw_buffer_load_b16(sres, offset_if(in, s_off) + (uint32_t)(kStepK / G * 2) * s, 0, 0);
    }
    if (wave < 4) *reinterpret_cast<u32x4*>(xs[buf] + 16 * threadIdx.x) = permute_a(xv);
    lds_barrier();
#pragma unroll
    for (int s = 0; s < kXSteps; ++s) {
      if (k0 + s * kStepK >= K) break;
      u32x4 a[4];
#pragma unroll
      for (int w = 0; w < 4; ++w)
        a[w] = *reinterpret_cast<const u32x4*>(xs[buf] + s * (2 * kStepK) + 64 * c + 16 * w);
      const f32x4 t = chunk_product(decode, spread_rows(wv[s], lane), a);
      acc = __builtin_fmaf(half_bits_to_float(spread_rows(sc[s], lane)), t[0], acc);
    }
  }
  const float gate = chunk_sums(f32x4{acc, 0.f, 0.f, 0.f}), up = next_row(gate);
  const uint32_t o = (uint32_t)(r0 + wave * 4 + lane) >> 1;      // (lanes 0 and 2)
  if (lane < 4 && !(lane & 1) && o < (uint32_t)rows >> 1) {
    uint16_t hi, lo;
    split_h(silu_product(gate, up) * kHScale, hi, lo);
    uint16_t* dst = h + ((size_t)p * h_steps(rows >> 1) + o / kStepK) * (kDirectStep / 2);
    dst[h_place(o, 2, 0)] = hi;
    dst[h_place(o, 2, 1)] = lo;
  }
}

// (sixteen waves, a step of one pair at a time each: 2 tokens 5.1, 8 tokens 10.3 us; eight waves with three steps in
// flight 6.4 and 12.3, with two 5.6 and 10.8; sixteen with three, more code than they save, 8.3 and 14.2)
constexpr int kDirectWaves = 16;

template <int G>
__global__ void __launch_bounds__(64 * kDirectWaves)
moe_down_direct_kernel(const uint16_t* __restrict__ h, const int32_t* __restrict__ ids, const float* __restrict__ weights,
                       const uint32_t* __restrict__ packed, const uint16_t* __restrict__ scales, const uint16_t* residual,
                       uint16_t* y, int pairs, int topk, int tokens, int experts, int N, int K) {
  __shared__ float part[kDirectPairs][8];        // a pair's result in the workgroup's columns, times its weight
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int li = lane & 3, c = lane >> 2, n0 = blockIdx.x * 8;
  const int id = lane < pairs ? ids[lane] : -1;                  // every wave: all pairs
  // this thread's output, at the end: token tid / 8, column tid % 8
  const int ot = tid >> 3, on = n0 + (tid & 7);
  const bool out = ot < tokens && on < N;
  const float res = out && residual ? half_bits_to_float(residual[(size_t)ot * N + on]) : 0.0f;
  const float weight = lane < pairs ? weights[lane] : 0.0f;

  const uint32_t row_w = (uint32_t)K >> 1, spr = (uint32_t)K / G;
  const int steps = h_steps(K);
  const uint32_t lrow = (uint32_t)lane >> 4, lchunk = (uint32_t)(lane & 15);
  const uint32_t w_off = lrow * row_w + 16u * lchunk, s_off = (lrow * spr + 32u * lchunk / G) * 2u;
  const Decoder decode;
  for (int p = wave; p < pairs; p += kDirectWaves) {
    const int e = __builtin_amdgcn_readlane(id, p);
    const bool live = e >= 0 && e < experts;
    const size_t first = (size_t)(live ? e : 0) * N + n0;
    f32x4 acc = f32x4{};                         // upper and lower parts' sums, columns 0-3 and 4-7
    for (int k0 = 0; k0 < K; k0 += kStepK) {
      const __amdgpu_buffer_rsrc_t wres = make_rsrc(reinterpret_cast<const uint8_t*>(packed) + first * row_w + k0 / 2,
                                                    live ? (uint32_t)(N - n0) * row_w - (uint32_t)k0 / 2 : 0u);
      const __amdgpu_buffer_rsrc_t sres = make_rsrc(scales + first * spr + k0 / G,
                                                    live ? ((uint32_t)(N - n0) * spr - (uint32_t)k0 / G) * 2u : 0u);
      const bool in = (uint32_t)k0 + 32u * lchunk < (uint32_t)K;
      const uint32_t wo = offset_if(in, w_off), so = offset_if(in, s_off);
      u32x4 wv[2], a[4];
      uint32_t sc[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        wv[g] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wres, wo + 4u * g * row_w, 0, kStream));
        sc[g] = __builtin_amdgcn_raw_buffer_load_b16(sres, so + 8u * g * spr, 0, 0);
      }
      // A rows: upper and lower parts, twice; chunks past K were never written
      const __amdgpu_buffer_rsrc_t hres =
          make_rsrc(reinterpret_cast<const uint8_t*>(h) + ((size_t)p * steps + k0 / kStepK) * kDirectStep, live ? kDirectStep : 0u);
      const uint32_t a_off = offset_if(k0 + 32 * c < K, 32u * c + 16u * (li & 1));
#pragma unroll
      for (int w = 0; w < 4; ++w)
        a[w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(hres, a_off + 512u * w, 0, 0));
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const f32x4 t = chunk_product(decode, spread_rows(wv[g], lane), a);
        const float f = half_bits_to_float(spread_rows(sc[g], lane));
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[2 * g + i] = __builtin_fmaf(f, t[i], acc[2 * g + i]);
      }
    }
    const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), p));
    const float r = chunk_sums(f32x4{__builtin_fmaf(acc[1], 1.0f / kLoScale, acc[0]),
                                     __builtin_fmaf(acc[3], 1.0f / kLoScale, acc[2]), 0.f, 0.f}) * (1.0f / kHScale);
    const int at = sum_index(lane);
    if (at < 2 && (lane & 12) == 0) part[p][4 * at + li] = live ? w * r : 0.0f;
  }
  __syncthreads();
  if (!out) return;
  float v = 0.0f;
  for (int s = 0; s < topk; ++s) v += part[ot * topk + s][tid & 7];
  y[(size_t)ot * N + on] = float_to_half_bits(v + res);
}

// ---- more pairs: an expert's blocks ----
constexpr size_t kBlocksBytes = (sizeof(Blocks) + 255) & ~(size_t)255;
constexpr int kXPitch = kXK * 2 + 16;            // bytes per staged row of x: rows shift by 4 banks
constexpr int kXBuf = kBlock * kXPitch;
constexpr uint32_t kHStep = 2 * kBlock * kStepK * 2;   // bytes of a block's h per step: upper parts, then lower parts

// h: [block][step][part] (h_place, four rows).  A workgroup's work items are blockIdx.x, + gridDim.x, ...: item = block * bands
// + band (32 weight rows); a piece of one, 2048 k, is what is loaded and computed at a time.
template <int G>
__global__ void __launch_bounds__(kThreads, 8)
moe_gate_up_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint32_t* __restrict__ packed,
                   const uint16_t* __restrict__ scales, uint16_t* __restrict__ h, Blocks* __restrict__ blocks, int pairs,
                   int topk, int experts, int rows, int K, int bands) {
  __shared__ __attribute__((aligned(16))) uint8_t xs[kXBuf];
  __shared__ __attribute__((aligned(16))) Blocks bl;
  __shared__ Places places;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int li = lane & 3, c = lane >> 2;        // weight row (and A row), chunk
  const int total = group_pairs(bl, places, ids, pairs, experts);
  // for the down product (the last workgroup: the others have as many work items or one more)
  if (blockIdx.x + 1 == gridDim.x && threadIdx.x < sizeof(Blocks) / 16)
    reinterpret_cast<u32x4*>(blocks)[threadIdx.x] = reinterpret_cast<const u32x4*>(&bl)[threadIdx.x];

  const uint32_t row_w = (uint32_t)K >> 1, spr = (uint32_t)K / G;
  const int pieces = (K + kXK - 1) / kXK;
  const int inter = rows >> 1;
  const float per_token = 1.0f / (float)topk;

  struct Work {
    int block, band, piece;
  };
  struct Data {
    u32x4 x[2], w[kXSteps];
    uint32_t sc[kXSteps];
  };
  const int dblock = (int)gridDim.x / bands, dband = (int)gridDim.x % bands;
  auto advance = [&](Work& k) {
    if (++k.piece < pieces) return;
    k.piece = 0;
    k.block += dblock;
    k.band += dband;
    if (k.band >= bands) {
      k.band -= bands;
      ++k.block;
    }
  };
  // A lane's place in a work item's rows, and how far its chunks are from the row's end.
  const uint32_t lrow = (uint32_t)(wave * 4 + (lane >> 4)), lchunk = (uint32_t)(lane & 15);
  const uint32_t w_off = lrow * row_w + 16u * lchunk, s_off = (lrow * spr + 32u * lchunk / G) * 2u;
  // Every load is made, in a fixed order (so each wait is for its own).  What is there is in the buffers'
  // descriptors, in scalar registers: they begin at the piece and end with the expert's last row, or
  // with the row of x, or are empty.
  auto load = [&](const Work& k, Data& d) __attribute__((always_inline)) {
    const int b = k.block, e = uniform(bl.expert[b]), n = uniform(bl.size[b]);
    // waves 2 r and 2 r + 1 stage the halves of row r
    const int row = wave >> 1, k0 = k.piece * kXK;
    const int pair = row < n ? uniform(bl.pair[kBlock * b + row]) : 0;
    const int token = uniform((int)(((float)pair + 0.5f) * per_token));
    const __amdgpu_buffer_rsrc_t xres = make_rsrc(x + (size_t)token * K + k0, row < n ? (uint32_t)(K - k0) * 2u : 0u);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      d.x[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             xres, (uint32_t)(wave & 1) * (4u * kStepK) + 16u * (uint32_t)lane +
                                                       2u * kStepK * s, 0, 0));
    __builtin_amdgcn_sched_barrier(0);           // (these first: they are waited for without the weights)
    const int r0 = k.band * kBandRows;
    const size_t first = (size_t)e * rows + r0;
    const __amdgpu_buffer_rsrc_t wres = make_rsrc(reinterpret_cast<const uint8_t*>(packed) + first * row_w + k0 / 2,
                                                  (uint32_t)(rows - r0) * row_w - (uint32_t)k0 / 2);
    const __amdgpu_buffer_rsrc_t sres =
        make_rsrc(scales + first * spr + k0 / G, ((uint32_t)(rows - r0) * spr - (uint32_t)k0 / G) * 2u);
#pragma unroll
    for (int s = 0; s < kXSteps; ++s) {
      const bool in = (uint32_t)(k0 + s * kStepK) + 32u * lchunk < (uint32_t)K;     // (else: the next row's)
      d.w[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             wres, offset_if(in, w_off) + (uint32_t)(kStepK / 2) * s, 0, kStream));
      d.sc[s] = __builtin_amdgcn_raw_buffer_load_b16(sres, offset_if(in, s_off) + (uint32_t)(kStepK / G * 2) * s, 0, 0);
    }
  };
  const Decoder decode;
  f32x4 acc = f32x4{};
  auto stage = [&](const Data& d, uint8_t* buf) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      *reinterpret_cast<u32x4*>(buf + (wave >> 1) * kXPitch + ((wave & 1) * 2 + s) * (2 * kStepK) + 16 * lane) =
          permute_a(d.x[s]);
  };
  auto compute = [&](const Work& k, const Data& d, const uint8_t* buf) {
    const uint8_t* xa = buf + li * kXPitch + 64 * c;
#pragma unroll
    for (int s = 0; s < kXSteps; ++s) {
      if (k.piece * kXK + s * kStepK >= K) break;
      u32x4 a[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) a[w] = *reinterpret_cast<const u32x4*>(xa + s * (2 * kStepK) + 16 * w);
      const f32x4 t = chunk_product(decode, spread_rows(d.w[s], lane), a);
      const float f = half_bits_to_float(spread_rows(d.sc[s], lane));
#pragma unroll
      for (int i = 0; i < kBlock; ++i) acc[i] = __builtin_fmaf(f, t[i], acc[i]);
    }
    if (k.piece + 1 < pieces) return;
    // the first four lanes of each row of sixteen have one pair's sums; the even ones (gate rows) store
    const int n = uniform(bl.size[k.block]), i = sum_index(lane);
    const float gate = chunk_sums(acc), up = next_row(gate);
    acc = f32x4{};
    const uint32_t o = (uint32_t)(k.band * kBandRows + wave * 4 + li) >> 1;
    if (i < n && (lane & 13) == 0 && o < (uint32_t)inter) {
      uint16_t hi, lo;
      split_h(silu_product(gate, up) * kHScale, hi, lo);
      uint16_t* dst = h + ((size_t)k.block * h_steps(inter) + o / kStepK) * (kHStep / 2) + h_place(o, kBlock, i);
      dst[0] = hi;
      dst[kHStep / 4] = lo;
    }
  };
  Work cur = {(int)blockIdx.x / bands, (int)blockIdx.x % bands, 0};
  Data d;
  while (cur.block < total) {
    load(cur, d);
    lds_barrier();                               // (the rows staged before are read)
    stage(d, xs);
    lds_barrier();
    compute(cur, d, xs);
    advance(cur);
  }
}

// Down: a work item is (block, band of 64 columns), eight columns per wave; a piece of one is 512 k.  part
// [pair][N] fp32 receives the pairs' results.
constexpr int kDownGroups = 2;                   // groups of four columns per wave (4: 64 tokens 41.2 against 38.2 us)
constexpr int kDownCols = 4 * kDownGroups * kWaves;

template <int G>
__global__ void __launch_bounds__(kThreads, 8)
moe_down_kernel(const uint16_t* __restrict__ h, const Blocks* __restrict__ blocks, const uint32_t* __restrict__ packed,
                const uint16_t* __restrict__ scales, float* __restrict__ part, int N, int K, int bands) {
  __shared__ __attribute__((aligned(16))) uint8_t hs[kHStep];
  __shared__ __attribute__((aligned(16))) Blocks bl;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int c = lane >> 2;
  if (threadIdx.x < sizeof(Blocks) / 16)
    reinterpret_cast<u32x4*>(&bl)[threadIdx.x] = reinterpret_cast<const u32x4*>(blocks)[threadIdx.x];
  __syncthreads();
  const int total = uniform(bl.total);

  const uint32_t row_w = (uint32_t)K >> 1, spr = (uint32_t)K / G;
  const int steps = h_steps(K);
  const uint32_t lrow = (uint32_t)(4 * kDownGroups * wave + (lane >> 4)), lchunk = (uint32_t)(lane & 15);
  const uint32_t w_off = lrow * row_w + 16u * lchunk, s_off = (lrow * spr + 32u * lchunk / G) * 2u;
  struct Work {
    int block, band, s;
  };
  struct Data {
    u32x4 h, w[kDownGroups];
    uint32_t sc[kDownGroups];
  };
  const int dblock = (int)gridDim.x / bands, dband = (int)gridDim.x % bands;
  auto advance = [&](Work& k) {
    if (++k.s < steps) return;
    k.s = 0;
    k.block += dblock;
    k.band += dband;
    if (k.band >= bands) {
      k.band -= bands;
      ++k.block;
    }
  };
  auto load = [&](const Work& k, Data& d) __attribute__((always_inline)) {
    const int b = k.block, k0 = k.s * kStepK, n0 = k.band * kDownCols;
    // wave w stages the w-th KB: word w % 4 of the upper (w < 4) or lower parts; chunks past K were never written
    const __amdgpu_buffer_rsrc_t hres =
        make_rsrc(reinterpret_cast<const uint8_t*>(h) + (size_t)(b * steps + k.s) * kHStep, kHStep);
    d.h = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                        hres, offset_if(k0 + 32 * c < K, 1024u * wave + 16u * lane), 0, 0));
    __builtin_amdgcn_sched_barrier(0);
    const size_t first = (size_t)uniform(bl.expert[b]) * N + n0;
    const __amdgpu_buffer_rsrc_t wres = make_rsrc(reinterpret_cast<const uint8_t*>(packed) + first * row_w + k0 / 2,
                                                  (uint32_t)(N - n0) * row_w - (uint32_t)k0 / 2);
    const __amdgpu_buffer_rsrc_t sres =
        make_rsrc(scales + first * spr + k0 / G, ((uint32_t)(N - n0) * spr - (uint32_t)k0 / G) * 2u);
    const bool in = (uint32_t)k0 + 32u * lchunk < (uint32_t)K;
    const uint32_t wo = offset_if(in, w_off), so = offset_if(in, s_off);
#pragma unroll
    for (int g = 0; g < kDownGroups; ++g) {
      d.w[g] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wres, wo + 4u * g * row_w, 0, kStream));
      d.sc[g] = __builtin_amdgcn_raw_buffer_load_b16(sres, so + 8u * g * spr, 0, 0);
    }
  };
  const Decoder decode;
  f32x4 acc[kDownGroups];
#pragma unroll
  for (int g = 0; g < kDownGroups; ++g) acc[g] = f32x4{};
  auto compute = [&](const Work& k, const Data& d, const uint8_t* buf) {
    f32x4 t[kDownGroups][2];
    u32x4 wv[kDownGroups];
#pragma unroll
    for (int g = 0; g < kDownGroups; ++g) {
      t[g][0] = t[g][1] = f32x4{};
      wv[g] = spread_rows(d.w[g], lane);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      u32x4 a[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) a[q] = *reinterpret_cast<const u32x4*>(buf + (4 * q + w) * 1024 + 16 * lane);
#pragma unroll
      for (int g = 0; g < kDownGroups; ++g) word_product(decode, wv[g][w], a, t[g]);
    }
#pragma unroll
    for (int g = 0; g < kDownGroups; ++g) {
      const float f = half_bits_to_float(spread_rows(d.sc[g], lane));
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        acc[g][i] = __builtin_fmaf(f, __builtin_fmaf(t[g][1][i], 1.0f / kLoScale, t[g][0][i]), acc[g][i]);
    }
    if (k.s + 1 < steps) return;
    // a row of sixteen lanes has one pair's sums, column li of each group in all its lanes: lane 4 g + li stores group g's
    float r = 0.0f;
#pragma unroll
    for (int g = 0; g < kDownGroups; ++g) {
      const float v = chunk_sums(acc[g]);
      if ((c & 3) == g) r = v;
      acc[g] = f32x4{};
    }
    const int i = sum_index(lane), n = k.band * kDownCols + 4 * kDownGroups * wave + (lane & 15);
    if (i < bl.size[k.block] && (lane & 15) < 4 * kDownGroups && n < N)
      part[(size_t)bl.pair[kBlock * k.block + i] * N + n] = r * (1.0f / kHScale);
  };
  Work cur = {(int)blockIdx.x / bands, (int)blockIdx.x % bands, 0};
  Data d;
  while (cur.block < total) {
    load(cur, d);
    lds_barrier();                               // (the rows staged before are read)
    *reinterpret_cast<u32x4*>(hs + 1024 * wave + 16 * lane) = d.h;
    lds_barrier();
    compute(cur, d, hs);
    advance(cur);
  }
}

// y = residual + sum over a token's slots of weight * part, four columns per thread.
__global__ void __launch_bounds__(256)
moe_ffn_combine_kernel(const float* __restrict__ part, const int32_t* __restrict__ ids, const float* __restrict__ weights,
                       const uint16_t* residual, uint16_t* y, int topk, int experts, int N) {
  const int n = 4 * (blockIdx.x * 256 + threadIdx.x), t = blockIdx.y;
  if (n >= N) return;
  const size_t at = (size_t)t * N + n;
  f16x4 res = f16x4{};
  if (residual) res = *reinterpret_cast<const f16x4*>(residual + at);
  f32x4 v = f32x4{};
  for (int s0 = 0; s0 < topk; s0 += 8) {         // eight slots' loads in flight
    f32x4 q[8];
    float w[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int p = t * topk + s0 + s;
      const bool in = s0 + s < topk && ids[p] >= 0 && ids[p] < experts;
      w[s] = in ? weights[p] : 0.0f;
      q[s] = in ? *reinterpret_cast<const f32x4*>(part + (size_t)p * N + n) : f32x4{};
    }
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(w[s], q[s][i], v[i]);
  }
  f16x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (_Float16)(v[i] + (float)res[i]);
  *reinterpret_cast<f16x4*>(y + at) = o;
}

}  // namespace

size_t moe_ffn_workspace_bytes(int pairs, int hidden, int inter) {
  if (pairs <= kDirectPairs) return kCounterBytes + (size_t)pairs * h_steps(inter) * kDirectStep;
  // (as many blocks as pairs at most)
  return kCounterBytes + kBlocksBytes + (size_t)pairs * h_steps(inter) * kHStep + (size_t)pairs * hidden * sizeof(float);
}

hipError_t launch_moe_ffn(const uint16_t* x, const int32_t* ids, const float* weights, const uint32_t* gate_up,
                          const uint16_t* gate_up_scales, const uint32_t* down, const uint16_t* down_scales,
                          const uint16_t* residual, uint16_t* y, int tokens, int topk, int experts, int hidden,
                          int inter, int group, void* workspace, const DeviceInfo& dev, hipStream_t stream) {
  const int pairs = tokens * topk;
  uint16_t* h = reinterpret_cast<uint16_t*>(behind_counters(workspace));
  const int up_bands = (2 * inter + kBandRows - 1) / kBandRows;
  const bool g32 = group == 32;
  if (pairs <= kDirectPairs) {
    const hipError_t e = launch_kernel(g32 ? moe_gate_up_direct_kernel<32> : moe_gate_up_direct_kernel<128>,
                                       dim3((unsigned)up_bands, (unsigned)pairs), dim3(kThreads), 0, stream, x, ids, gate_up,
                                       gate_up_scales, h, topk, experts, 2 * inter, hidden);
    if (e != hipSuccess) return e;
    return launch_kernel(g32 ? moe_down_direct_kernel<32> : moe_down_direct_kernel<128>, dim3((unsigned)((hidden + 7) / 8)),
                         dim3(64 * kDirectWaves), 0, stream, h, ids, weights, down, down_scales, residual, y, pairs, topk,
                         tokens, experts, hidden, inter);
  }
  Blocks* blocks = reinterpret_cast<Blocks*>(behind_counters(workspace));
  h += kBlocksBytes / sizeof(uint16_t);
  float* part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(h) + (size_t)pairs * h_steps(inter) * kHStep);
  const int down_bands = (hidden + kDownCols - 1) / kDownCols;
  // four workgroups per CU, fewer where there are fewer work items
  auto grid = [&](int bands) {
    const int64_t items = (int64_t)pairs * bands;
    return dim3((unsigned)(items < 4 * dev.num_cu ? items : 4 * dev.num_cu));
  };
  hipError_t e = launch_kernel(g32 ? moe_gate_up_kernel<32> : moe_gate_up_kernel<128>, grid(up_bands), dim3(kThreads), 0, stream,
                               x, ids, gate_up, gate_up_scales, h, blocks, pairs, topk, experts, 2 * inter, hidden, up_bands);
  if (e != hipSuccess) return e;
  e = launch_kernel(g32 ? moe_down_kernel<32> : moe_down_kernel<128>, grid(down_bands), dim3(kThreads), 0, stream, h,
                    blocks, down, down_scales, part, hidden, inter, down_bands);
  if (e != hipSuccess) return e;
  return launch_kernel(moe_ffn_combine_kernel, dim3((unsigned)((hidden + 1023) / 1024), (unsigned)tokens), dim3(256), 0, stream,
                       part, ids, weights, residual, y, topk, experts, hidden);
}

}  // namespace w4a16
