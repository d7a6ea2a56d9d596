// moe_ffn.hip -- the routed experts' feed-forward for a few tokens, in two kernels on gfx950.
//
//     y[t] = residual[t] + sum_s w[t, s] * W2[e] h(t, s),   e = ids[t, s],
//     h(t, s) = SiLU(g) u,   (g, u) = W1[e] x[t]
//
// With up to 512 (token, slot) pairs nearly every expert that is used is used once or twice, so
// the layer is a stream of the used experts' weights: 1.77 MB each at 2048 x 512, g32.
//
// * gate/up: one workgroup per (pair, 32 weight rows).  Every wave reads all pairs' experts itself;
//   the first pair of an expert does the expert's work for all its pairs, the others leave at once.
//   So no routing kernel runs first, and an expert's weights are read once.  A wave owns 8 rows.
// * down and combine: one workgroup per 8 output columns, for all experts: a wave takes every eighth
//   used expert, the pairs' results meet in LDS, and the router's weights add them in slot order
//   with the residual, one rounding at the end: no partial results in memory, no atomics.
//
// Both run on v_mfma_f32_4x4x4_16b_f16: block b of 16 is four weight rows (B columns) at 32 k of their
// own (one 16-byte load per lane: 4 rows x 256 contiguous bytes), times four activation rows (A).  A
// lane's 32 k lie in one scale group, so the codes enter as the integers u - 8 (exact in fp16) and
// the scale is applied to the fp32 result: weights are exact.
//
// h goes between the kernels as two fp16 parts, h 2^-8 = hi + lo 2^-11 (22 bits, |h| up to 2^24):
// rounded once to fp16 it would add as much error again as the rounding of y.  The parts are two
// of the four A rows, so they cost no extra instruction while an expert has one or two pairs.
#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "mfma_operands.hpp"

namespace w4a16 {
namespace {

constexpr int kStepK = 512;                      // k of one step: 16 chunks of 32
constexpr int kRowsWave = 8;                     // weight rows of a wave (two groups of four)
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// What the first kernel leaves about a pair: the next pair of the same expert, and whether it is the first.
constexpr uint32_t kNoPair = 0xFFFFu, kFirst = 0x10000u;
constexpr float kHScale = 0x1p-8f, kLoScale = 0x1p11f;

// The eight codes of a packed word as fp16 integers u - 8, in the order of permute_a: a nibble
// under the exponent of 1024 (mantissa bits 0-3) or of 64 (bits 4-7), less 1032 or 72.
__device__ inline void decode_codes(uint32_t q, f16x4& a, f16x4& b) {
  const uint32_t q8 = q >> 8;
  const f16x2 c1 = {(_Float16)-1032.f, (_Float16)-1032.f}, c2 = {(_Float16)-72.f, (_Float16)-72.f};
  const f16x2 p0 = __builtin_bit_cast(f16x2, (q & 0x000F000Fu) | 0x64006400u) + c1;    // (0, 4)
  const f16x2 p1 = __builtin_bit_cast(f16x2, (q8 & 0x000F000Fu) | 0x64006400u) + c1;   // (2, 6)
  const f16x2 p2 = __builtin_bit_cast(f16x2, (q & 0x00F000F0u) | 0x54005400u) + c2;    // (1, 5)
  const f16x2 p3 = __builtin_bit_cast(f16x2, (q8 & 0x00F000F0u) | 0x54005400u) + c2;   // (3, 7)
  a = f16x4{p0[0], p0[1], p1[0], p1[1]};
  b = f16x4{p2[0], p2[1], p3[0], p3[1]};
}

// Four activation rows times a lane's four weight rows over its chunk of 32 k: a[w] is the lane's
// activations of word w, in permute_a's order.
__device__ inline f32x4 chunk_product(const u32x4& wv, const u32x4 (&a)[4]) {
  f32x4 t = f32x4{};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f16x4 b0, b1;
    decode_codes(wv[w], b0, b1);
    t = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, u32x2{a[w].x, a[w].y}), b0, t, 0, 0, 0);
    t = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, u32x2{a[w].z, a[w].w}), b1, t, 0, 0, 0);
  }
  return t;
}

// Sum over a lane's sixteen chunks (lanes 4 c + column); every lane gets it, the same bits (8 before
// 4: the sums then have a period of 8 lanes, so every lane adds the same two), whichever lane
// serves a token.
__device__ inline float chunk_sum(float v) {
  v = dpp_add<0x128>(v);   // row_ror:8
  v = dpp_add<0x124>(v);   // row_ror:4
  v += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));   // lane ^ 16
  v += __shfl_xor(v, 32, 64);
  return v;
}

// ---- gate/up ----
constexpr int kUpThreads = 256, kUpWaves = kUpThreads / 64;
constexpr int kUpRows = kUpWaves * kRowsWave;    // weight rows of a workgroup
constexpr int kUpSteps = 4;                      // steps of a staged piece of x
constexpr int kUpK = kUpSteps * kStepK;          // 2048 k
constexpr int kUpTokens = 4;                     // pairs per pass: the A rows
constexpr int kXPitch = kUpK * 2 + 16;           // bytes per staged row: rows shift by 4 banks

// NC: 64-pair blocks (pairs <= 64 NC).  h: [pair][2][inter] fp16.
template <int G, int NC>
__global__ void __launch_bounds__(kUpThreads)
moe_gate_up_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint32_t* __restrict__ packed,
                   const uint16_t* __restrict__ scales, uint16_t* __restrict__ h, uint32_t* __restrict__ link,
                   int pairs, int topk, int experts, int rows, int K) {
  __shared__ __attribute__((aligned(16))) uint8_t xs[kUpTokens * kXPitch];
  __shared__ uint16_t lists[kUpWaves][64 * NC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 3, c = lane >> 2;        // weight row (and A row), chunk
  const int band = blockIdx.x, p = blockIdx.y;

  // ---- this pair's expert, and the pairs that share it ----
  int id[NC];
#pragma unroll
  for (int b = 0; b < NC; ++b) id[b] = 64 * b + lane < pairs ? ids[64 * b + lane] : -1;
  int e = -1;
#pragma unroll
  for (int b = 0; b < NC; ++b)
    if (b == p >> 6) e = __builtin_amdgcn_readlane(id[b], p & 63);
  const bool known = e >= 0 && e < experts;
  int count = 0;
  uint32_t next = kNoPair;
  bool first = known;
  uint16_t* list = lists[wave];                  // (each wave's own: no barrier)
#pragma unroll
  for (int b = 0; b < NC; ++b) {
    const uint64_t m = __builtin_amdgcn_ballot_w64(id[b] == e && known);
    const uint64_t at_p = b == p >> 6 ? 1ull << (p & 63) : 0ull;
    const uint64_t below = b < p >> 6 ? ~0ull : (b == p >> 6 ? at_p - 1 : 0ull);
    if (m & below) first = false;
    const uint64_t above = m & ~below & ~at_p;
    if (above && next == kNoPair) next = 64 * b + (uint32_t)__builtin_ctzll(above);
    if (known && id[b] == e) list[count + __builtin_popcountll(m & ((1ull << lane) - 1))] = (uint16_t)(64 * b + lane);
    count += __builtin_popcountll(m);
  }
  __builtin_amdgcn_wave_barrier();
  if (band == 0 && threadIdx.x == 0) link[p] = next | (first ? kFirst : 0u);
  if (!first) return;

  const uint32_t row_w = (uint32_t)K >> 1, spr = (uint32_t)K / G;
  const __amdgpu_buffer_rsrc_t wres =
      make_rsrc(reinterpret_cast<const uint8_t*>(packed) + (size_t)e * rows * row_w, (uint32_t)rows * row_w);
  const __amdgpu_buffer_rsrc_t sres = make_rsrc(scales + (size_t)e * rows * spr, (uint32_t)rows * spr * 2u);
  const int r0 = band * kUpRows + wave * kRowsWave;
  const int pieces = (K + kUpK - 1) / kUpK;
  const int inter = rows >> 1;

  u32x4 raw[kUpSteps][2];
  uint32_t sc[kUpSteps][2];
  // (a row past the expert's last, or a chunk past K, reads zero codes and a zero scale)
  auto load_weights = [&](int piece) {
#pragma unroll
    for (int s = 0; s < kUpSteps; ++s)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t k = (uint32_t)(piece * kUpK + s * kStepK + 32 * c), r = (uint32_t)(r0 + 4 * g + li);
        const bool in = k < (uint32_t)K;
        raw[s][g] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  wres, in ? r * row_w + (k >> 1) : kOutOfRange, 0, kStream));
        sc[s][g] = __builtin_amdgcn_raw_buffer_load_b16(sres, in ? (r * spr + k / G) * 2u : kOutOfRange, 0, 0);
      }
  };
  for (int i0 = 0; i0 < count; i0 += kUpTokens) {
    const int here = min(kUpTokens, count - i0);
    f32x4 acc[2] = {f32x4{}, f32x4{}};
    for (int piece = 0; piece < pieces; ++piece) {
      // wave w stages row w of the pass
      u32x4 xv[kUpSteps];
      if (wave < here) {
        const int token = __builtin_amdgcn_readfirstlane(list[i0 + wave]) / topk;
        const uint16_t* src = x + (size_t)token * K;
#pragma unroll
        for (int s = 0; s < kUpSteps; ++s) {
          const int k = piece * kUpK + s * kStepK + 8 * lane;
          xv[s] = k < K ? *reinterpret_cast<const u32x4*>(src + k) : u32x4{};
        }
      }
      if (pieces > 1 || i0 == 0) load_weights(piece);
      if (piece > 0 || i0 > 0) __syncthreads();  // the rows staged before are read
      if (wave < here) {
#pragma unroll
        for (int s = 0; s < kUpSteps; ++s)
          *reinterpret_cast<u32x4*>(xs + wave * kXPitch + s * (2 * kStepK) + 16 * lane) = permute_a(xv[s]);
      }
      __syncthreads();
      const uint8_t* xa = xs + min(li, here - 1) * kXPitch + 64 * c;
#pragma unroll
      for (int s = 0; s < kUpSteps; ++s) {
        if (piece * kUpK + s * kStepK >= K) break;
        u32x4 a[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) a[w] = *reinterpret_cast<const u32x4*>(xa + s * (2 * kStepK) + 16 * w);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f32x4 t = chunk_product(raw[s][g], a);
          const float f = half_bits_to_float(sc[s][g]);
#pragma unroll
          for (int i = 0; i < kUpTokens; ++i) acc[g][i] = __builtin_fmaf(f, t[i], acc[g][i]);
        }
      }
    }
    // the lane of chunk 4 g + i and an even row stores output (row / 2) of pair i
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < kUpTokens; ++i) {
        const float v = chunk_sum(acc[g][i]);
        const float o = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf,
                                                                              0xf, false));
        if (c == 4 * g + i) {
          gate = v;
          up = o;
        }
      }
    const int r = r0 + 4 * (c >> 2) + li, i = c & 3, o = r >> 1;
    if (c < 8 && !(li & 1) && i < here && o < inter) {
      const float v = gate / (1.0f + __expf(-gate)) * up * kHScale;
      const _Float16 hi = (_Float16)v;
      // (past fp16's range the upper part says it alone)
      const _Float16 lo = __builtin_fabsf((float)hi) <= 65504.0f ? (_Float16)((v - (float)hi) * kLoScale) : (_Float16)0.f;
      const int at = (o & ~7) + ((o & 1) << 2) + (o & 2) + ((o >> 2) & 1);   // permute_a's order
      uint16_t* dst = h + (size_t)list[i0 + i] * 2 * inter + at;
      dst[0] = __builtin_bit_cast(uint16_t, hi);
      dst[inter] = __builtin_bit_cast(uint16_t, lo);
    }
  }
}

// ---- down and combine ----
constexpr int kDownThreads = 512, kDownWaves = kDownThreads / 64;
static_assert(kDownThreads >= kMoeFfnPairs && kDownThreads >= 8 * kMoeFfnTokens, "one pair, and one output, per thread");

template <int G>
__global__ void __launch_bounds__(kDownThreads)
moe_down_kernel(const uint16_t* __restrict__ h, const uint32_t* __restrict__ link, const int32_t* __restrict__ ids,
                const float* __restrict__ weights, const uint32_t* __restrict__ packed,
                const uint16_t* __restrict__ scales, const uint16_t* residual, uint16_t* y, int pairs, int topk,
                int tokens, int experts, int N, int K) {
  __shared__ float part[kMoeFfnPairs][8];        // a pair's result in the workgroup's columns
  __shared__ int ids_l[kMoeFfnPairs];
  __shared__ float weights_l[kMoeFfnPairs];
  __shared__ uint32_t link_l[kMoeFfnPairs];
  __shared__ uint16_t list[kMoeFfnPairs];        // the first pair of each used expert
  __shared__ int counts[kDownWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 3, c = lane >> 2;
  const int n0 = blockIdx.x * 8;

  const uint32_t my_link = tid < pairs ? link[tid] : 0u;
  if (tid < pairs) {
    link_l[tid] = my_link;
    ids_l[tid] = ids[tid];
    weights_l[tid] = weights[tid];
  }
  // this thread's output, at the end: token tid / 8, column tid % 8
  const int ot = tid >> 3, on = n0 + (tid & 7);
  const bool out = ot < tokens && on < N;
  const float res = out && residual ? half_bits_to_float(residual[(size_t)ot * N + on]) : 0.0f;
  const bool first = (my_link & kFirst) != 0;
  const uint64_t firsts = __builtin_amdgcn_ballot_w64(first);
  if (lane == 0) counts[wave] = __builtin_popcountll(firsts);
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kDownWaves; ++w) {
    before += w < wave ? counts[w] : 0;
    total += counts[w];
  }
  total = __builtin_amdgcn_readfirstlane(total);
  if (first) list[before + __builtin_popcountll(firsts & ((1ull << lane) - 1))] = (uint16_t)tid;
  __syncthreads();

  const uint32_t row_w = (uint32_t)K >> 1, spr = (uint32_t)K / G;
  const int steps = (K + kStepK - 1) / kStepK;
  const __amdgpu_buffer_rsrc_t hres = make_rsrc(h, (uint32_t)pairs * 2u * (uint32_t)K * 2u);
  // one step: 512 k of the 8 columns for up to two pairs (p0; p1 or none) of one expert
  struct Step {
    int it, p0, p1, e, s;
  };
  struct Data {
    u32x4 w[2], a[4];
    uint32_t sc[2];
  };
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  auto pair_of = [&](Step& st, int p0) {
    st.p0 = p0;
    st.p1 = uniform((int)(link_l[p0] & kNoPair));
    st.s = 0;
  };
  auto item_of = [&](Step& st, int it) {
    st.it = it;
    if (it >= total) return;
    pair_of(st, uniform(list[it]));
    st.e = uniform(ids_l[st.p0]);
  };
  auto advance = [&](Step& st) {
    if (++st.s < steps) return;
    const int p2 = st.p1 == (int)kNoPair ? (int)kNoPair : uniform((int)(link_l[st.p1] & kNoPair));
    if (p2 != (int)kNoPair) pair_of(st, p2);
    else item_of(st, st.it + kDownWaves);
  };
  auto load = [&](const Step& st, Data& d) {
    const __amdgpu_buffer_rsrc_t wres =
        make_rsrc(reinterpret_cast<const uint8_t*>(packed) + (size_t)st.e * N * row_w, (uint32_t)N * row_w);
    const __amdgpu_buffer_rsrc_t sres = make_rsrc(scales + (size_t)st.e * N * spr, (uint32_t)N * spr * 2u);
    const uint32_t k = (uint32_t)(st.s * kStepK + 32 * c);
    const bool in = k < (uint32_t)K;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t r = (uint32_t)(n0 + 4 * g + li);
      d.w[g] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             wres, in ? r * row_w + (k >> 1) : kOutOfRange, 0, kStream));
      d.sc[g] = __builtin_amdgcn_raw_buffer_load_b16(sres, in ? (r * spr + k / G) * 2u : kOutOfRange, 0, 0);
    }
    // A rows: the upper parts of p0 and p1, then their lower parts (no p1: p0's again, not stored)
    const uint32_t pair = (uint32_t)((li & 1) && st.p1 != (int)kNoPair ? st.p1 : st.p0);
    const uint32_t at = ((pair * 2u + (uint32_t)(li >> 1)) * (uint32_t)K + k) * 2u;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      d.a[w] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(hres, in ? at + 16u * w : kOutOfRange, 0, 0));
  };
  f32x4 acc[2] = {f32x4{}, f32x4{}};
  auto compute = [&](const Step& st, const Data& d) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const f32x4 t = chunk_product(d.w[g], d.a);
      const float f = half_bits_to_float(d.sc[g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[g][i] = __builtin_fmaf(f, t[i], acc[g][i]);
    }
    if (st.s + 1 < steps) return;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = chunk_sum(__builtin_fmaf(acc[g][2 + i], 1.0f / kLoScale, acc[g][i])) * (1.0f / kHScale);
        if (c == 2 * g + i && (i == 0 || st.p1 != (int)kNoPair)) part[i ? st.p1 : st.p0][4 * g + li] = v;
      }
    acc[0] = acc[1] = f32x4{};
  };
  // the next step's loads go out before this one's arithmetic
  Step cur;
  item_of(cur, wave);
  Data d;
  if (cur.it < total) load(cur, d);
  while (cur.it < total) {
    Step nxt = cur;
    advance(nxt);
    Data dn = d;
    if (nxt.it < total) load(nxt, dn);
    compute(cur, d);
    cur = nxt;
    d = dn;
  }
  __syncthreads();
  if (!out) return;
  float v = 0.0f;
  for (int s = 0; s < topk; ++s) {
    const int p = ot * topk + s;
    const int e = ids_l[p];
    if (e >= 0 && e < experts) v = __builtin_fmaf(weights_l[p], part[p][tid & 7], v);
  }
  y[(size_t)ot * N + on] = float_to_half_bits(v + res);
}

}  // namespace

size_t moe_ffn_workspace_bytes(int pairs, int inter) {
  const size_t links = ((size_t)pairs * sizeof(uint32_t) + 255) & ~(size_t)255;
  return kCounterBytes + links + (size_t)pairs * 2 * inter * sizeof(uint16_t);
}

hipError_t launch_moe_ffn(const uint16_t* x, const int32_t* ids, const float* weights, const uint32_t* gate_up,
                          const uint16_t* gate_up_scales, const uint32_t* down, const uint16_t* down_scales,
                          const uint16_t* residual, uint16_t* y, int tokens, int topk, int experts, int hidden,
                          int inter, int group, void* workspace, hipStream_t stream) {
  const int pairs = tokens * topk;
  uint32_t* link = reinterpret_cast<uint32_t*>(behind_counters(workspace));
  uint16_t* h = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(link) +
                                            (((size_t)pairs * sizeof(uint32_t) + 255) & ~(size_t)255));
  auto up = group == 32 ? (pairs <= 64 ? moe_gate_up_kernel<32, 1> : moe_gate_up_kernel<32, kMoeFfnPairs / 64>)
                        : (pairs <= 64 ? moe_gate_up_kernel<128, 1> : moe_gate_up_kernel<128, kMoeFfnPairs / 64>);
  const hipError_t err =
      launch_kernel(up, dim3((unsigned)((2 * inter + kUpRows - 1) / kUpRows), (unsigned)pairs), dim3(kUpThreads), 0,
                    stream, x, ids, gate_up, gate_up_scales, h, link, pairs, topk, experts, 2 * inter, hidden);
  if (err != hipSuccess) return err;
  return launch_kernel(group == 32 ? moe_down_kernel<32> : moe_down_kernel<128>, dim3((unsigned)((hidden + 7) / 8)),
                       dim3(kDownThreads), 0, stream, h, link, ids, weights, down, down_scales, residual, y, pairs, topk,
                       tokens, experts, hidden, inter);
}

}  // namespace w4a16
