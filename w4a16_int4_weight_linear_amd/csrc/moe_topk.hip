// moe_topk.hip -- the router's choice and its gradient on gfx950.
//
// Choice: of a token's E logits the topk largest, in falling order, equal ones by rising expert
// number; an expert whose logit is -inf is masked out and never chosen (its slot gets id -1 and
// weight 0, which moe_route and moe_ffn pass over).  Weights are the softmax
//     w_s = exp(l_s - max) / sum exp(l_j - max),   j over all experts, or over the chosen ones,
// in fp32 with the row's maximum taken off.  The choice compares the logits themselves (as
// integers whose order is the floats'), so it is exact whatever the rounding of the softmax.
//
// A token's row is held in registers by LANES lanes, V logits each; a round takes the row's
// largest key (DPP steps), then the lowest expert that has it, and strikes it out: three scans of the lane's V keys and two
// reductions.  Many tokens are bound by these instructions: 16384 tokens of 256 experts, 8 slots, fp32 9.6 us with operands from
// memory, of which 891 vector instructions a wave, four waves a SIMD, are 5.9 (fp32 8.1, fp16 7.7 us from the caches; all
// experts' softmax 9.3, 9.4); few tokens by a launch and one trip to memory (4.9 us).
//
// Gradient: with mean = sum_s w_s dw_s, dl[id_s] = w_s (dw_s - mean) where the weights were
// normalised over the chosen, else dl[e] = (dw_e if chosen - mean) p_e with p the softmax over all.
#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "moe_topk_plan.hpp"

namespace w4a16 {
namespace {

using topk_plan::kThreads;
constexpr uint32_t kMaskedKey = 0x007FFFFFu;     // the key of -inf; 0 is no logit at all

// Floats as integers in the same order: -0 as +0, every NaN above +inf.
__device__ inline uint32_t key_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return x != x ? 0xFFFFFFFFu : k;
}
__device__ inline float value_of(uint32_t key) {
  return __builtin_bit_cast(float, key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// Reductions over the LANES lanes of a token (16: a DPP row, or the whole wave); every lane gets the same result, of sums
// too: after the turn by 8 values have a period of 8 lanes, so the turn by 4 adds the same two everywhere.
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int LANES, typename F>
__device__ inline uint32_t row_reduce(uint32_t v, F f) {
  v = f(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
  v = f(v, dpp<0x128>(v));   // row_ror:8
  v = f(v, dpp<0x124>(v));   // row_ror:4
  if constexpr (LANES == 64) {
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    v = f(f(a, b), f(c, d));
  }
  return v;
}
template <int LANES>
__device__ inline uint32_t row_max(uint32_t v) {
  return row_reduce<LANES>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LANES>
__device__ inline uint32_t row_min(uint32_t v) {
  return row_reduce<LANES>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int LANES>
__device__ inline float row_sum(float v) {
  return __builtin_bit_cast(float, row_reduce<LANES>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }));
}

// The token of a thread (the grid may have several rows of workgroups).
template <int LANES>
__device__ inline int64_t token_of() {
  return ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
}

// What any lane of the wave wrote to LDS before is there for every lane after (no instruction: LDS serves a wave in order).
__device__ inline void lanes_meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The expert of a lane's value v: runs of four, so that a lane reads 16 (or 8) bytes at a time.
template <int LANES>
__device__ inline int expert_of(int lane, int v) { return 4 * lane + 4 * LANES * (v >> 2) + (v & 3); }

__device__ inline float to_float(float x) { return x; }
__device__ inline float to_float(_Float16 x) { return (float)x; }

// An expert to read in place of one that does not exist (the empty asm keeps the choice a value, not a
// branch around each load).
__device__ inline int readable(int e, int experts) {
  int r = e < experts ? e : 0;
  asm("" : "+v"(r));
  return r;
}

// A lane's logits of row x, all loads in flight together (e >= experts: expert 0's, to be passed over).  VEC:
// rows start on four elements.
template <int LANES, int V, bool VEC, typename T>
__device__ inline void load_row(const T* x, int lane, int experts, float (&val)[V]) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    t4 q[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j)
      q[j] = *reinterpret_cast<const t4*>(x + readable(expert_of<LANES>(lane, 4 * j), experts));
#pragma unroll
    for (int v = 0; v < V; ++v) val[v] = to_float(q[v / 4][v % 4]);
  } else {
    T q[V];
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = x[readable(expert_of<LANES>(lane, v), experts)];
#pragma unroll
    for (int v = 0; v < V; ++v) val[v] = to_float(q[v]);
  }
}

template <int LANES, int V, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads)
moe_topk_kernel(const T* __restrict__ logits, int32_t* __restrict__ ids, float* __restrict__ weights, int tokens,
                int experts, int topk, int renormalize) {
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t t = token_of<LANES>();
  const bool live = t < tokens;                    // (all lanes run: the reductions cross them)
  float val[V];
  load_row<LANES, V, VEC>(logits + (live ? t : 0) * experts, lane, experts, val);
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = expert_of<LANES>(lane, v) < experts ? key_of(val[v]) : 0u;

  auto largest = [&]() {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
    return row_max<LANES>(m);
  };
  uint32_t won = largest();
  const float peak = value_of(won);
  float total = 0.0f;
  if (!renormalize) {
#pragma unroll
    for (int v = 0; v < V; ++v) total += key[v] > kMaskedKey ? expf(val[v] - peak) : 0.0f;
    total = row_sum<LANES>(total);
  }
  int my_id = -1;                                  // slot `lane`'s choice
  uint32_t my_key = 0;
  for (int s = 0; s < topk; ++s) {
    uint32_t first = 0xFFFFFFFFu;                  // the lowest expert with that key
#pragma unroll
    for (int v = V - 1; v >= 0; --v) first = key[v] == won ? (uint32_t)expert_of<LANES>(lane, v) : first;
    first = row_min<LANES>(first);
    const bool mine = lane == s && won > kMaskedKey;
    my_id = mine ? (int)first : my_id;
    my_key = mine ? won : my_key;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = first == (uint32_t)expert_of<LANES>(lane, v) ? 0u : key[v];
    won = largest();
  }
  const float p = my_id >= 0 ? expf(value_of(my_key) - peak) : 0.0f;
  if (renormalize) total = row_sum<LANES>(p);
  if (live && lane < topk) {
    ids[t * topk + lane] = my_id;
    weights[t * topk + lane] = my_id >= 0 ? p / total : 0.0f;
  }
}

template <int LANES, int V, bool VEC, typename T>
__global__ void __launch_bounds__(kThreads)
moe_topk_backward_kernel(const float* __restrict__ dweights, const T* __restrict__ logits,
                         const int32_t* __restrict__ ids, const float* __restrict__ weights, T* __restrict__ dlogits,
                         int tokens, int experts, int topk, int renormalize) {
  // a token's gradient is put together in LDS, by one wave: its own LDS accesses keep their order, and the fences keep
  // the compiler from moving a lane's own past what the other lanes do
  __shared__ float rows[kThreads / LANES][LANES * V];
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t t = token_of<LANES>();
  const bool live = t < tokens;
  float* row = rows[threadIdx.x / LANES];
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (live && lane < topk) {
    id = ids[t * topk + lane];
    if (id >= 0 && id < experts) {
      w = weights[t * topk + lane];
      dw = dweights[t * topk + lane];
    } else {
      id = -1;
    }
  }
  const float mean = row_sum<LANES>(w * dw);
  float val[V];
#pragma unroll
  for (int v = 0; v < V; ++v) val[v] = 0.0f;
  if (!renormalize) {
    load_row<LANES, V, VEC>(logits + (live ? t : 0) * experts, lane, experts, val);
    uint32_t mine = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t k = expert_of<LANES>(lane, v) < experts ? key_of(val[v]) : 0u;
      if (k > mine) mine = k;
      if (k <= kMaskedKey) val[v] = -__builtin_inff();
    }
    const uint32_t top = row_max<LANES>(mine);
    const float peak = top > kMaskedKey ? value_of(top) : 0.0f;
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      val[v] = expf(val[v] - peak);
      total += val[v];
    }
    total = row_sum<LANES>(total);
    const float f = top > kMaskedKey ? -mean / total : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) val[v] *= f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) row[expert_of<LANES>(lane, v)] = val[v];
  lanes_meet();
  if (id >= 0) atomicAdd(row + id, w * (renormalize ? dw - mean : dw));
  lanes_meet();
  if (!live) return;
  T* out = dlogits + t * experts;
  typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    const int e = expert_of<LANES>(lane, j);
    const f32x4 q = *reinterpret_cast<const f32x4*>(row + e);
    if constexpr (VEC) {
      if (e < experts) *reinterpret_cast<t4*>(out + e) = t4{(T)q[0], (T)q[1], (T)q[2], (T)q[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < experts) out[e + i] = (T)q[i];
    }
  }
}

template <int LANES>
dim3 grid_of(int tokens) {
  const topk_plan::Grid g = topk_plan::grid_of(tokens, LANES);
  return dim3(g.x, g.y);
}
struct Forward {
  template <int LANES, int V, bool VEC, typename T>
  static hipError_t launch(const T* logits, int32_t* ids, float* weights, int tokens, int experts, int topk,
                           int renormalize, hipStream_t stream) {
    return launch_kernel(moe_topk_kernel<LANES, V, VEC, T>, grid_of<LANES>(tokens), dim3(kThreads), 0, stream, logits, ids,
                         weights, tokens, experts, topk, renormalize);
  }
};
struct Backward {
  template <int LANES, int V, bool VEC, typename T>
  static hipError_t launch(const float* dweights, const T* logits, const int32_t* ids, const float* weights, T* dlogits,
                           int tokens, int experts, int topk, int renormalize, hipStream_t stream) {
    return launch_kernel(moe_topk_backward_kernel<LANES, V, VEC, T>, grid_of<LANES>(tokens), dim3(kThreads), 0, stream,
                         dweights, logits, ids, weights, dlogits, tokens, experts, topk, renormalize);
  }
};
template <typename K, bool VEC, typename T, typename... A>
hipError_t by_size(int tokens, int experts, int topk, A... a) {
  if (topk_plan::lanes_of(tokens, experts, topk) == 16) {
    if (experts <= 64) return K::template launch<16, 4, VEC, T>(a...);
    if (experts <= 128) return K::template launch<16, 8, VEC, T>(a...);
    return K::template launch<16, 16, VEC, T>(a...);
  }
  if (experts <= 256) return K::template launch<64, 4, VEC, T>(a...);
  if (experts <= 512) return K::template launch<64, 8, VEC, T>(a...);
  return K::template launch<64, 16, VEC, T>(a...);
}
// rows that start on four elements are read four at a time
template <typename K, typename T, typename... A>
hipError_t by_layout(int tokens, int experts, int topk, A... a) {
  return experts % 4 ? by_size<K, false, T>(tokens, experts, topk, a...) : by_size<K, true, T>(tokens, experts, topk, a...);
}

}  // namespace

hipError_t launch_moe_topk(const void* logits, bool half, int32_t* ids, float* weights, int tokens, int experts,
                           int topk, bool renormalize, hipStream_t stream) {
  if (half)
    return by_layout<Forward, _Float16>(tokens, experts, topk, static_cast<const _Float16*>(logits), ids, weights, tokens,
                                        experts, topk, (int)renormalize, stream);
  return by_layout<Forward, float>(tokens, experts, topk, static_cast<const float*>(logits), ids, weights, tokens, experts,
                                   topk, (int)renormalize, stream);
}

hipError_t launch_moe_topk_backward(const float* dweights, const void* logits, bool half, const int32_t* ids,
                                    const float* weights, void* dlogits, int tokens, int experts, int topk,
                                    bool renormalize, hipStream_t stream) {
  if (half)
    return by_layout<Backward, _Float16>(tokens, experts, topk, dweights, static_cast<const _Float16*>(logits), ids, weights,
                                         static_cast<_Float16*>(dlogits), tokens, experts, topk, (int)renormalize,
                                         stream);
  return by_layout<Backward, float>(tokens, experts, topk, dweights, static_cast<const float*>(logits), ids, weights,
                                    static_cast<float*>(dlogits), tokens, experts, topk, (int)renormalize, stream);
}

}  // namespace w4a16
