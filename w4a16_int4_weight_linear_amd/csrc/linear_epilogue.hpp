// linear_epilogue.hpp -- what the linear layer folds into its product: with z = x . deq(W)^T + bias,
// y = act(z) + residual, in fp32 on the fp32 sums and rounded once; z, rounded once, on request.
//
// The product kernels take a LinearEpilogue behind their own arguments or nothing at all: the plain
// product's instances are those without.  The activation is a run-time choice, the same for the whole
// launch (a branch that no lane takes alone): a kernel per activation would differ by some twenty
// instructions per output.
#pragma once

#include <type_traits>

#include "device.hpp"
#include "kernels.hpp"

namespace w4a16 {

constexpr float kGeluTanh = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// (the reciprocal and exponential instructions: within about one and two fp32 units in the last place)
__device__ inline float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }

// 0.5 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) = 1 / (1 + e^-t): one exponential, no cancellation
__device__ inline float gelu_tanh_gate(float z) {
  return reciprocal(1.0f + __expf(-kGeluTanh * __builtin_fmaf(kGeluCubic * z * z, z, z)));
}

// Phi(z), the normal distribution, and e = exp(-z^2 / 2).  Phi(-|z|) = e t P(t) with t = 1 / (1 + 0.3 |z|):
// P is the polynomial of degree 7 with the smallest relative error over 0 <= |z| <= 14 (below fp32's
// range from there on), found by linear programming against scipy's erfcx: 2^-22.8.  Evaluated in
// fp32, the rounding of z^2 / 2 before the exponential grows with it: largest relative error (numpy's fp32 in
// these steps, 2 million values a range) 2^-20.7 to |z| = 2, 2^-20.1 to 4, 2^-18.5 to 8, 2^-17.0 to 13, where Phi is
// 1e-38; half a step of fp16 is 2^-11.  17 instructions; erfcf takes some 60.
__device__ inline float normal_gate(float z, float& e) {
  e = __expf(-0.5f * z * z);
  const float t = reciprocal(__builtin_fmaf(0.3f, __builtin_fabsf(z), 1.0f));
  float p = 0.0355625241f;
  p = __builtin_fmaf(p, t, -0.156767259f);
  p = __builtin_fmaf(p, t, 0.205660417f);
  p = __builtin_fmaf(p, t, -0.053099666f);
  p = __builtin_fmaf(p, t, 0.12828037f);
  p = __builtin_fmaf(p, t, 0.0999908793f);
  p = __builtin_fmaf(p, t, 0.1207427f);
  p = __builtin_fmaf(p, t, 0.119629966f);
  p *= e * t;
  return z < 0.0f ? p : 1.0f - p;
}

template <int ACT>
__device__ inline float activation_of(float z) {
  if constexpr (ACT == W4A16_ACT_RELU) {
    return z < 0.0f ? 0.0f : z;                       // (NaN stays)
  } else if constexpr (ACT == W4A16_ACT_SILU) {
    return z * reciprocal(1.0f + __expf(-z));
  } else if constexpr (ACT == W4A16_ACT_GELU) {
    float e;
    return z * normal_gate(z, e);
  } else if constexpr (ACT == W4A16_ACT_GELU_TANH) {
    return z * gelu_tanh_gate(z);
  } else {
    return z;
  }
}

// act'(z); relu' is 0 at 0.  z is what the forward pass kept in fp16, where a pre-activation past 65504 is infinite
// (the forward pass took it as it was): its slope is that of fp16's largest value, 0 or 1 in every activation, as
// infinity times the 0 that the formulas have there would be NaN.  (NaN stays.)
__device__ inline float finite_of(float z) {
  return __builtin_isinf(z) ? __builtin_copysignf(65504.0f, z) : z;
}
template <int ACT>
__device__ inline float slope_of(float z) {
  if constexpr (ACT == W4A16_ACT_SILU || ACT == W4A16_ACT_GELU || ACT == W4A16_ACT_GELU_TANH) z = finite_of(z);
  if constexpr (ACT == W4A16_ACT_RELU) {
    return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  } else if constexpr (ACT == W4A16_ACT_SILU) {
    const float sig = reciprocal(1.0f + __expf(-z));
    return sig * (1.0f + z * (1.0f - sig));
  } else if constexpr (ACT == W4A16_ACT_GELU) {
    float e;
    const float gate = normal_gate(z, e);
    return __builtin_fmaf(z * 0.39894228040143268f, e, gate);          // 1 / sqrt(2 pi)
  } else if constexpr (ACT == W4A16_ACT_GELU_TANH) {
    const float sig = gelu_tanh_gate(z);
    return sig + z * sig * (1.0f - sig) * (kGeluTanh * (1.0f + 3.0f * kGeluCubic * z * z));
  } else {
    return 1.0f;
  }
}

// f(std::integral_constant of the activation): one branch around all the values that f deals with.
template <typename F>
__device__ inline void with_activation(int act, F f) {
  switch (act) {
    case W4A16_ACT_RELU: f(std::integral_constant<int, W4A16_ACT_RELU>{}); break;
    case W4A16_ACT_SILU: f(std::integral_constant<int, W4A16_ACT_SILU>{}); break;
    case W4A16_ACT_GELU: f(std::integral_constant<int, W4A16_ACT_GELU>{}); break;
    case W4A16_ACT_GELU_TANH: f(std::integral_constant<int, W4A16_ACT_GELU_TANH>{}); break;
    default: break;
  }
}
template <int N>
__device__ inline void activate(int act, float (&v)[N]) {
  with_activation(act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activation_of<decltype(a)::value>(v[i]);
  });
}
// d *= act'(z)
template <int N>
__device__ inline void times_slope(int act, const float (&z)[N], float (&d)[N]) {
  with_activation(act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] *= slope_of<decltype(a)::value>(z[i]);
  });
}

// Eight elements of a row (left: how many of them there are).  VEC: on 16 bytes; else two-byte alignment.
template <bool VEC>
__device__ inline void store_eight(uint16_t* p, int left, const f16x8& o) {
  if constexpr (VEC) {
    *reinterpret_cast<f16x8*>(p) = o;
  } else {
    const u32x4 v = __builtin_bit_cast(u32x4, o);
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    } else if (reinterpret_cast<uintptr_t>(p) & 2) {
      p[0] = (uint16_t)v[0];
#pragma unroll
      for (int j = 0; j < 3; ++j) *reinterpret_cast<uint32_t*>(p + 1 + 2 * j) = __builtin_amdgcn_alignbit(v[j + 1], v[j], 16);
      p[7] = (uint16_t)(v[3] >> 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(p + 2 * j) = v[j];
    }
  }
}

// One output: element `at` of y (ep.y; and of residual and pre), column n, from the product's sum v.
__device__ inline void store_result(uint16_t* y, size_t at, int, float v) { y[at] = float_to_half_bits(v); }
__device__ inline void store_result(uint16_t*, size_t at, int n, float v, const LinearEpilogue& ep) {
  const float z = ep.bias ? v + half_bits_to_float(ep.bias[n]) : v;
  if (ep.pre) ep.pre[at] = float_to_half_bits(z);
  float o[1] = {z};
  activate(ep.act, o);
  if (ep.residual) o[0] += half_bits_to_float(ep.residual[at]);
  ep.y[at] = float_to_half_bits(o[0]);
}

}  // namespace w4a16
