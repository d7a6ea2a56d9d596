// linear_epilogue.hpp -- what the linear layer folds into its product: with z = x . deq(W)^T + bias,
// y = act(z) + residual, in fp32 on the fp32 sums and rounded once; z, rounded once, on request.
//
// The product kernels take a LinearEpilogue behind their own arguments or nothing at all: the plain
// product's instances are those without.  The activation is a run-time choice, the same for the whole
// launch (a branch that no lane takes alone): a kernel per activation would differ by some twenty
// instructions per output.
#pragma once

#include "device.hpp"
#include "kernels.hpp"

namespace w4a16 {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kGeluTanh = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// 0.5 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) = 1 / (1 + e^-t): one exponential, no cancellation
__device__ inline float gelu_tanh_gate(float z) {
  return 1.0f / (1.0f + __expf(-kGeluTanh * __builtin_fmaf(kGeluCubic * z * z, z, z)));
}

__device__ inline float activate(int act, float z) {
  switch (act) {
    case W4A16_ACT_RELU: return z < 0.0f ? 0.0f : z;           // (NaN stays)
    case W4A16_ACT_SILU: return z / (1.0f + __expf(-z));
    case W4A16_ACT_GELU: return 0.5f * z * erfcf(-kSqrtHalf * z);
    case W4A16_ACT_GELU_TANH: return z * gelu_tanh_gate(z);
    default: return z;
  }
}

// act'(z); relu' is 0 at 0
__device__ inline float activation_slope(int act, float z) {
  switch (act) {
    case W4A16_ACT_RELU: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case W4A16_ACT_SILU: {
      const float sig = 1.0f / (1.0f + __expf(-z));
      return sig * (1.0f + z * (1.0f - sig));
    }
    case W4A16_ACT_GELU:
      return __builtin_fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f * erfcf(-kSqrtHalf * z));
    case W4A16_ACT_GELU_TANH: {
      const float sig = gelu_tanh_gate(z);
      return sig + z * sig * (1.0f - sig) * (kGeluTanh * (1.0f + 3.0f * kGeluCubic * z * z));
    }
    default: return 1.0f;
  }
}

// One output: element `at` of y (and of residual and pre), column n, from the product's sum v.
__device__ inline void store_result(uint16_t* y, size_t at, int, float v) { y[at] = float_to_half_bits(v); }
__device__ inline void store_result(uint16_t* y, size_t at, int n, float v, const LinearEpilogue& ep) {
  const float z = ep.bias ? v + half_bits_to_float(ep.bias[n]) : v;
  if (ep.pre) ep.pre[at] = float_to_half_bits(z);
  float o = activate(ep.act, z);
  if (ep.residual) o += half_bits_to_float(ep.residual[at]);
  y[at] = float_to_half_bits(o);
}

}  // namespace w4a16
