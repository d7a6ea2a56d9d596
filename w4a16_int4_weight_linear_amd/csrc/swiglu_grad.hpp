// swiglu_grad.hpp -- gradient of h = SiLU(g) u for one pair: sig = 1 / (1 + e^-g),
// dg = dh u sig (1 + g (1 - sig)), du = dh g sig, in fp32, each rounded once to fp16 (the
// gradient is an output, and the fp16 operand of the product that follows).
#pragma once
#include "device.hpp"

namespace w4a16 {

__device__ inline f16x2 grad_pair(_Float16 g16, _Float16 u16, _Float16 dh16) {
  const float g = (float)g16, u = (float)u16, dh = (float)dh16;
  const float sig = __builtin_amdgcn_rcpf(1.0f + __expf(-g));   // (within one fp32 unit in the last place)
  return f16x2{(_Float16)(dh * u * sig * (1.0f + g * (1.0f - sig))), (_Float16)(dh * g * sig)};
}

}  // namespace w4a16
