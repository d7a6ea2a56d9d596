// swiglu_grad.hip -- gradient of h = SiLU(g) u with respect to g and u, elementwise on gfx950.
//
// The formula is in swiglu_grad.hpp.  gate_up and dgate_up interleave the pairs, so output i of the
// flattened [m, n] owns elements 2 i and 2 i + 1 and rows need no alignment of their own.
//
// Bound by memory: 10 bytes per output (2048 x 17408: 357 MB in 64-66 us = 5.5 TB/s; without
// non-temporal loads 70-86).  A thread takes eight outputs (one 16-byte load
// of dh, two of gate_up, two stores).
#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "swiglu_grad.hpp"

namespace w4a16 {
namespace {

__global__ void __launch_bounds__(256)
swiglu_grad_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gate_up,
                   uint16_t* __restrict__ dgate_up, size_t count) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i + 8 <= count) {
    // (both inputs are read once: non-temporal)
    const f16x8 d = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(dh + i));
    f16x8 zv[2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
      zv[p] = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(gate_up + 2 * i + 8 * p));
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f16x8 z = zv[p];
      f16x8 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f16x2 r = grad_pair(z[2 * e], z[2 * e + 1], d[4 * p + e]);
        o[2 * e] = r[0];
        o[2 * e + 1] = r[1];
      }
      *reinterpret_cast<f16x8*>(dgate_up + 2 * i + 8 * p) = o;
    }
  } else {
    for (size_t e = i; e < count; ++e) {
      const f16x2 r = grad_pair(__builtin_bit_cast(_Float16, gate_up[2 * e]),
                                __builtin_bit_cast(_Float16, gate_up[2 * e + 1]), __builtin_bit_cast(_Float16, dh[e]));
      dgate_up[2 * e] = __builtin_bit_cast(uint16_t, (_Float16)r[0]);
      dgate_up[2 * e + 1] = __builtin_bit_cast(uint16_t, (_Float16)r[1]);
    }
  }
}

// The same for rows of 2 n elements that are no multiple of 8: one output per thread, written
// to dgate_up and to the padded copy that the product reads (np: its pairs per row).
__global__ void __launch_bounds__(256)
swiglu_grad_padded_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gate_up,
                          uint16_t* __restrict__ dgate_up, uint16_t* __restrict__ padded, int n, int np, size_t count) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;     // over m x np
  if (i >= count) return;
  const size_t m = i / (uint32_t)np;
  const int c = (int)(i - m * (uint32_t)np);
  f16x2 r = {};
  if (c < n) {
    const size_t at = m * (size_t)n + c;
    const f16x2 z = *reinterpret_cast<const f16x2*>(gate_up + 2 * at);
    r = grad_pair(z[0], z[1], __builtin_bit_cast(_Float16, dh[at]));
    *reinterpret_cast<f16x2*>(dgate_up + 2 * at) = r;
  }
  *reinterpret_cast<f16x2*>(padded + 2 * i) = r;
}

}  // namespace

hipError_t launch_swiglu_grad(const uint16_t* dh, const uint16_t* gate_up, uint16_t* dgate_up, uint16_t* padded, int m,
                              int n, hipStream_t stream) {
  if (padded) {
    const int np = (2 * n + 7) / 8 * 4;
    const size_t count = (size_t)m * np;
    return launch_kernel(swiglu_grad_padded_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, stream, dh,
                         gate_up, dgate_up, padded, n, np, count);
  }
  const size_t count = (size_t)m * n;
  return launch_kernel(swiglu_grad_kernel, dim3((unsigned)((count + 2047) / 2048)), dim3(256), 0, stream, dh, gate_up,
                       dgate_up, count);
}

}  // namespace w4a16
