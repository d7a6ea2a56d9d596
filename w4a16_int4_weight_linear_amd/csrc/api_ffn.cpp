// api_ffn.cpp -- the C ABI of the feed-forward block's training operators:
// argument validation and dispatch, in the order and with the codes of api.cpp.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "../../include/w4a16.h"
#include "checks.hpp"
#include "dispatch.hpp"
#include "kernels.hpp"

namespace {

using w4a16::aligned;
using w4a16::as_status;
using w4a16::common_dense_checks;
using w4a16::DeviceInfo;
using w4a16::kMaxBufferBytes;
using w4a16::kMaxDim;
using w4a16::launch_t;
using w4a16::outputs_overlap;
using w4a16::status_of;
using w4a16::swiglu_skinny;
using w4a16::t_skinny;
using w4a16::t_workspace_bytes;
using w4a16::transposed_checks;
using w4a16::valid_group;

}  // namespace

extern "C" {

size_t w4a16_gemm_t_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group) || m <= 0 || n <= 0 || k <= 0 || k % group) return 0;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return 0;
  return t_workspace_bytes(m, n, k, group, dev);
}

w4a16_status w4a16_gemm_t(const uint16_t* d, const uint32_t* packed, const uint16_t* scales, uint16_t* y, int64_t m,
                          int64_t n, int64_t k, int32_t group, void* workspace, size_t workspace_bytes,
                          w4a16_stream_t stream) {
  const int c = transposed_checks(d, packed, scales, y, m, n, k, group);
  if (c < 0) return W4A16_OK;
  if (c != W4A16_OK) return as_status(c);
  if (!aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (n == 0) return status_of(w4a16::launch_zero_fill(y, (size_t)(m * k), st));
  const size_t need = t_workspace_bytes(m, n, k, group, dev);
  if (need && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (outputs_overlap({{y, 2 * m * k}, {workspace, (int64_t)need}},
                      {{d, 2 * m * n}, {packed, n * (k / 2)}, {scales, 2 * n * (k / group)}}))
    return W4A16_ERR_OVERLAP;
  return status_of(launch_t(d, packed, scales, y, m, n, k, group, need ? workspace : nullptr, dev, st));
}

size_t w4a16_gemm_swiglu_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group) || m <= 0 || n <= 0 || k <= 0 || k % group) return 0;
  if (m > kMaxDim || n > kMaxDim / 2 || k > kMaxDim) return 0;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return 0;
  if (swiglu_skinny(m, 2 * n, k, dev)) return 0;
  return w4a16::gemm_swiglu_workspace_bytes((int)m, (int)n, (int)k, dev);
}

w4a16_status w4a16_gemm_swiglu(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, uint16_t* y,
                               uint16_t* gate_up, int64_t m, int64_t n, int64_t k, int32_t group, void* workspace,
                               size_t workspace_bytes, w4a16_stream_t stream) {
  if (!valid_group(group)) return W4A16_ERR_GROUP;
  if (n < 0 || n > kMaxDim / 2) return W4A16_ERR_SHAPE;
  // the weights and the kept products have 2n columns (the size bounds are taken on those)
  const int c = common_dense_checks(x, packed, scales, y, m, 2 * n, k, group);
  if (c < 0) return W4A16_OK;
  if (c != W4A16_OK) return as_status(c);
  if (!aligned(gate_up, 16) || !aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (k == 0) {   // SiLU(0) * 0
    const hipError_t e = gate_up ? w4a16::launch_zero_fill(gate_up, (size_t)(2 * m * n), st) : hipSuccess;
    return status_of(e != hipSuccess ? e : w4a16::launch_zero_fill(y, (size_t)(m * n), st));
  }
  const bool streams = (!gate_up && m <= 16) || swiglu_skinny(m, 2 * n, k, dev);
  const size_t need = streams ? 0 : w4a16::gemm_swiglu_workspace_bytes((int)m, (int)n, (int)k, dev);
  if (need && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (outputs_overlap({{y, 2 * m * n}, {gate_up, gate_up ? 4 * m * n : 0}, {workspace, (int64_t)need}},
                      {{x, 2 * m * k}, {packed, n * k}, {scales, 4 * n * (k / group)}}))
    return W4A16_ERR_OVERLAP;
  // up to 16 rows with nothing kept: the decode product (its kernels for 1-4 rows are faster)
  if (!gate_up && m <= 16) return w4a16_gemv_swiglu(x, packed, scales, y, m, n, k, group, stream);
  if (streams) {
    return status_of(gate_up ? w4a16::launch_swiglu_skinny_keep(x, packed, scales, y, gate_up, (int)m, (int)n, (int)k,
                                                                group, dev, st)
                             : w4a16::launch_swiglu_skinny(x, packed, scales, y, (int)m, (int)n, (int)k, group, dev, st));
  }
  return status_of(w4a16::launch_gemm_swiglu(x, packed, scales, y, gate_up, (int)m, (int)n, (int)k, group,
                                             need ? workspace : nullptr, dev, st));
}

size_t w4a16_gemm_swiglu_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group) {
  if (n > kMaxDim / 2) return 0;
  return w4a16_gemm_t_workspace_bytes(m, n < 0 ? n : 2 * n, k, group);
}

w4a16_status w4a16_gemm_swiglu_backward(const uint16_t* dy, const uint16_t* gate_up, const uint32_t* packed,
                                        const uint16_t* scales, uint16_t* dgate_up, uint16_t* dx, int64_t m, int64_t n,
                                        int64_t k, int32_t group, void* workspace, size_t workspace_bytes,
                                        w4a16_stream_t stream) {
  if (!valid_group(group)) return W4A16_ERR_GROUP;
  if (n < 0 || n > kMaxDim / 2) return W4A16_ERR_SHAPE;
  // the product's sizes and buffers, with the pairs' gradient as its left side; k == 0 leaves
  // the pairs' gradient to write
  int c = transposed_checks(dgate_up, packed, scales, dx, m, 2 * n, k, group);
  if (c > 0) return as_status(c);
  if (m == 0 || (n == 0 && k == 0)) return W4A16_OK;
  if (n > 0) {
    if (!dy || !gate_up || !dgate_up) return W4A16_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(gate_up, 16) || !aligned(dgate_up, 16)) return W4A16_ERR_ALIGN;
    if (m > kMaxDim || 4 * m * n >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  }
  if (!aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const bool product = n > 0 && k > 0;
  const size_t need = product ? t_workspace_bytes(m, 2 * n, k, group, dev) : 0;
  if (need && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (outputs_overlap({{dgate_up, 4 * m * n}, {dx, 2 * m * k}, {workspace, (int64_t)need}},
                      {{dy, 2 * m * n}, {gate_up, 4 * m * n}, {packed, n * k}, {scales, 4 * n * (k / group)}}))
    return W4A16_ERR_OVERLAP;
  const bool few_rows = product && t_skinny(m, 2 * n, k, group, dev);
  if (few_rows && w4a16::swiglu_backward_skinny_fits((int)m, (int)(2 * n), (int)k, group, dev))
    return status_of(w4a16::launch_swiglu_backward_skinny(dy, gate_up, dgate_up, packed, scales, dx, (int)m,
                                                          (int)(2 * n), (int)k, group, need ? workspace : nullptr, dev,
                                                          st));
  // (the tiled product's padded copy of its left side, where it needs one, is filled on the way)
  uint16_t* padded = product && !few_rows ? w4a16::gemm_t_padded((int)(2 * n), workspace) : nullptr;
  if (n > 0) {
    const hipError_t e = w4a16::launch_swiglu_grad(dy, gate_up, dgate_up, padded, (int)m, (int)n, st);
    if (e != hipSuccess) return W4A16_ERR_HIP;
  }
  if (!product) return k > 0 ? status_of(w4a16::launch_zero_fill(dx, (size_t)(m * k), st)) : W4A16_OK;
  return status_of(launch_t(padded ? nullptr : dgate_up, packed, scales, dx, m, 2 * n, k, group,
                            need ? workspace : nullptr, dev, st));
}

size_t w4a16_gemm_dscales_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group) || m <= 0 || n <= 0 || k <= 0 || k % group) return 0;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return 0;
  return w4a16::dscales_workspace_bytes((int)m, (int)n, (int)k, group, dev);
}

w4a16_status w4a16_gemm_dscales(const uint16_t* d, const uint16_t* x, const uint32_t* packed, float* dscales, int64_t m,
                                int64_t n, int64_t k, int32_t group, void* workspace, size_t workspace_bytes,
                                w4a16_stream_t stream) {
  if (!valid_group(group)) return W4A16_ERR_GROUP;
  if (m < 0 || n < 0 || k < 0 || k % group) return W4A16_ERR_SHAPE;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return W4A16_ERR_SHAPE;
  if (n == 0 || k == 0) return W4A16_OK;
  if (!dscales || (m > 0 && (!d || !x || !packed))) return W4A16_ERR_NULL;
  if (!aligned(dscales, 16) || !aligned(workspace, 16) ||
      (m > 0 && (!aligned(d, 16) || !aligned(x, 16) || !aligned(packed, 16))))
    return W4A16_ERR_ALIGN;
  const int64_t n8 = (n + 7) / 8 * 8;
  if (n * (k / 2) >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  if (2 * m * k >= kMaxBufferBytes || 2 * m * n8 >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (m == 0)   // the empty sum (two 16-bit zeros per value)
    return status_of(w4a16::launch_zero_fill(reinterpret_cast<uint16_t*>(dscales), (size_t)(2 * n * (k / group)), st));
  const size_t need = w4a16::dscales_workspace_bytes((int)m, (int)n, (int)k, group, dev);
  if (need && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  if (outputs_overlap({{dscales, 4 * n * (k / group)}, {workspace, (int64_t)need}},
                      {{d, 2 * m * n}, {x, 2 * m * k}, {packed, n * (k / 2)}}))
    return W4A16_ERR_OVERLAP;
  return status_of(w4a16::launch_dscales(d, x, packed, dscales, (int)m, (int)n, (int)k, group,
                                         need ? workspace : nullptr, dev, st));
}

}  // extern "C"
