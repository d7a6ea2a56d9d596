// api_linear.cpp -- the C ABI of the linear layer with bias, activation and residual: argument
// validation and dispatch, in the order and with the codes of api_ffn.cpp.
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
using w4a16::kCounterBytes;
using w4a16::kMaxBufferBytes;
using w4a16::kMaxDim;
using w4a16::LinearEpilogue;
using w4a16::outputs_overlap;
using w4a16::status_of;
using w4a16::valid_group;

bool valid_activation(int32_t a) { return a >= W4A16_ACT_NONE && a <= W4A16_ACT_GELU_TANH; }

// The kernels of a layer of checked sizes: one row and two to four on the decode kernels while the rows fit
// in LDS, few rows on the weight-streaming kernel (the rule at kSkinnyRows), else the tiles.
enum class Path { kOneRow, kFourRows, kStream, kTiles };
struct Route {
  Path path = Path::kTiles;
  w4a16::GemvPlan gemv;
  int blocks = 0;
  size_t lds = 0;
};
Route route(int64_t m, int64_t n, int64_t k, int32_t group, const DeviceInfo& dev) {
  Route r;
  if (m == 1) {
    r.gemv = w4a16::gemv_plan(1, (int)n, (int)k, group, dev);
    if (r.gemv.ok) r.path = Path::kOneRow;
  } else if (m <= 4 && w4a16::gemv_mfma_plan((int)m, (int)n, (int)k, group, dev, &r.blocks, &r.lds)) {
    r.path = Path::kFourRows;
  }
  if (r.path == Path::kTiles && w4a16::swiglu_skinny(m, n, k, dev)) r.path = Path::kStream;
  return r;
}

size_t grad_bytes(int64_t m, int64_t n, bool bias) {
  return w4a16::linear_grad_workspace_bytes((int)m, (int)n, bias);
}
// The product's workspace and the column sums' share one: counters first, then either's.
size_t backward_bytes(int64_t m, int64_t n, int64_t k, int32_t group, bool bias, const DeviceInfo& dev) {
  const size_t product = n > 0 && k > 0 ? w4a16::t_workspace_bytes(m, n, k, group, dev) : 0;
  const size_t sums = m > 0 && n > 0 ? grad_bytes(m, n, bias) : 0;
  const size_t base = product ? (product + 255) & ~(size_t)255 : (sums ? kCounterBytes : 0);
  return sums ? base + sums : product;
}

}  // namespace

extern "C" {

size_t w4a16_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group) || m <= 0 || n <= 0 || k <= 0 || k % group) return 0;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return 0;
  if (route(m, n, k, group, dev).path != Path::kTiles) return 0;
  return w4a16::gemm_linear_workspace_bytes((int)m, (int)n, (int)k, dev);
}

w4a16_status w4a16_linear(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, const uint16_t* bias,
                          const uint16_t* residual, uint16_t* y, uint16_t* pre, int64_t m, int64_t n, int64_t k,
                          int32_t group, int32_t activation, void* workspace, size_t workspace_bytes,
                          w4a16_stream_t stream) {
  if (!valid_activation(activation)) return W4A16_ERR_RANGE;
  const int c = common_dense_checks(x, packed, scales, y, m, n, k, group);
  if (c < 0) return W4A16_OK;
  if (c != W4A16_OK) return as_status(c);
  if (k == 0) return W4A16_ERR_SHAPE;
  if (!aligned(bias, 16) || !aligned(residual, 16) || !aligned(pre, 16) || !aligned(workspace, 16))
    return W4A16_ERR_ALIGN;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const Route r = route(m, n, k, group, dev);
  const size_t need = r.path == Path::kTiles ? w4a16::gemm_linear_workspace_bytes((int)m, (int)n, (int)k, dev) : 0;
  if (need && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  // (every element of the residual is read by the thread that then writes y's: it may be y itself)
  const int64_t plane = 2 * m * n;
  if (outputs_overlap({{y, plane}, {pre, pre ? plane : 0}, {workspace, (int64_t)need}},
                      {{x, 2 * m * k}, {packed, n * (k / 2)}, {scales, 2 * n * (k / group)}, {bias, bias ? 2 * n : 0},
                       {residual, residual && residual != y ? plane : 0}}))
    return W4A16_ERR_OVERLAP;
  const LinearEpilogue ep = {bias, residual, pre, activation};
  const int mi = (int)m, ni = (int)n, ki = (int)k;
  switch (r.path) {
    case Path::kOneRow:
      return status_of(w4a16::launch_gemv_linear(x, packed, scales, y, ni, ki, group, ep, r.gemv, dev, st));
    case Path::kFourRows:
      return status_of(w4a16::launch_gemv_mfma_linear(x, packed, scales, y, mi, ni, ki, group, ep, r.blocks, r.lds, dev, st));
    case Path::kStream:
      return status_of(w4a16::launch_linear_skinny(x, packed, scales, y, mi, ni, ki, group, ep, dev, st));
    default:
      return status_of(w4a16::launch_gemm_linear(x, packed, scales, y, mi, ni, ki, group, ep, need ? workspace : nullptr,
                                                 dev, st));
  }
}

size_t w4a16_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group) || m <= 0 || n <= 0 || k < 0 || k % group) return 0;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return 0;
  return backward_bytes(m, n, k, group, true, dev);
}

w4a16_status w4a16_linear_backward(const uint16_t* dy, const uint16_t* pre, const uint32_t* packed,
                                   const uint16_t* scales, uint16_t* dpre, float* dbias, uint16_t* dx, int64_t m,
                                   int64_t n, int64_t k, int32_t group, int32_t activation, void* workspace,
                                   size_t workspace_bytes, w4a16_stream_t stream) {
  if (!valid_activation(activation)) return W4A16_ERR_RANGE;
  // the product's sizes and buffers; k == 0 leaves the pre-activations' and the bias's gradient to write
  const bool slope = activation != W4A16_ACT_NONE;
  int c = w4a16::transposed_checks(dy, packed, scales, dx, m, n, k, group);
  if (c > 0) return as_status(c);
  if (n > 0 && m > 0) {
    if (!dy || (slope ? (!pre || !dpre) : false)) return W4A16_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(pre, 16) || !aligned(dpre, 16)) return W4A16_ERR_ALIGN;
    if (2 * m * ((n + 7) / 8 * 8) >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  }
  if (!slope && (pre || dpre)) return W4A16_ERR_SHAPE;
  if (!aligned(dbias, 16) || !aligned(workspace, 16)) return W4A16_ERR_ALIGN;
  if ((m == 0 && (n == 0 || !dbias)) || (n == 0 && k == 0)) return W4A16_OK;
  DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (m == 0)   // the empty sum (two 16-bit zeros per value)
    return status_of(w4a16::launch_zero_fill(reinterpret_cast<uint16_t*>(dbias), (size_t)(2 * n), st));
  if (n == 0) return status_of(w4a16::launch_zero_fill(dx, (size_t)(m * k), st));
  const size_t need = backward_bytes(m, n, k, group, dbias != nullptr, dev);
  if (need && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
  const int64_t plane = 2 * m * n;
  if (outputs_overlap({{dpre, slope ? plane : 0}, {dx, 2 * m * k}, {dbias, dbias ? 4 * n : 0}, {workspace, (int64_t)need}},
                      {{dy, plane}, {pre, slope ? plane : 0}, {packed, n * (k / 2)}, {scales, 2 * n * (k / group)}}))
    return W4A16_ERR_OVERLAP;
  const bool product = k > 0;
  const bool tw = product && w4a16::t_workspace_bytes(m, n, k, group, dev) != 0;
  if (product && (slope || dbias) && w4a16::t_skinny(m, n, k, group, dev) &&
      w4a16::linear_backward_skinny_fits((int)m, (int)n, (int)k, group, dev))
    return status_of(w4a16::launch_linear_backward_skinny(dy, pre, dpre, dbias, packed, scales, dx, (int)m, (int)n, (int)k,
                                                          group, activation, tw ? workspace : nullptr, dev, st));
  // (the tiled product's padded copy of its left side, where it needs one, is filled on the way)
  uint16_t* padded = product && slope && !w4a16::t_skinny(m, n, k, group, dev)
                         ? w4a16::gemm_t_padded((int)n, workspace)
                         : nullptr;
  if (slope || dbias) {
    const size_t sums = dbias ? grad_bytes(m, n, true) : 0;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const hipError_t e = w4a16::launch_linear_grad(
        dy, slope ? pre : nullptr, dpre, padded, dbias, (int)m, (int)n, activation,
        reinterpret_cast<uint32_t*>(sums ? ws : nullptr), reinterpret_cast<float*>(sums ? ws + (need - sums) : nullptr), st);
    if (e != hipSuccess) return W4A16_ERR_HIP;
  }
  if (!product) return W4A16_OK;
  return status_of(w4a16::launch_t(padded ? nullptr : (slope ? dpre : dy), packed, scales, dx, m, n, k, group,
                                   tw ? workspace : nullptr, dev, st));
}

}  // extern "C"
