// api_moe.cpp -- the C ABI of the router's choice and of the routed experts' feed-forward for a few
// tokens: argument validation and dispatch, in the order and with the codes of api.cpp.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "../../include/w4a16.h"
#include "checks.hpp"
#include "kernels.hpp"
#include "moe_topk_plan.hpp"

namespace {

using w4a16::aligned;
using w4a16::as_status;
using w4a16::kMaxBufferBytes;
using w4a16::kMaxDim;
using w4a16::kMoeFfnPairs;
using w4a16::kMoeFfnTokens;
using w4a16::outputs_overlap;
using w4a16::status_of;
using w4a16::valid_group;

int topk_checks(int32_t dtype, int64_t tokens, int32_t experts, int32_t topk) {
  if (dtype != W4A16_F32 && dtype != W4A16_F16) return W4A16_ERR_RANGE;
  namespace plan = w4a16::topk_plan;
  if (tokens < 0 || tokens > plan::kTokens || topk < 1 || topk > experts || topk > plan::kSlots || experts > plan::kExperts)
    return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

int ffn_sizes(int64_t tokens, int32_t topk, int64_t hidden, int64_t inter, int32_t group) {
  if (!valid_group(group)) return W4A16_ERR_GROUP;
  if (tokens < 0 || tokens > kMoeFfnTokens || topk < 1 || topk > kMoeFfnPairs || tokens * topk > kMoeFfnPairs)
    return W4A16_ERR_SHAPE;
  if (hidden < 0 || hidden > w4a16::kMoeFfnHidden || hidden % group || inter < group || inter > kMaxDim || inter % group)
    return W4A16_ERR_SHAPE;
  // one expert's weights in 32-bit offsets
  if (inter * hidden >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

}  // namespace

extern "C" {

w4a16_status w4a16_moe_topk(const void* logits, int32_t dtype, int32_t* ids, float* weights, int64_t tokens,
                            int32_t experts, int32_t topk, int32_t renormalize, w4a16_stream_t stream) {
  const int c = topk_checks(dtype, tokens, experts, topk);
  if (c != W4A16_OK) return as_status(c);
  if (tokens == 0) return W4A16_OK;
  if (!logits || !ids || !weights) return W4A16_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(ids, 4) || !aligned(weights, 4)) return W4A16_ERR_ALIGN;
  const int64_t row = (int64_t)experts * (dtype == W4A16_F16 ? 2 : 4), slots = 4 * tokens * topk;
  if (outputs_overlap({{ids, slots}, {weights, slots}}, {{logits, tokens * row}})) return W4A16_ERR_OVERLAP;
  w4a16::DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  return status_of(w4a16::launch_moe_topk(logits, dtype == W4A16_F16, ids, weights, (int)tokens, experts, topk,
                                          renormalize != 0, reinterpret_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_moe_topk_backward(const float* dweights, const void* logits, int32_t dtype, const int32_t* ids,
                                     const float* weights, void* dlogits, int64_t tokens, int32_t experts,
                                     int32_t topk, int32_t renormalize, w4a16_stream_t stream) {
  const int c = topk_checks(dtype, tokens, experts, topk);
  if (c != W4A16_OK) return as_status(c);
  if (tokens == 0) return W4A16_OK;
  if (!dweights || !ids || !weights || !dlogits || (!renormalize && !logits)) return W4A16_ERR_NULL;
  if (!aligned(dlogits, 16) || (!renormalize && !aligned(logits, 16)) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(dweights, 4))
    return W4A16_ERR_ALIGN;
  const int64_t row = (int64_t)experts * (dtype == W4A16_F16 ? 2 : 4), slots = 4 * tokens * topk;
  if (outputs_overlap({{dlogits, tokens * row}},
                      {{dweights, slots}, {ids, slots}, {weights, slots}, {logits, renormalize ? 0 : tokens * row}}))
    return W4A16_ERR_OVERLAP;
  w4a16::DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  return status_of(w4a16::launch_moe_topk_backward(dweights, logits, dtype == W4A16_F16, ids, weights, dlogits,
                                                   (int)tokens, experts, topk, renormalize != 0,
                                                   reinterpret_cast<hipStream_t>(stream)));
}

size_t w4a16_moe_ffn_workspace_bytes(int64_t tokens, int32_t topk, int64_t hidden, int64_t inter, int32_t group) {
  if (ffn_sizes(tokens, topk, hidden, inter, group) != W4A16_OK || tokens == 0 || hidden == 0) return 0;
  return w4a16::moe_ffn_workspace_bytes((int)(tokens * topk), (int)hidden, (int)inter);
}

w4a16_status w4a16_moe_ffn(const uint16_t* x, const int32_t* ids, const float* weights, const uint32_t* gate_up,
                           const uint16_t* gate_up_scales, const uint32_t* down, const uint16_t* down_scales,
                           const uint16_t* residual, uint16_t* y, int64_t tokens, int32_t topk, int32_t experts,
                           int64_t hidden, int64_t inter, int32_t group, void* workspace, size_t workspace_bytes,
                           w4a16_stream_t stream) {
  const int c = ffn_sizes(tokens, topk, hidden, inter, group);
  if (c != W4A16_OK) return as_status(c);
  if (experts < 1) return W4A16_ERR_SHAPE;
  if (tokens == 0 || hidden == 0) return W4A16_OK;
  if (!x || !ids || !weights || !gate_up || !gate_up_scales || !down || !down_scales || !y) return W4A16_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(gate_up, 16) || !aligned(down, 16) ||
      !aligned(gate_up_scales, 2) || !aligned(down_scales, 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(workspace, 16))
    return W4A16_ERR_ALIGN;
  const size_t need = w4a16::moe_ffn_workspace_bytes((int)(tokens * topk), (int)hidden, (int)inter);
  if (!workspace || workspace_bytes < need) return W4A16_ERR_WORKSPACE;
  // (the residual's elements are read by the threads that then write y's: it may be y itself; an
  // expert's weights are below 2 GiB and experts below 2^31: the banks' sizes fit 64 bits)
  const int64_t rows = 2 * tokens * hidden, pairs = 4 * tokens * topk, banks = experts;
  if (outputs_overlap({{y, rows}, {workspace, (int64_t)need}},
                      {{x, rows}, {residual, residual && residual != y ? rows : 0}, {ids, pairs}, {weights, pairs},
                       {gate_up, banks * inter * hidden}, {gate_up_scales, banks * 4 * inter * (hidden / group)},
                       {down, banks * hidden * (inter / 2)}, {down_scales, banks * 2 * hidden * (inter / group)}}))
    return W4A16_ERR_OVERLAP;
  w4a16::DeviceInfo dev;
  if (w4a16::current_device_info(&dev) != hipSuccess) return W4A16_ERR_HIP;
  return status_of(w4a16::launch_moe_ffn(x, ids, weights, gate_up, gate_up_scales, down, down_scales, residual, y,
                                         (int)tokens, topk, experts, (int)hidden, (int)inter, group, workspace, dev,
                                         reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
