// block_recording_launchers.cpp -- host stand-ins for the device launchers that api_linear.cpp and api_moe.cpp
// call, and for the device, which note who called them and report success.
#include "block_recording_launchers.hpp"

#include "../../w4a16_int4_weight_linear_amd/csrc/kernels.hpp"

BlockRecorded g_rec;
BlockAnswers g_ans;

namespace w4a16 {

static hipError_t note(const char* name) {
  g_rec.launches.push_back(name);
  return hipSuccess;
}
static hipError_t product(const char* name, const void* left, const void* workspace) {
  g_rec.left = left;
  g_rec.workspace = workspace;
  return note(name);
}

hipError_t current_device_info(DeviceInfo* out) {
  out->device = 0;
  out->num_cu = 256;
  out->max_lds = 160 * 1024;
  return hipSuccess;
}
GemvPlan gemv_plan(int, int, int, int, const DeviceInfo&, bool) {
  GemvPlan p;
  p.ok = g_ans.one_row;
  return p;
}
bool gemv_mfma_plan(int, int, int, int, const DeviceInfo&, int*, size_t*, bool) { return g_ans.four_rows; }
bool gemm_skinny_fits(int, int, int, const DeviceInfo&) { return g_ans.skinny_fits; }
bool gemm_t_skinny_fits(int, int, int, int, const DeviceInfo&) { return g_ans.skinny_fits; }
bool linear_backward_skinny_fits(int, int, int, int, const DeviceInfo&) { return g_ans.grad_fits; }
size_t gemm_linear_workspace_bytes(int, int, int, const DeviceInfo&) { return g_ans.product; }
size_t gemm_t_workspace_bytes(int, int, int, const DeviceInfo&) { return g_ans.product; }
size_t gemm_t_skinny_workspace_bytes(int, int, int, int, const DeviceInfo&) { return g_ans.product; }
size_t linear_grad_workspace_bytes(int, int, bool bias) { return bias ? g_ans.sums : 0; }
size_t moe_ffn_workspace_bytes(int, int, int) { return g_ans.moe; }
uint16_t* gemm_t_padded(int n, void* workspace) {
  return n % 8 ? reinterpret_cast<uint16_t*>(behind_counters(workspace)) : nullptr;
}

hipError_t launch_gemv_linear(const uint16_t* x, const uint32_t*, const uint16_t*, uint16_t*, int, int, int,
                              const LinearEpilogue&, const GemvPlan&, const DeviceInfo&, hipStream_t) {
  return product("gemv", x, nullptr);
}
hipError_t launch_gemv_mfma_linear(const uint16_t* x, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                                   const LinearEpilogue&, int, size_t, const DeviceInfo&, hipStream_t) {
  return product("gemv_mfma", x, nullptr);
}
hipError_t launch_linear_skinny(const uint16_t* x, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                                const LinearEpilogue&, const DeviceInfo&, hipStream_t) {
  return product("skinny", x, nullptr);
}
hipError_t launch_gemm_linear(const uint16_t* x, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                              const LinearEpilogue&, void* workspace, const DeviceInfo&, hipStream_t) {
  return product("tiles", x, workspace);
}
hipError_t launch_linear_grad(const uint16_t*, const uint16_t* pre, uint16_t*, uint16_t* padded, float*, int, int, int,
                              uint32_t* counters, float* partials, hipStream_t) {
  g_rec.pre = pre;
  g_rec.padded = padded;
  g_rec.counters = counters;
  g_rec.partials = partials;
  return note("grad");
}
hipError_t launch_linear_backward_skinny(const uint16_t* dy, const uint16_t*, uint16_t*, float*, const uint32_t*,
                                         const uint16_t*, uint16_t*, int, int, int, int, int, void* workspace,
                                         const DeviceInfo&, hipStream_t) {
  return product("grad_in_skinny", dy, workspace);
}
hipError_t launch_gemm_t(const uint16_t* d, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                         void* workspace, const DeviceInfo&, hipStream_t) {
  return product("gemm_t", d, workspace);
}
hipError_t launch_gemm_t_skinny(const uint16_t* d, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                                void* workspace, const DeviceInfo&, hipStream_t) {
  return product("gemm_t_skinny", d, workspace);
}
hipError_t launch_zero_fill(uint16_t*, size_t, hipStream_t) { return note("zero_fill"); }
hipError_t launch_moe_topk(const void*, bool half, int32_t*, float*, int, int, int, bool, hipStream_t) {
  return note(half ? "topk16" : "topk32");
}
hipError_t launch_moe_topk_backward(const float*, const void*, bool half, const int32_t*, const float*, void*, int, int,
                                    int, bool, hipStream_t) {
  return note(half ? "topk_backward16" : "topk_backward32");
}
hipError_t launch_moe_ffn(const uint16_t* x, const int32_t*, const float*, const uint32_t*, const uint16_t*,
                          const uint32_t*, const uint16_t*, const uint16_t*, uint16_t*, int, int, int, int, int, int,
                          void* workspace, const DeviceInfo&, hipStream_t) {
  return product("moe_ffn", x, workspace);
}

}  // namespace w4a16
