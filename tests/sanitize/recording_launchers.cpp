// recording_launchers.cpp -- host stand-ins for the device launchers that note who called them
// and report success, for driving the C ABI's dispatch without a GPU.
#include "recording_launchers.hpp"

#include "../../w4a16_int4_weight_linear_amd/csrc/kernels.hpp"

Recorded g_rec;
Answers g_ans;

namespace w4a16 {

static hipError_t note(const char* name) {
  g_rec.launches.push_back(name);
  return hipSuccess;
}

GemvPlan gemv_plan(int m, int, int, int, const DeviceInfo&, bool) {
  GemvPlan p;
  p.ok = m <= 4;
  return p;
}
int64_t gemv_max_k(int, int, const DeviceInfo&) { return 0; }
hipError_t launch_gemv(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                       const GemvPlan&, const DeviceInfo&, hipStream_t) { return note("gemv"); }
bool gemv_mfma_plan(int, int, int, int, const DeviceInfo&, int*, size_t*, bool) { return false; }
hipError_t launch_gemv_mfma(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int, int,
                            size_t, const DeviceInfo&, hipStream_t, bool) { return note("gemv_mfma"); }
bool gemm_skinny_fits(int, int, int, const DeviceInfo&) { return g_ans.skinny_fits; }
hipError_t launch_gemm_skinny(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                              const DeviceInfo&, hipStream_t) { return note("gemm_skinny"); }
hipError_t launch_swiglu_skinny(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                                const DeviceInfo&, hipStream_t) { return note("swiglu_skinny"); }
hipError_t launch_swiglu_skinny_keep(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, uint16_t*, int, int,
                                     int, int, const DeviceInfo&, hipStream_t) { return note("swiglu_skinny_keep"); }
size_t gemm_workspace_bytes(int64_t, int64_t, int64_t, int, const DeviceInfo&) { return 0; }
hipError_t gemm_scratch(const DeviceInfo&, void**, size_t*) { return hipErrorNoDevice; }
size_t gemm_workspace_flags_offset(int64_t, int64_t, int64_t, const DeviceInfo&) { return 0; }
hipError_t launch_gemm(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int, void*,
                       const DeviceInfo&, hipStream_t) { return note("gemm"); }
hipError_t launch_grouped_gemm(const uint16_t*, const uint32_t*, const uint16_t*, const int32_t*, uint16_t*, int,
                               int, int, int, int, const DeviceInfo&, hipStream_t) { return note("grouped"); }
hipError_t launch_grouped_gemm_gather(const uint16_t*, const int32_t*, int, const uint32_t*, const uint16_t*,
                                      const int32_t*, uint16_t*, int, int, int, int, int, const DeviceInfo&,
                                      hipStream_t) { return note("grouped_gather"); }
hipError_t launch_grouped_gemm_swiglu(const uint16_t*, const int32_t*, int, const uint32_t*, const uint16_t*,
                                      const int32_t*, uint16_t*, int, int, int, int, int, const DeviceInfo&,
                                      hipStream_t) { return note("grouped_swiglu"); }
size_t moe_route_lds(int experts) { return (size_t)experts * 4; }
hipError_t launch_moe_route(const int32_t*, int, int, int, int32_t*, int32_t*, int32_t*, const DeviceInfo&,
                            hipStream_t) { return note("moe_route"); }
hipError_t launch_moe_combine(const uint16_t*, const int32_t*, const float*, uint16_t*, int, int, int, int,
                              hipStream_t) { return note("moe_combine"); }
hipError_t launch_zero_fill(uint16_t*, size_t, hipStream_t) { return note("zero_fill"); }
int probe_sink_words(const DeviceInfo& dev) { return dev.num_cu * 8; }
hipError_t launch_stream_read(const void*, size_t, uint32_t*, const DeviceInfo&, hipStream_t) { return note("probe"); }

size_t gemm_swiglu_workspace_bytes(int, int, int, const DeviceInfo&) { return g_ans.workspace; }
hipError_t launch_gemm_swiglu(const uint16_t* x, const uint32_t*, const uint16_t*, uint16_t*, uint16_t*, int, int, int,
                              int, void* workspace, const DeviceInfo&, hipStream_t) {
  g_rec.left = x;
  g_rec.workspace = workspace;
  return note("gemm_swiglu");
}
size_t gemm_t_workspace_bytes(int, int, int, const DeviceInfo&) { return g_ans.workspace; }
uint16_t* gemm_t_padded(int n, void* workspace) {
  return n % 8 ? reinterpret_cast<uint16_t*>(behind_counters(workspace)) : nullptr;
}
hipError_t launch_gemm_t(const uint16_t* d, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                         void* workspace, const DeviceInfo&, hipStream_t) {
  g_rec.left = d;
  g_rec.workspace = workspace;
  return note("gemm_t");
}
bool gemm_t_skinny_fits(int, int, int, int, const DeviceInfo&) { return g_ans.skinny_fits; }
size_t gemm_t_skinny_workspace_bytes(int, int, int, int, const DeviceInfo&) { return g_ans.workspace; }
hipError_t launch_gemm_t_skinny(const uint16_t* d, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int,
                                void* workspace, const DeviceInfo&, hipStream_t) {
  g_rec.left = d;
  g_rec.workspace = workspace;
  return note("gemm_t_skinny");
}
bool swiglu_backward_skinny_fits(int, int n, int, int, const DeviceInfo&) { return g_ans.grad_fits && n % 8 == 0; }
hipError_t launch_swiglu_backward_skinny(const uint16_t* dh, const uint16_t*, uint16_t*, const uint32_t*,
                                         const uint16_t*, uint16_t*, int, int, int, int, void* workspace,
                                         const DeviceInfo&, hipStream_t) {
  g_rec.left = dh;
  g_rec.workspace = workspace;
  return note("swiglu_backward_skinny");
}
hipError_t launch_swiglu_grad(const uint16_t*, const uint16_t*, uint16_t*, uint16_t* padded, int, int, hipStream_t) {
  g_rec.padded = padded;
  return note("swiglu_grad");
}
size_t dscales_workspace_bytes(int, int, int, int, const DeviceInfo&) { return g_ans.workspace; }
hipError_t launch_dscales(const uint16_t* d, const uint16_t*, const uint32_t*, float*, int, int, int, int,
                          void* workspace, const DeviceInfo&, hipStream_t) {
  g_rec.left = d;
  g_rec.workspace = workspace;
  return note("dscales");
}

}  // namespace w4a16
