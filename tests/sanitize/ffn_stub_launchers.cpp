// ffn_stub_launchers.cpp -- host-only stand-ins for the device launchers of the
// feed-forward block's operators (see stub_launchers.cpp).  Every launcher
// reports "no device"; nothing here touches a GPU.
#include "../../w4a16_int4_weight_linear_amd/csrc/kernels.hpp"

namespace w4a16 {

hipError_t launch_swiglu_skinny_keep(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, uint16_t*, int, int,
                                     int, int, const DeviceInfo&, hipStream_t) { return hipErrorNoDevice; }
size_t gemm_swiglu_workspace_bytes(int, int, int, const DeviceInfo&) { return 0; }
hipError_t launch_gemm_swiglu(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, uint16_t*, int, int, int,
                              int, void*, const DeviceInfo&, hipStream_t) { return hipErrorNoDevice; }
size_t gemm_t_workspace_bytes(int, int, int, const DeviceInfo&) { return 0; }
uint16_t* gemm_t_padded(int, void*) { return nullptr; }
hipError_t launch_gemm_t(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int, void*,
                         const DeviceInfo&, hipStream_t) { return hipErrorNoDevice; }
bool gemm_t_skinny_fits(int, int, int, int, const DeviceInfo&) { return false; }
size_t gemm_t_skinny_workspace_bytes(int, int, int, int, const DeviceInfo&) { return 0; }
hipError_t launch_gemm_t_skinny(const uint16_t*, const uint32_t*, const uint16_t*, uint16_t*, int, int, int, int, void*,
                                const DeviceInfo&, hipStream_t) { return hipErrorNoDevice; }
bool swiglu_backward_skinny_fits(int, int, int, int, const DeviceInfo&) { return false; }
hipError_t launch_swiglu_backward_skinny(const uint16_t*, const uint16_t*, uint16_t*, const uint32_t*, const uint16_t*,
                                         uint16_t*, int, int, int, int, void*, const DeviceInfo&, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_swiglu_grad(const uint16_t*, const uint16_t*, uint16_t*, uint16_t*, int, int, hipStream_t) {
  return hipErrorNoDevice;
}
size_t dscales_workspace_bytes(int, int, int, int, const DeviceInfo&) { return 0; }
hipError_t launch_dscales(const uint16_t*, const uint16_t*, const uint32_t*, float*, int, int, int, int, void*,
                          const DeviceInfo&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace w4a16
