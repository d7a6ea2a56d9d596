// fake_hip.cpp -- the few HIP runtime functions that the C ABI's host code calls, as a host
// without a GPU can serve them: one device of 256 CUs with 160 KB of LDS.  With it and the
// recording launchers, dispatch runs to its end on the CPU.
#include <hip/hip_runtime_api.h>

extern "C" {

hipError_t hipGetDevice(int* device) {
  *device = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t attr, int) {
  if (attr == hipDeviceAttributeMultiprocessorCount) *value = 256;
  else if (attr == hipDeviceAttributeMaxSharedMemoryPerBlock) *value = 160 * 1024;
  else return hipErrorInvalidValue;
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipErrorNoDevice; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipErrorNoDevice; }

}
