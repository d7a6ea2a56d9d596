// ffn_driver.cpp -- drives the C ABI's host code of the feed-forward block's
// operators (validation and dispatch, stand-in launchers, no GPU) under
// AddressSanitizer and UndefinedBehaviorSanitizer.  Exit status 0 and "ffn
// driver: ok" when every expectation holds.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "../../include/w4a16.h"

static int g_checks = 0, g_fail = 0;
static void expect(bool ok, const char* what, int line) {
  ++g_checks;
  if (!ok) {
    ++g_fail;
    std::fprintf(stderr, "FAILED line %d: %s\n", line, what);
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)

// A 16-byte aligned address (plus extra) that is never dereferenced.
template <typename T> static T* F(uintptr_t extra = 0) { return reinterpret_cast<T*>((uintptr_t)0x10000 + extra); }

int main() {
  const uint16_t* x = F<const uint16_t>();
  const uint32_t* p = F<const uint32_t>();
  const uint16_t* s = F<const uint16_t>();
  uint16_t* y = F<uint16_t>();
  uint16_t* z = F<uint16_t>();
  float* f = F<float>();
  void* w = F<void>();
  const int64_t lo = INT64_MIN, hi = INT64_MAX;

  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, 8, 64, 128, 64, w, 0, nullptr) == W4A16_ERR_GROUP);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, 8, 64, 100, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, lo, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, 8, lo, 128, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, 8, hi, 128, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, hi, hi, hi, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu(x, p, s, nullptr, z, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_swiglu(x, nullptr, s, y, z, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, F<uint16_t>(8), 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, 8, 64, 128, 32, F<void>(4), 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_swiglu(nullptr, nullptr, nullptr, nullptr, nullptr, 0, 64, 128, 32, nullptr, 0, nullptr) == W4A16_OK);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, 4, 1 << 28, 128, 128, w, 0, nullptr) == W4A16_ERR_SHAPE);   // 2 GiB of weights
  for (int64_t m : {1, 20, 600}) EXPECT(w4a16_gemm_swiglu(x, p, s, y, z, m, 64, 128, 32, w, 1 << 20, nullptr) == W4A16_ERR_HIP);
  EXPECT(w4a16_gemm_swiglu(x, p, s, y, nullptr, 3, 64, 0, 32, w, 0, nullptr) == W4A16_ERR_HIP);
  for (int64_t v : {lo, hi, (int64_t)-1, (int64_t)0, (int64_t)64}) {
    EXPECT(w4a16_gemm_swiglu_workspace_bytes(v, v, v, 32) == 0);
    EXPECT(w4a16_gemm_t_workspace_bytes(v, v, v, 32) == 0);
    EXPECT(w4a16_gemm_swiglu_backward_workspace_bytes(v, v, v, 32) == 0);
    EXPECT(w4a16_gemm_dscales_workspace_bytes(v, v, v, 32) == 0);
  }

  EXPECT(w4a16_gemm_t(x, p, s, y, 8, 64, 128, 16, w, 0, nullptr) == W4A16_ERR_GROUP);
  EXPECT(w4a16_gemm_t(x, p, s, y, 8, 64, 96, 128, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_t(x, p, s, y, lo, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_t(x, p, s, y, hi, hi, hi, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_t(x, p, s, y, 1 << 20, 1 << 10, 128, 128, w, 0, nullptr) == W4A16_ERR_SHAPE);     // d of 2 GiB
  EXPECT(w4a16_gemm_t(x, p, s, nullptr, 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_t(nullptr, p, s, y, 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_t(F<const uint16_t>(2), p, s, y, 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_t(x, p, s, y, 8, 64, 128, 128, F<void>(8), 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_t(nullptr, nullptr, nullptr, nullptr, 0, 64, 128, 128, nullptr, 0, nullptr) == W4A16_OK);
  EXPECT(w4a16_gemm_t(x, p, s, nullptr, 8, 64, 0, 128, nullptr, 0, nullptr) == W4A16_OK);
  EXPECT(w4a16_gemm_t(nullptr, nullptr, nullptr, y, 8, 0, 128, 128, nullptr, 0, nullptr) == W4A16_ERR_HIP);   // writes zeros
  EXPECT(w4a16_gemm_t(x, p, s, y, 8, 64, 128, 128, w, 1 << 20, nullptr) == W4A16_ERR_HIP);

  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, y, 8, 64, 128, 48, w, 0, nullptr) == W4A16_ERR_GROUP);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, y, 8, lo, 128, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, y, hi, hi, hi, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, y, 1 << 20, 512, 32, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_swiglu_backward(nullptr, z, p, s, z, y, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_swiglu_backward(x, nullptr, p, s, z, y, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, nullptr, y, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, nullptr, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_swiglu_backward(F<const uint16_t>(8), z, p, s, z, y, 8, 64, 128, 32, w, 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, y, 8, 64, 128, 32, F<void>(2), 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_swiglu_backward(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 64, 128, 32, nullptr, 0,
                                    nullptr) == W4A16_OK);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, p, s, z, y, 8, 64, 128, 32, w, 1 << 20, nullptr) == W4A16_ERR_HIP);
  EXPECT(w4a16_gemm_swiglu_backward(x, z, nullptr, nullptr, z, nullptr, 8, 64, 0, 32, nullptr, 0, nullptr) == W4A16_ERR_HIP);

  EXPECT(w4a16_gemm_dscales(x, x, p, f, 8, 64, 128, 0, w, 0, nullptr) == W4A16_ERR_GROUP);
  EXPECT(w4a16_gemm_dscales(x, x, p, f, 8, 64, 128 + 32, 128, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_dscales(x, x, p, f, lo, lo, lo, 128, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_dscales(x, x, p, f, hi, hi, hi, 32, w, 0, nullptr) == W4A16_ERR_SHAPE);
  EXPECT(w4a16_gemm_dscales(x, x, p, nullptr, 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_dscales(x, nullptr, p, f, 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_NULL);
  EXPECT(w4a16_gemm_dscales(x, x, p, F<float>(4), 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_dscales(x, F<const uint16_t>(8), p, f, 8, 64, 128, 128, w, 0, nullptr) == W4A16_ERR_ALIGN);
  EXPECT(w4a16_gemm_dscales(nullptr, nullptr, nullptr, nullptr, 8, 0, 128, 128, nullptr, 0, nullptr) == W4A16_OK);
  EXPECT(w4a16_gemm_dscales(nullptr, nullptr, nullptr, f, 0, 64, 128, 128, nullptr, 0, nullptr) == W4A16_ERR_HIP);
  EXPECT(w4a16_gemm_dscales(x, x, p, f, 8, 64, 128, 128, w, 1 << 20, nullptr) == W4A16_ERR_HIP);

  if (g_fail) {
    std::fprintf(stderr, "ffn driver: %d of %d checks failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("ffn driver: ok (%d checks)\n", g_checks);
  return 0;
}
