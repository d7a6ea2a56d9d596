// dispatch.hpp -- which kernels serve a product, and the checks of the products over n: shared by the
// C ABI's source files of the feed-forward block and of the linear layer.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "../../include/w4a16.h"
#include "checks.hpp"
#include "kernels.hpp"

namespace w4a16 {

// Up to 16 rows the gate/up product is a weight stream: the weight-streaming kernel.  17 to 32
// rows are two passes of it, side by side in one launch, or the tiles, whose fixed costs are
// larger.  Weight-streaming against tiles, products kept, device time in us at group 128 (at group 32,
// where only the first keeps products of exact weights): 16 rows 2048 -> 512 (5.3 / 13.1), 16 rows 5120 -> 17408
// (89 MB of weights) 37.8 / 43.8 (48.6 / 55.1), 1 row 36.2 / 42.7 (44.9 / 51.5); 24 rows 2048 -> 1024
// (2 MB) 5.6 / 12.9 (5.7 / 14.2), 32 rows 4096 -> 2048 (8 MB) 13.5 / 16.8 (13.9 / 18.0), 32 rows 5120 ->
// 17408 61.1 / 45.6 (70.6 / 55.1).
constexpr int64_t kSkinnyRows = 32;
constexpr int64_t kSkinnyTwicePassBytes = (int64_t)32 << 20;

inline bool swiglu_skinny(int64_t m, int64_t n2, int64_t k, const DeviceInfo& dev) {
  return m <= kSkinnyRows && (m <= 16 || n2 * (k / 2) < kSkinnyTwicePassBytes) &&
         gemm_skinny_fits((int)(m < 16 ? m : 16), (int)n2, (int)k, dev);
}

// The product over n of checked arguments (m, n, k > 0): up to kSkinnyTRows rows on the
// weight-streaming kernel, beyond on the tiles.
inline bool t_skinny(int64_t m, int64_t n, int64_t k, int32_t group, const DeviceInfo& dev) {
  return m <= kSkinnyTRows && gemm_t_skinny_fits((int)m, (int)n, (int)k, group, dev);
}

inline size_t t_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t group, const DeviceInfo& dev) {
  return t_skinny(m, n, k, group, dev)
             ? gemm_t_skinny_workspace_bytes((int)m, (int)n, (int)k, group, dev)
             : gemm_t_workspace_bytes((int)m, (int)n, (int)k, dev);
}

inline hipError_t launch_t(const uint16_t* d, const uint32_t* packed, const uint16_t* scales, uint16_t* y, int64_t m, int64_t n,
                    int64_t k, int32_t group, void* workspace, const DeviceInfo& dev, hipStream_t st) {
  auto launch = t_skinny(m, n, k, group, dev) ? launch_gemm_t_skinny : launch_gemm_t;
  return launch(d, packed, scales, y, (int)m, (int)n, (int)k, group, workspace, dev, st);
}

// The checks of the products over n (m rows of d, weights [n, k]): W4A16_OK, an
// error, or -1 when there is no output.  n may be 0 (an empty sum).
inline int transposed_checks(const uint16_t* d, const uint32_t* packed, const uint16_t* scales, uint16_t* y, int64_t m,
                      int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group)) return W4A16_ERR_GROUP;
  if (m < 0 || n < 0 || k < 0 || k % group) return W4A16_ERR_SHAPE;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return W4A16_ERR_SHAPE;
  if (m == 0 || k == 0) return -1;
  if (!y) return W4A16_ERR_NULL;
  if (n > 0 && (!d || !packed || !scales)) return W4A16_ERR_NULL;
  if (!aligned(y, 16) || (n > 0 && (!aligned(d, 16) || !aligned(packed, 16) || !aligned(scales, 2))))
    return W4A16_ERR_ALIGN;
  if (n * (k / 2) >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  const int64_t n8 = (n + 7) / 8 * 8;   // rows of d are padded to 8 elements where n is not a multiple
  if (2 * m * k >= kMaxBufferBytes || 2 * m * n8 >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

}  // namespace w4a16
