// checks.hpp -- host-side argument checks shared by the C ABI's source files.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/w4a16.h"

namespace w4a16 {

inline bool valid_group(int32_t g) { return g == 32 || g == 128; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Activations, packed weights and scales are addressed with 32-bit buffer
// offsets below 2^31 (an offset of 2^31 marks an out-of-range load).
constexpr int64_t kMaxBufferBytes = (int64_t)1 << 31;
constexpr int64_t kMaxDim = (int64_t)1 << 30;
// W4A16_OK, an error, or -1 for a valid call with nothing to do.
inline int common_dense_checks(const uint16_t* x, const uint32_t* packed, const uint16_t* scales, uint16_t* y,
                               int64_t m, int64_t n, int64_t k, int32_t group) {
  if (!valid_group(group)) return W4A16_ERR_GROUP;
  if (m < 0 || n < 0 || k < 0 || k % group) return W4A16_ERR_SHAPE;
  if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return W4A16_ERR_SHAPE;
  if (m == 0 || n == 0) return -1;  // no-op
  if (!y) return W4A16_ERR_NULL;
  if (k > 0 && (!x || !packed || !scales)) return W4A16_ERR_NULL;
  if (!aligned(y, 16) || (k > 0 && (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 2))))
    return W4A16_ERR_ALIGN;
  if (n * (k / 2) >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  if (2 * m * k >= kMaxBufferBytes || 2 * m * n >= kMaxBufferBytes) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// One operand's bytes (none: a pointer that is not looked at).
struct Span {
  const void* p;
  int64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes);
}

// Whether what a call writes shares memory with what it reads, or two of the things it writes
// with each other: workgroups read an input while others already store, so the results would
// depend on timing.
inline bool outputs_overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    for (auto b = o + 1; b != outputs.end(); ++b)
      if (overlap(*o, *b)) return true;
    for (const Span& i : inputs)
      if (overlap(*o, i)) return true;
  }
  return false;
}

inline w4a16_status status_of(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }
inline w4a16_status as_status(int s) { return static_cast<w4a16_status>(s); }

}  // namespace w4a16
