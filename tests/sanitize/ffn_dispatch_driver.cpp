// ffn_dispatch_driver.cpp -- the C ABI of the feed-forward block's operators past its refusals:
// which launcher each call reaches, with which operands, and which calls stop at the workspace
// or at operands that share memory (a stand-in device and recording launchers, no GPU), under
// AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/w4a16.h"
#include "recording_launchers.hpp"

static int g_checks = 0, g_fail = 0;
static void expect(bool ok, const char* what, int line) {
  ++g_checks;
  if (!ok) {
    ++g_fail;
    std::fprintf(stderr, "FAILED line %d: %s\n", line, what);
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)

// Operands 16 MB apart, never dereferenced; `extra` bytes in.
template <typename T> static T* at(int place, int64_t extra = 0) {
  return reinterpret_cast<T*>((uintptr_t)((int64_t)(place + 1) * (16 << 20) + extra));
}

static std::string run;   // the launches of the last call
static w4a16_status ran(w4a16_status s) {
  run.clear();
  for (const std::string& l : g_rec.launches) run += (run.empty() ? "" : " ") + l;
  g_rec.launches.clear();
  return s;
}

static const uint16_t* const x = at<const uint16_t>(0);
static const uint32_t* const p = at<const uint32_t>(1);
static const uint16_t* const s = at<const uint16_t>(2);
static const uint16_t* const dy = at<const uint16_t>(3);
static const uint16_t* const z = at<const uint16_t>(4);
static uint16_t* const y = at<uint16_t>(5);
static uint16_t* const dz = at<uint16_t>(6);
static float* const f = at<float>(7);
static void* const w = at<void>(8);
constexpr size_t kRoom = 4 << 20;

static w4a16_status swiglu(const uint16_t* x_, uint16_t* y_, uint16_t* z_, int64_t m, int64_t n, int64_t k, void* w_ = w,
                           size_t room = kRoom) {
  return ran(w4a16_gemm_swiglu(x_, p, s, y_, z_, m, n, k, 32, w_, room, nullptr));
}
static w4a16_status t(const uint16_t* d, uint16_t* y_, int64_t m, int64_t n, int64_t k, void* w_ = w, size_t room = kRoom) {
  return ran(w4a16_gemm_t(d, p, s, y_, m, n, k, 32, w_, room, nullptr));
}
static w4a16_status back(const uint16_t* dy_, const uint16_t* z_, uint16_t* dz_, uint16_t* dx, int64_t m, int64_t n,
                         int64_t k, void* w_ = w, size_t room = kRoom) {
  return ran(w4a16_gemm_swiglu_backward(dy_, z_, p, s, dz_, dx, m, n, k, 32, w_, room, nullptr));
}
static w4a16_status scales(const uint16_t* d, const uint16_t* x_, float* o, int64_t m, int64_t n, int64_t k, void* w_ = w,
                           size_t room = kRoom) {
  return ran(w4a16_gemm_dscales(d, x_, p, o, m, n, k, 32, w_, room, nullptr));
}

static void dispatch() {
  // which launcher
  EXPECT(swiglu(x, y, nullptr, 3, 64, 128) == W4A16_OK && run == "gemv");
  EXPECT(swiglu(x, y, dz, 3, 64, 128) == W4A16_OK && run == "swiglu_skinny_keep");
  EXPECT(swiglu(x, y, dz, 32, 64, 128) == W4A16_OK && run == "swiglu_skinny_keep");
  EXPECT(swiglu(x, y, dz, 33, 64, 128) == W4A16_OK && run == "gemm_swiglu" && !g_rec.workspace);
  EXPECT(swiglu(x, y, dz, 20, 8192, 4096) == W4A16_OK && run == "gemm_swiglu");            // 32 MB of weights
  EXPECT(swiglu(x, y, dz, 3, 64, 0) == W4A16_OK && run == "zero_fill zero_fill");
  EXPECT(t(dy, y, 32, 63, 128) == W4A16_OK && run == "gemm_t_skinny" && g_rec.left == dy);
  EXPECT(t(dy, y, 33, 63, 128) == W4A16_OK && run == "gemm_t" && g_rec.left == dy);
  EXPECT(t(dy, y, 33, 0, 128) == W4A16_OK && run == "zero_fill");
  EXPECT(back(dy, z, dz, y, 8, 64, 128) == W4A16_OK && run == "swiglu_grad gemm_t_skinny" && !g_rec.padded &&
         g_rec.left == dz);
  g_ans.grad_fits = true;
  EXPECT(back(dy, z, dz, y, 8, 64, 128) == W4A16_OK && run == "swiglu_backward_skinny" && g_rec.left == dy);
  EXPECT(back(dy, z, dz, y, 8, 63, 128) == W4A16_OK && run == "swiglu_grad gemm_t_skinny");  // rows of 126
  g_ans.grad_fits = false;
  EXPECT(back(dy, z, dz, y, 40, 64, 128) == W4A16_OK && run == "swiglu_grad gemm_t" && !g_rec.padded &&
         g_rec.left == dz);
  g_ans.workspace = kRoom;
  EXPECT(back(dy, z, dz, y, 40, 63, 128) == W4A16_OK && run == "swiglu_grad gemm_t" && g_rec.left == nullptr &&
         g_rec.padded == at<void>(8, 16384) && g_rec.workspace == w);
  g_ans.workspace = 0;
  EXPECT(back(dy, z, dz, y, 8, 0, 128) == W4A16_OK && run == "zero_fill");
  EXPECT(back(dy, z, dz, nullptr, 8, 64, 0) == W4A16_OK && run == "swiglu_grad");
  EXPECT(scales(dy, x, f, 8, 64, 128) == W4A16_OK && run == "dscales");
  EXPECT(scales(dy, x, f, 0, 64, 128) == W4A16_OK && run == "zero_fill");

  // a workspace that is missing or too small
  g_ans.workspace = kRoom;
  EXPECT(swiglu(x, y, dz, 40, 64, 128, nullptr, kRoom) == W4A16_ERR_WORKSPACE && run.empty());
  EXPECT(swiglu(x, y, dz, 40, 64, 128, w, kRoom - 1) == W4A16_ERR_WORKSPACE && run.empty());
  EXPECT(swiglu(x, y, dz, 40, 64, 128) == W4A16_OK && g_rec.workspace == w);
  EXPECT(swiglu(x, y, dz, 16, 64, 128, nullptr, 0) == W4A16_OK && run == "swiglu_skinny_keep");   // needs none
  EXPECT(t(dy, y, 8, 64, 128, w, 0) == W4A16_ERR_WORKSPACE && run.empty());
  EXPECT(t(dy, y, 8, 0, 128, nullptr, 0) == W4A16_OK && run == "zero_fill");
  EXPECT(back(dy, z, dz, y, 8, 64, 128, nullptr, 0) == W4A16_ERR_WORKSPACE && run.empty());
  EXPECT(back(dy, z, dz, nullptr, 8, 64, 0, nullptr, 0) == W4A16_OK && run == "swiglu_grad");     // needs none
  EXPECT(scales(dy, x, f, 8, 64, 128, nullptr, 0) == W4A16_ERR_WORKSPACE && run.empty());
  g_ans.workspace = 0;
}

// m rows of c fp16 columns, in bytes
static int64_t rows(int64_t m, int64_t c) { return 2 * m * c; }

static void shared_memory() {
  const w4a16_status no = W4A16_ERR_OVERLAP;
  for (int64_t m : {3, 16, 40}) {
    // n == k == 64: an output as large as an input, whole, in its last 16 bytes and just behind it
    const int64_t n = 64, k = 64, last = rows(m, 64) - 16, past = rows(m, 64);
    uint16_t* const over = const_cast<uint16_t*>(x);
    EXPECT(swiglu(x, over, nullptr, m, n, k) == no && run.empty());
    EXPECT(swiglu(x, over + last / 2, nullptr, m, n, k) == no && run.empty());
    EXPECT(swiglu(x, over + past / 2, nullptr, m, n, k) == W4A16_OK && !run.empty());
    EXPECT(swiglu(x, over - last / 2, nullptr, m, n, k) == no && run.empty());
    EXPECT(swiglu(x, over - past / 2, nullptr, m, n, k) == W4A16_OK);
    EXPECT(swiglu(x, y, y, m, n, k) == no && swiglu(x, y, y + past / 2, m, n, k) == W4A16_OK);
    EXPECT(swiglu(x, y + past, y, m, n, k) == W4A16_OK && swiglu(x, y + past - 8, y, m, n, k) == no);
    EXPECT(swiglu(x, y, over + last / 2, m, n, k) == no);
    EXPECT(swiglu(x, reinterpret_cast<uint16_t*>(const_cast<uint32_t*>(p)), nullptr, m, n, k) == no);
    EXPECT(swiglu(x, const_cast<uint16_t*>(s), nullptr, m, n, k) == no);

    uint16_t* const d = const_cast<uint16_t*>(dy);
    EXPECT(t(dy, d, m, n, k) == no && t(dy, d + last / 2, m, n, k) == no && t(dy, d - last / 2, m, n, k) == no);
    EXPECT(t(dy, d + past / 2, m, n, k) == W4A16_OK && t(dy, d - past / 2, m, n, k) == W4A16_OK);

    // the pairs' gradient over the pairs, whole and in part; dx over each input and over dgate_up
    uint16_t* const pairs = const_cast<uint16_t*>(z);
    const int64_t two = rows(m, 128);
    EXPECT(back(dy, z, pairs, y, m, n, k) == no && run.empty());
    EXPECT(back(dy, z, pairs + (two - 16) / 2, y, m, n, k) == no && run.empty());
    EXPECT(back(dy, z, pairs - (two - 16) / 2, y, m, n, k) == no);
    EXPECT(back(dy, z, pairs + two / 2, y, m, n, k) == W4A16_OK && back(dy, z, pairs - two / 2, y, m, n, k) == W4A16_OK);
    EXPECT(back(dy, z, d, y, m, n, k) == no && back(dy, z, dz, d, m, n, k) == no);
    EXPECT(back(dy, z, dz, pairs + (two - 16) / 2, m, n, k) == no);
    EXPECT(back(dy, z, dz, dz, m, n, k) == no && back(dy, z, dz, dz + two / 2, m, n, k) == W4A16_OK);
    EXPECT(back(dy, z, pairs, nullptr, m, n, 0) == no);          // k == 0: only the pairs' gradient

    EXPECT(scales(dy, x, reinterpret_cast<float*>(d), m, n, k) == no);
    EXPECT(scales(dy, x, reinterpret_cast<float*>(over), m, n, k) == no);
    EXPECT(scales(x, x, f, m, n, k) == W4A16_OK);                // inputs may share
  }
  // the workspace, in the bytes that the call needs
  g_ans.workspace = 1 << 20;
  EXPECT(t(dy, at<uint16_t>(8, (1 << 20) - 16), 40, 64, 64) == no);
  EXPECT(t(dy, at<uint16_t>(8, 1 << 20), 40, 64, 64) == W4A16_OK);
  EXPECT(t(at<uint16_t>(8, 16), y, 40, 64, 64) == no);
  EXPECT(swiglu(x, y, at<uint16_t>(8), 40, 64, 64) == no);
  EXPECT(back(dy, z, at<uint16_t>(8), y, 40, 64, 64) == no);
  EXPECT(scales(dy, x, at<float>(8), 40, 64, 64) == no);
  g_ans.workspace = 0;
  EXPECT(t(dy, at<uint16_t>(8), 40, 64, 64) == W4A16_OK);        // none needed: the pointer is not looked at
  EXPECT(std::string(w4a16_status_str(W4A16_ERR_OVERLAP)).find("OVERLAP") != std::string::npos);
}

int main() {
  dispatch();
  shared_memory();
  if (g_fail) {
    std::fprintf(stderr, "ffn dispatch driver: %d of %d checks failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("ffn dispatch driver: ok (%d checks)\n", g_checks);
  return 0;
}
