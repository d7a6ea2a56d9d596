// block_dispatch_driver.cpp -- the C ABI of the linear layer, its backward pass, the router's choice and the few-token
// feed-forward past their refusals: which launchers each call reaches and with which operands, sizes past 32
// bits, workspaces, operands that share memory (a stand-in device and recording launchers, no GPU).
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/w4a16.h"
#include "block_recording_launchers.hpp"

static int g_checks = 0, g_fail = 0;
static void expect(bool ok, const char* what, int line) {
  ++g_checks;
  if (!ok) {
    ++g_fail;
    std::fprintf(stderr, "FAILED line %d: %s\n", line, what);
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)

// Operands 16 GB apart, never dereferenced; `extra` bytes in.
template <typename T> static T* at(int place, int64_t extra = 0) {
  return reinterpret_cast<T*>((uintptr_t)(((int64_t)(place + 1) << 34) + extra));
}

static std::string run;   // the launches of the last call
static w4a16_status ran(w4a16_status s) {
  run.clear();
  for (const std::string& l : g_rec.launches) run += (run.empty() ? "" : " ") + l;
  g_rec.launches.clear();
  return s;
}

static const w4a16_status kOk = W4A16_OK, kNo = W4A16_ERR_OVERLAP, kRoomErr = W4A16_ERR_WORKSPACE;
static const uint16_t* const x = at<const uint16_t>(0);
static const uint32_t* const p = at<const uint32_t>(1);
static const uint16_t* const s = at<const uint16_t>(2);
static const uint16_t* const b = at<const uint16_t>(3);
static const uint16_t* const r = at<const uint16_t>(4);
static uint16_t* const y = at<uint16_t>(5);
static uint16_t* const z = at<uint16_t>(6);
static uint16_t* const dz = at<uint16_t>(7);
static float* const f = at<float>(8);
static void* const w = at<void>(9);
constexpr size_t kRoom = 4 << 20;

struct Linear {
  const uint16_t *x_ = x, *b_ = b, *r_ = r;
  uint16_t *y_ = y, *z_ = z;
  void* w_ = w;
  size_t room = kRoom;
  w4a16_status operator()(int64_t m, int64_t n, int64_t k) const {
    return ran(w4a16_linear(x_, p, s, b_, r_, y_, z_, m, n, k, 32, W4A16_ACT_SILU, w_, room, nullptr));
  }
};
struct Back {
  const uint16_t *dy_ = x, *z_ = z;
  uint16_t *dz_ = dz, *dx_ = y;
  float* f_ = f;
  int act = W4A16_ACT_GELU;
  void* w_ = w;
  size_t room = kRoom;
  w4a16_status operator()(int64_t m, int64_t n, int64_t k) const {
    return ran(w4a16_linear_backward(dy_, z_, p, s, dz_, f_, dx_, m, n, k, 32, act, w_, room, nullptr));
  }
};
static Linear linear(const uint16_t* x_, uint16_t* y_, uint16_t* z_, const uint16_t* r_) {
  Linear l;
  l.x_ = x_; l.y_ = y_; l.z_ = z_; l.r_ = r_;
  return l;
}
static Back back(const uint16_t* dy_, const uint16_t* z_, uint16_t* dz_, uint16_t* dx_, float* f_) {
  Back c;
  c.dy_ = dy_; c.z_ = z_; c.dz_ = dz_; c.dx_ = dx_; c.f_ = f_;
  return c;
}

static void linear_dispatch() {
  Linear l;
  EXPECT(l(1, 64, 128) == kOk && run == "gemv");
  EXPECT(l(2, 64, 128) == kOk && run == "gemv_mfma" && l(4, 64, 128) == kOk && run == "gemv_mfma");
  EXPECT(l(5, 64, 128) == kOk && run == "skinny" && l(32, 64, 128) == kOk && run == "skinny");
  EXPECT(l(33, 64, 128) == kOk && run == "tiles" && !g_rec.workspace);
  EXPECT(l(16, 16384, 4096) == kOk && run == "skinny" && l(17, 16384, 4096) == kOk && run == "tiles");   // 32 MB
  g_ans.one_row = g_ans.four_rows = false;
  EXPECT(l(1, 64, 128) == kOk && run == "skinny" && l(3, 64, 128) == kOk && run == "skinny");
  g_ans.skinny_fits = false;
  EXPECT(l(1, 64, 128) == kOk && run == "tiles");
  g_ans = {};
  EXPECT(l(0, 64, 128) == kOk && run.empty() && l(3, 0, 128) == kOk && run.empty());
  EXPECT(l(3, 64, 0) == W4A16_ERR_SHAPE && run.empty());
  g_ans.product = kRoom;
  EXPECT(l(33, 64, 128) == kOk && g_rec.workspace == w);
  EXPECT(w4a16_linear_workspace_bytes(33, 64, 128, 32) == kRoom && w4a16_linear_workspace_bytes(32, 64, 128, 32) == 0);
  l.room = kRoom - 1;
  EXPECT(l(33, 64, 128) == kRoomErr && run.empty() && l(32, 64, 128) == kOk);
  l.w_ = nullptr; l.room = kRoom;
  EXPECT(l(33, 64, 128) == kRoomErr && l(1, 64, 128) == kOk && l(4, 64, 128) == kOk);
  g_ans = {};
}

static void backward_dispatch() {
  const Back c;
  Back plain;      // no activation
  plain.act = W4A16_ACT_NONE; plain.z_ = nullptr; plain.dz_ = nullptr;
  Back bare = plain;
  bare.f_ = nullptr;
  EXPECT(c(8, 64, 128) == kOk && run == "grad gemm_t_skinny" && g_rec.left == dz && g_rec.pre == z && !g_rec.padded);
  EXPECT(plain(8, 64, 128) == kOk && run == "grad gemm_t_skinny" && g_rec.left == x && !g_rec.pre);
  EXPECT(bare(8, 64, 128) == kOk && run == "gemm_t_skinny" && g_rec.left == x);
  g_ans.grad_fits = true;
  EXPECT(c(32, 63, 128) == kOk && run == "grad_in_skinny" && g_rec.left == x && !g_rec.workspace);
  EXPECT(plain(8, 64, 128) == kOk && run == "grad_in_skinny" && bare(8, 64, 128) == kOk && run == "gemm_t_skinny");
  EXPECT(c(33, 64, 128) == kOk && run == "grad gemm_t");                      // past the weight-streaming kernel
  EXPECT(c(8, 64, 0) == kOk && run == "grad");                                // no product
  g_ans = {};
  EXPECT(c(40, 64, 128) == kOk && run == "grad gemm_t" && g_rec.left == dz && !g_rec.padded);
  EXPECT(c(0, 64, 128) == kOk && run == "zero_fill" && c(0, 0, 128) == kOk && run.empty());
  EXPECT(c(8, 0, 128) == kOk && run == "zero_fill" && c(8, 0, 0) == kOk && run.empty());
  EXPECT(bare(0, 64, 128) == kOk && run.empty());

  // the product's workspace, then the column sums'
  g_ans.product = 100000;
  g_ans.sums = 5000;
  EXPECT(w4a16_linear_backward_workspace_bytes(40, 63, 128, 32) == 100096 + 5000);
  EXPECT(c(40, 63, 128) == kOk && run == "grad gemm_t" && g_rec.left == nullptr && g_rec.padded == at<void>(9, 16384) &&
         g_rec.workspace == w && g_rec.counters == w && g_rec.partials == at<void>(9, 100096));
  EXPECT(c(8, 63, 128) == kOk && run == "grad gemm_t_skinny" && g_rec.left == dz && !g_rec.padded);
  Back tight = c;
  tight.room = 105095;
  EXPECT(tight(40, 63, 128) == kRoomErr && run.empty());
  tight.room = 100000;
  tight.f_ = nullptr;
  EXPECT(tight(40, 63, 128) == kOk && run == "grad gemm_t" && !g_rec.counters && !g_rec.partials);
  tight.room = 99999;
  EXPECT(tight(40, 63, 128) == kRoomErr);
  g_ans.product = 0;
  EXPECT(c(40, 64, 128) == kOk && g_rec.counters == w && g_rec.partials == at<void>(9, 16384) && !g_rec.workspace);
  EXPECT(c(40, 64, 0) == kOk && run == "grad" && g_rec.partials == at<void>(9, 16384));
  EXPECT(w4a16_linear_backward_workspace_bytes(40, 64, 0, 32) == 16384 + 5000);
  g_ans = {};
}

static void linear_shared_memory() {
  uint16_t *const ox = const_cast<uint16_t*>(x), *const orr = const_cast<uint16_t*>(r);
  for (int64_t m : {1, 3, 16, 40}) {
    const int64_t last = (2 * m * 64 - 16) / 2, past = m * 64;      // elements
    EXPECT(linear(x, ox, nullptr, r)(m, 64, 64) == kNo && run.empty());
    EXPECT(linear(x, ox + last, nullptr, r)(m, 64, 64) == kNo && linear(x, ox + past, nullptr, r)(m, 64, 64) == kOk);
    EXPECT(linear(x, orr, z, r)(m, 64, 64) == kOk);                                  // into the residual
    EXPECT(linear(x, orr + past, z, r)(m, 64, 64) == kOk && linear(x, orr - past, z, r)(m, 64, 64) == kOk);
    if (last > 0) EXPECT(linear(x, orr + last, z, r)(m, 64, 64) == kNo && linear(x, orr - last, z, r)(m, 64, 64) == kNo);
    EXPECT(linear(x, y, y, r)(m, 64, 64) == kNo && linear(x, y, y + past, r)(m, 64, 64) == kOk);
    EXPECT(linear(x, y, orr, r)(m, 64, 64) == kNo && linear(x, y, ox, r)(m, 64, 64) == kNo);
    EXPECT(linear(x, y, const_cast<uint16_t*>(b), r)(m, 64, 64) == kNo);
    EXPECT(linear(x, const_cast<uint16_t*>(s), nullptr, r)(m, 64, 64) == kNo);
    EXPECT(linear(x, y, z, x)(m, 64, 64) == kOk);                                    // inputs may share

    uint16_t* const oz = z;
    EXPECT(back(x, z, oz, y, f)(m, 64, 64) == kNo && back(x, z, oz + past, y, f)(m, 64, 64) == kOk);
    EXPECT(back(x, z, ox, y, f)(m, 64, 64) == kNo && back(x, z, dz, ox, f)(m, 64, 64) == kNo);
    EXPECT(back(x, z, dz, dz, f)(m, 64, 64) == kNo && back(x, z, dz, dz + past, f)(m, 64, 64) == kOk);
    EXPECT(back(x, z, dz, oz + last, f)(m, 64, 64) == kNo);
    EXPECT(back(x, z, dz, y, at<float>(7))(m, 64, 64) == kNo && back(x, z, dz, y, at<float>(5))(m, 64, 64) == kNo);
    EXPECT(back(x, z, dz, y, at<float>(1))(m, 64, 64) == kNo && back(x, x, dz, y, f)(m, 64, 64) == kOk);
  }
  g_ans.product = kRoom;
  EXPECT(linear(x, at<uint16_t>(9, kRoom - 16), z, r)(40, 64, 64) == kNo && linear(x, at<uint16_t>(9, kRoom), z, r)(40, 64, 64) == kOk);
  EXPECT(back(x, z, at<uint16_t>(9, kRoom - 16), y, f)(40, 64, 64) == kNo);
  g_ans = {};
}

// moe: places 0 x, 1 ids, 2 weights, 3 and 4 gate/up, 5 and 6 down, 7 residual, 8 y, 9 workspace
static w4a16_status ffn(const uint16_t* r_, uint16_t* y_, int64_t t, int32_t topk, int32_t e, int64_t h, int64_t i,
                        size_t room = kRoom) {
  return ran(w4a16_moe_ffn(at<const uint16_t>(0), at<const int32_t>(1), at<const float>(2), at<const uint32_t>(3),
                           at<const uint16_t>(4), at<const uint32_t>(5), at<const uint16_t>(6), r_, y_, t, topk, e, h, i, 32,
                           w, room, nullptr));
}

static void moe() {
  const uint16_t* const res = at<const uint16_t>(7);
  uint16_t* const out = at<uint16_t>(8);
  g_ans.moe = kRoom;
  EXPECT(ffn(res, out, 4, 2, 8, 256, 128) == kOk && run == "moe_ffn" && g_rec.workspace == w);
  EXPECT(ffn(nullptr, out, 64, 8, 8, 256, 128) == kOk && ffn(res, out, 64, 9, 8, 256, 128) == W4A16_ERR_SHAPE);
  EXPECT(ffn(res, out, 65, 1, 8, 256, 128) == W4A16_ERR_SHAPE && ffn(res, out, 4, 2, 0, 256, 128) == W4A16_ERR_SHAPE);
  EXPECT(ffn(res, out, 0, 2, 8, 256, 128) == kOk && run.empty() && ffn(res, out, 4, 2, 8, 0, 128) == kOk && run.empty());
  EXPECT(ffn(res, out, 4, 2, 8, 256, 128, kRoom - 1) == kRoomErr && run.empty());
  EXPECT(ffn(res, const_cast<uint16_t*>(res), 4, 2, 8, 256, 128) == kOk);                       // into the residual
  EXPECT(ffn(res, const_cast<uint16_t*>(res) + 8, 4, 2, 8, 256, 128) == kNo && run.empty());
  EXPECT(ffn(res, at<uint16_t>(0), 4, 2, 8, 256, 128) == kNo && ffn(res, at<uint16_t>(9, 16), 4, 2, 8, 256, 128) == kNo);
  EXPECT(ffn(res, at<uint16_t>(9, kRoom), 4, 2, 8, 256, 128) == kOk);
  // banks past 32 bits: 4096 experts of 2 x 1024 x 1024 (4 GiB of words) and 128 MiB of scales
  const int64_t words = (int64_t)4096 * 1024 * 1024;
  EXPECT(ffn(res, at<uint16_t>(3, words - 16), 4, 2, 4096, 1024, 1024) == kNo);
  EXPECT(ffn(res, at<uint16_t>(3, words), 4, 2, 4096, 1024, 1024) == kOk);
  EXPECT(ffn(res, at<uint16_t>(5, words / 2 - 16), 4, 2, 4096, 1024, 1024) == kNo);
  EXPECT(ffn(res, at<uint16_t>(5, words / 2), 4, 2, 4096, 1024, 1024) == kOk);
  EXPECT(ffn(res, at<uint16_t>(4, words / 8 - 16), 4, 2, 4096, 1024, 1024) == kNo);
  EXPECT(ffn(res, at<uint16_t>(4, words / 8), 4, 2, 4096, 1024, 1024) == kOk);
  EXPECT(ffn(res, out, 4, 2, 8, 65536, 32768) == W4A16_ERR_SHAPE);                              // an expert of 2 GiB
  EXPECT(ffn(res, out, 4, 2, 8, 1 << 24, 32) == kOk && ffn(res, out, 4, 2, 8, (1 << 24) + 32, 32) == W4A16_ERR_SHAPE);
  g_ans = {};

  int32_t* const ids = at<int32_t>(1);
  float* const wt = at<float>(2);
  const void* const l = at<const void>(0);
  auto topk = [&](const void* l_, int32_t* i_, float* w_, int64_t t, int32_t e, int32_t k, int32_t type) {
    return ran(w4a16_moe_topk(l_, type, i_, w_, t, e, k, 1, nullptr));
  };
  EXPECT(topk(l, ids, wt, 10, 64, 4, W4A16_F32) == kOk && run == "topk32" && topk(l, ids, wt, 10, 64, 4, W4A16_F16) == kOk &&
         run == "topk16");
  EXPECT(topk(l, ids, wt, 0, 64, 4, W4A16_F32) == kOk && run.empty() && topk(l, ids, wt, 10, 64, 4, 2) == W4A16_ERR_RANGE);
  EXPECT(topk(l, ids, at<float>(1, 156), 10, 64, 4, W4A16_F32) == kNo && topk(l, ids, at<float>(1, 160), 10, 64, 4, W4A16_F32) == kOk);
  // 8 Mi tokens of 1024 experts: 32 GiB of logits are past the next operands
  EXPECT(topk(l, ids, wt, 1 << 23, 1024, 4, W4A16_F32) == kNo && topk(l, at<int32_t>(7), at<float>(8), 1 << 23, 1024, 4, W4A16_F32) == kOk);
  EXPECT(topk(l, at<int32_t>(7), at<float>(8), (1 << 26) - 1, 8, 4, W4A16_F16) == kOk && topk(l, ids, wt, 1 << 26, 8, 4, W4A16_F16) == W4A16_ERR_SHAPE);
  auto grad = [&](float* d, const void* l_, void* o, int32_t renorm) {
    return ran(w4a16_moe_topk_backward(d, l_, W4A16_F32, ids, wt, o, 10, 64, 4, renorm, nullptr));
  };
  EXPECT(grad(at<float>(3), l, at<void>(4), 0) == kOk && run == "topk_backward32" && grad(at<float>(3), nullptr, at<void>(4), 1) == kOk);
  EXPECT(grad(at<float>(3), nullptr, at<void>(4), 0) == W4A16_ERR_NULL && grad(at<float>(3), l, at<void>(0, 2544), 0) == kNo);
  EXPECT(grad(at<float>(3), l, at<void>(0), 1) == kOk);                 // renormalised: the logits are not read
  EXPECT(grad(at<float>(3), l, at<void>(3), 1) == kNo && grad(at<float>(3), l, at<void>(2), 1) == kNo);
}

int main() {
  linear_dispatch();
  backward_dispatch();
  linear_shared_memory();
  moe();
  if (g_fail) {
    std::fprintf(stderr, "block dispatch driver: %d of %d checks failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("block dispatch driver: ok (%d checks)\n", g_checks);
  return 0;
}
