// linear_grad.hip -- gradient of the linear layer's epilogue on gfx950: dz = dy act'(z) in fp32, rounded
// once to fp16 (an output, and the fp16 operand of the product that follows), and the bias's
// gradient, the column sums of the unrounded dz in fp32.  (Few rows and short ranges: within the
// product itself, gemm_t_skinny.hip.)
//
// Bound by memory: 6 bytes per element.  A workgroup takes 128 columns of kRowsWG rows, sixteen
// threads of eight columns side by side, sixteen rows at a time; column sums meet in LDS, and the
// last workgroup of a column block to finish adds the row blocks' sums in order (deterministic, no
// second launch).
#include "arrive.hpp"
#include "device.hpp"
#include "kernels.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 128;                       // columns of a workgroup
constexpr int kRowLanes = 16;                    // rows at a time
constexpr int kRowsWG = 128;                     // rows of a workgroup, at most
constexpr int kLeastRows = 32, kManyWG = 256;    // ... and at least, unless there are this many workgroups
constexpr int kUnroll = 2;                       // rows of a thread loaded together

struct GradPlan {
  int col_blocks, row_blocks, rows;              // rows: of a workgroup
};
GradPlan grad_plan(int m, int n, bool bias) {
  GradPlan p;
  p.col_blocks = (n + kCols - 1) / kCols;
  // fewer rows per workgroup where there would be few workgroups (300 x 2001 7.6 against 11.4 us, 130 x 520 5.6 / 10.4)
  p.rows = kRowsWG;
  while (p.rows > kLeastRows && (int64_t)p.col_blocks * ((m + p.rows - 1) / p.rows) < kManyWG) p.rows /= 2;
  p.row_blocks = (m + p.rows - 1) / p.rows;
  // (a counter per column block, and 65535 row blocks in a grid: beyond, a workgroup takes more rows)
  const int most = bias && p.col_blocks > kCounters ? 1 : 65535;
  if (p.row_blocks > most) {
    p.rows = (m + most - 1) / most;
    p.row_blocks = (m + p.rows - 1) / p.rows;
  }
  return p;
}

// Eight elements of a row, from column c (c < N).  VEC: rows start on 16 bytes; else the dwords that hold them (buf
// ends with a whole dword), turned, with zeros past the row's end: as eight 2-byte accesses the 2048 x
// 17407 gradient takes 104 us instead of 69.
struct Eight {
  u32x4 v;
  uint32_t last;
};
template <bool VEC>
__device__ inline Eight load_eight(__amdgpu_buffer_rsrc_t buf, uint32_t at) {
  Eight e;
  if constexpr (VEC) {
    e.v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, kStream));
    e.last = 0;
  } else {
    const uint32_t from = at & ~3u;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.v[j] = __builtin_amdgcn_raw_buffer_load_b32(buf, from + 4u * j, 0, 0);
    e.last = __builtin_amdgcn_raw_buffer_load_b32(buf, from + 16u, 0, 0);
  }
  return e;
}
template <bool VEC>
__device__ inline void turn_eight(const Eight& e, uint32_t at, int left, float (&out)[8]) {
  u32x4 v = e.v;
  if constexpr (!VEC) {
    const uint32_t turn = (at & 2u) * 8u;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __builtin_amdgcn_alignbit(j < 3 ? e.v[j + 1] : e.last, e.v[j], turn);
  }
  const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = VEC || i < left ? (float)h[i] : 0.0f;
}
// VEC: rows of n start on eight elements.  SLOPE: dz is written (pre given); else only the sums of dy.
template <bool VEC, bool SLOPE>
__global__ void __launch_bounds__(kThreads)
linear_grad_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ pre, uint16_t* __restrict__ dpre,
                   uint16_t* __restrict__ padded, float* __restrict__ dbias, int M, int N, int act, int rows,
                   uint32_t* __restrict__ counters, float* __restrict__ partials) {
  __shared__ __attribute__((aligned(16))) float red[kRowLanes][kCols];
  __shared__ uint32_t flag;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int c0 = blockIdx.x * kCols, c = c0 + 8 * tx, left = N - c;
  const int m_end = min(M, ((int)blockIdx.y + 1) * rows);
  const uint32_t bytes = ((uint32_t)M * (uint32_t)N * 2u + 3u) & ~3u;
  const __amdgpu_buffer_rsrc_t dres = make_rsrc(dy, bytes), zres = make_rsrc(pre, SLOPE ? bytes : 0u);
  float sum[8] = {};
  // kUnroll rows' loads in flight together (rows past the end: the last one's, passed over)
  for (int r0 = blockIdx.y * rows + ty; r0 < m_end; r0 += kUnroll * kRowLanes) {
    if (left <= 0) break;
    Eight de[kUnroll], ze[SLOPE ? kUnroll : 1];
    uint32_t at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      at[u] = ((uint32_t)min(r0 + u * kRowLanes, m_end - 1) * (uint32_t)N + (uint32_t)c) * 2u;
      de[u] = load_eight<VEC>(dres, at[u]);
      if constexpr (SLOPE) ze[u] = load_eight<VEC>(zres, at[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kRowLanes;
      if (r >= m_end) break;
      float d[8];
      turn_eight<VEC>(de[u], at[u], left, d);
      if constexpr (SLOPE) {
        float z[8];
        turn_eight<VEC>(ze[u], at[u], left, z);
        times_slope(act, z, d);
        f16x8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (_Float16)d[i];
        store_eight<VEC>(dpre + (size_t)r * N + c, left, o);
        if (!VEC && padded) {
          // (0 times a slope is 0 past the row's end: act' is finite at 0)
          const int np = (N + 7) & ~7;
          *reinterpret_cast<f16x8*>(padded + (size_t)r * np + c) = o;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
    }
  }
  if (!dbias) return;
#pragma unroll
  for (int i = 0; i < 8; i += 4)
    *reinterpret_cast<f32x4*>(&red[ty][8 * tx + i]) = f32x4{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]};
  __syncthreads();
  const int n = c0 + tid;
  const bool mine = tid < kCols && n < N;
  float v = 0.0f;
  if (tid < kCols) {
#pragma unroll
    for (int r = 0; r < kRowLanes; ++r) v += red[r][tid];
  }
  if (gridDim.y == 1) {
    if (mine) dbias[n] = v;
    return;
  }
  if (mine)
    __hip_atomic_store(partials + (size_t)blockIdx.y * N + n, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!arrive_last(counters + blockIdx.x, gridDim.y, &flag)) return;
  if (!mine) return;
  v = 0.0f;
  for (int b0 = 0; b0 < (int)gridDim.y; b0 += 8) {           // eight loads in flight
    float p[8];
#pragma unroll
    for (int b = 0; b < 8; ++b)
      p[b] = __hip_atomic_load(partials + (size_t)min(b0 + b, (int)gridDim.y - 1) * N + n, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int b = 0; b < 8; ++b)
      if (b0 + b < (int)gridDim.y) v += p[b];
  }
  dbias[n] = v;
}

}  // namespace

size_t linear_grad_workspace_bytes(int m, int n, bool bias) {
  const GradPlan p = grad_plan(m, n, bias);
  return bias && p.row_blocks > 1 ? (size_t)p.row_blocks * n * sizeof(float) : 0;
}

hipError_t launch_linear_grad(const uint16_t* dy, const uint16_t* pre, uint16_t* dpre, uint16_t* padded, float* dbias,
                              int m, int n, int act, uint32_t* counters, float* partials, hipStream_t stream) {
  const GradPlan p = grad_plan(m, n, dbias != nullptr);
  auto kern = n % 8 ? (pre ? linear_grad_kernel<false, true> : linear_grad_kernel<false, false>)
                    : (pre ? linear_grad_kernel<true, true> : linear_grad_kernel<true, false>);
  return launch_kernel(kern, dim3((unsigned)p.col_blocks, (unsigned)p.row_blocks), dim3(kThreads), 0, stream, dy, pre,
                       dpre, padded, dbias, m, n, act, p.rows, counters, partials);
}

}  // namespace w4a16
