// linear_grad.hip -- gradient of the linear layer's epilogue on gfx950: dz = dy act'(z) in fp32, rounded
// once to fp16 (an output, and the fp16 operand of the product that follows), and the bias's
// gradient, the column sums of the unrounded dz in fp32.
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
constexpr int kRowsWG = 128;                     // rows of a workgroup

struct GradPlan {
  int col_blocks, row_blocks, rows;              // rows: of a workgroup
};
GradPlan grad_plan(int m, int n, bool bias) {
  GradPlan p;
  p.col_blocks = (n + kCols - 1) / kCols;
  p.rows = kRowsWG;
  p.row_blocks = (m + p.rows - 1) / p.rows;
  // (a counter per column block, and 65535 row blocks in a grid: beyond, a workgroup takes more rows)
  const int most = bias && p.col_blocks > kCounters ? 1 : 65535;
  if (p.row_blocks > most) {
    p.rows = (m + most - 1) / most;
    p.row_blocks = (m + p.rows - 1) / p.rows;
  }
  return p;
}

// VEC: rows of n start on eight elements; else element by element, a thread's columns sixteen apart.
// SLOPE: dz is written (pre given); else only the sums of dy.
template <bool VEC, bool SLOPE>
__global__ void __launch_bounds__(kThreads)
linear_grad_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ pre, uint16_t* __restrict__ dpre,
                   uint16_t* __restrict__ padded, float* __restrict__ dbias, int M, int N, int act, int rows,
                   uint32_t* __restrict__ counters, float* __restrict__ partials) {
  __shared__ float red[kRowLanes][kCols];
  __shared__ uint32_t flag;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int c0 = blockIdx.x * kCols;
  const int m_end = min(M, ((int)blockIdx.y + 1) * rows);
  const int np = (N + 7) & ~7;
  auto col = [&](int i) { return VEC ? c0 + 8 * tx + i : c0 + tx + 16 * i; };
  float sum[8] = {};
  for (int r = blockIdx.y * rows + ty; r < m_end; r += kRowLanes) {
    const size_t row = (size_t)r * N;
    float d[8];
    if constexpr (VEC) {
      if (col(0) >= N) break;
      const f16x8 v = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(dy + row + col(0)));
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = (float)v[i];
      if constexpr (SLOPE) {
        const f16x8 z = __builtin_nontemporal_load(reinterpret_cast<const f16x8*>(pre + row + col(0)));
        float zf[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) zf[i] = (float)z[i];
        times_slope(act, zf, d);
        f16x8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (_Float16)d[i];
        *reinterpret_cast<f16x8*>(dpre + row + col(0)) = o;
      }
    } else {
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = col(i) < N ? half_bits_to_float(dy[row + col(i)]) : 0.0f;
        z[i] = SLOPE && col(i) < N ? half_bits_to_float(pre[row + col(i)]) : 0.0f;
      }
      if constexpr (SLOPE) {
        times_slope(act, z, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col(i) < N) dpre[row + col(i)] = float_to_half_bits(d[i]);
          if (padded && col(i) < np) padded[(size_t)r * np + col(i)] = float_to_half_bits(col(i) < N ? d[i] : 0.0f);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += d[i];
  }
  if (!dbias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[ty][col(i) - c0] = sum[i];
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
