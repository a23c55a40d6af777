// The elementwise part of a dense product's backward pass: dz = dy act'(z) and
// the bias gradient, its column sums.
#include "block_device.h"

namespace moe_fp4 {
namespace {

constexpr int kSlopeCols = 32, kSlopeRows = 8;  // threads of a workgroup

// One pass over dy and z, bound by their bytes.  Thread (r, c) takes eight
// neighbouring columns of every eighth row of the workgroup's rows and sums them
// in fp32 before dz is rounded; the eight sums of a column are joined in order
// and written to part[workgroup row].  dz is rounded to the products' type
// because it feeds the matrix cores (one rounding, 2^-9 or 2^-12 relative at
// most); the bias gradient does not see that rounding.
template <typename T, typename TD>
__global__ void __launch_bounds__(256) slope_kernel(SlopeArgs g) {
  constexpr int V = 8;
  __shared__ float s[kSlopeRows][kSlopeCols * V];
  const int tc = threadIdx.x & (kSlopeCols - 1), tr = threadIdx.x / kSlopeCols;
  const int j = (blockIdx.x * kSlopeCols + tc) * V, have = g.N - j;
  float sum[V] = {};
  if (have > 0)
    for (int64_t i = (int64_t)blockIdx.y * kSlopeRows + tr; i < g.M; i += (int64_t)gridDim.y * kSlopeRows) {
      float d[V], z[V];
      load8_as_f32<TD>(g.dy, i * g.lddy + j, have, d);
      if (g.act != kActNone) {
        load8_as_f32<T>(g.z, i * g.ldz + j, have, z);
#pragma unroll
        for (int r = 0; r < V; ++r) d[r] *= activate_slope(z[r], g.act);
      }
#pragma unroll
      for (int r = 0; r < V; ++r)
        if (r < have) sum[r] += d[r];
      if (g.dz) {
        uint16_t* const o = g.dz + i * g.N + j;
        if (have >= V) {
          u32x4 a;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            a[r] = (uint32_t)T::from_f32(d[2 * r]) | ((uint32_t)T::from_f32(d[2 * r + 1]) << 16);
          *reinterpret_cast<u32x4_any*>(o) = a;
        } else {
#pragma unroll
          for (int r = 0; r < V; ++r)
            if (r < have) o[r] = T::from_f32(d[r]);
        }
      }
    }
  if (!g.db) return;
#pragma unroll
  for (int r = 0; r < V; ++r) s[tr][tc * V + r] = sum[r];
  __syncthreads();
  const int col = blockIdx.x * kSlopeCols * V + threadIdx.x;
  if (col >= g.N) return;
  float v = s[0][threadIdx.x];
#pragma unroll
  for (int r = 1; r < kSlopeRows; ++r) v += s[r][threadIdx.x];
  g.part[(int64_t)blockIdx.y * g.N + col] = v;
}

__global__ void __launch_bounds__(256) slope_columns_kernel(const float* part, int parts, int N,
                                                            float* db, int accumulate) {
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), p0 = threadIdx.x >> 5;
  float v = 0.f;
  if (col < N)
    v = column_sum(part + col, N, p0, parts);
  s[p0][threadIdx.x & 31] = v;
  __syncthreads();
  if (p0 || col >= N) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x & 31];
  db[col] = accumulate ? db[col] + v : v;
}

}  // namespace

int slope_blocks(int M) {
  const int b = (M + 31) / 32;
  return b < 1 ? 1 : b > 256 ? 256 : b;
}

hipError_t launch_slope(const SlopeArgs& a, hipStream_t stream) {
  const dim3 grid((a.N + kSlopeCols * 8 - 1) / (kSlopeCols * 8), slope_blocks(a.M));
  const auto run = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, a); };
  if (a.type == kBf16)
    a.dy_type == kF32 ? run(slope_kernel<Bf16, F32>) : run(slope_kernel<Bf16, Bf16>);
  else
    a.dy_type == kF32 ? run(slope_kernel<F16, F32>) : run(slope_kernel<F16, F16>);
  if (a.db)
    hipLaunchKernelGGL(slope_columns_kernel, dim3((a.N + 31) / 32), dim3(256), 0, stream, a.part,
                       slope_blocks(a.M), a.N, a.db, a.accumulate);
  return hipGetLastError();
}

}  // namespace moe_fp4
