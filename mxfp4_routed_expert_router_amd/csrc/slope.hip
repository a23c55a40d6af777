// The elementwise part of a dense product's backward pass: dz = dy act'(z) and
// the bias gradient, its column sums.
#include "block_device.h"

namespace moe_fp4 {
namespace {

constexpr int kSlopeCols = 32, kSlopeRows = 8;  // threads of a workgroup

// dz of the eight columns from j on of row i, `have` of them in it, zeros behind.
template <typename T, typename TD>
__device__ __forceinline__ void load_dz(const SlopeArgs& g, int64_t i, int j, int have, float (&d)[8]) {
  load8_as_f32<TD>(g.dy, i * g.lddy + j, have, d);
  if (g.act == kActNone) return;
  float z[8];
  load8_as_f32<T>(g.z, i * g.ldz + j, have, z);
#pragma unroll
  for (int r = 0; r < 8; ++r) d[r] *= activate_slope(z[r], g.act);
}

// The largest of a value over the workgroup's 256 threads.
__device__ __forceinline__ uint32_t workgroup_max(uint32_t v) {
  __shared__ uint32_t of_wave[4];
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) v = of_wave[w] > v ? of_wave[w] : v;
  return v;
}

// fp16 holds 2^-24 to 65504, an fp32 dy or its product with a slope may lie anywhere:
// 1e5 would become inf and 1e-8 zero on the way into fp32 sums that hold both.  So
// fp16 dz is multiplied by 2^s, s such that the largest finite |dz| lies in [2^14, 2^15).
// This pass finds that largest value, one part a workgroup (non-negative floats are
// ordered as their bits are); slope_kernel joins the parts.  It reads dy and z once
// more: the backward pass of 8192 x 2304 x 5120, f16, gelu, takes 388 us, 361 without.
template <typename T, typename TD>
__global__ void __launch_bounds__(256) slope_top_kernel(SlopeArgs g) {
  const int tc = threadIdx.x & (kSlopeCols - 1), tr = threadIdx.x / kSlopeCols;
  const int j = (blockIdx.x * kSlopeCols + tc) * 8, have = g.N - j;
  uint32_t top = 0;
  if (have > 0)
    for (int64_t i = (int64_t)blockIdx.y * kSlopeRows + tr; i < g.M; i += (int64_t)gridDim.y * kSlopeRows) {
      float d[8];
      load_dz<T, TD>(g, i, j, have, d);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t b = __float_as_uint(d[r]) & 0x7FFFFFFFu;
        if (r < have && b < 0x7F800000u && b > top) top = b;
      }
    }
  top = workgroup_max(top);
  if (threadIdx.x == 0) g.top[blockIdx.y * gridDim.x + blockIdx.x] = __uint_as_float(top);
}

// One pass over dy and z, bound by their bytes.  Thread (r, c) takes eight
// neighbouring columns of every eighth row of the workgroup's rows and sums them
// in fp32 before dz is rounded; the eight sums of a column are joined in order
// and written to part[workgroup row].  dz is rounded to the products' type
// because it feeds the matrix cores: one rounding, of 2^-8 (bf16) or 2^-11 (fp16)
// relative at most, and in fp16 of 2^-39 of the largest |dz| where that is more.
// The bias gradient does not see that rounding.
template <typename T, typename TD>
__global__ void __launch_bounds__(256) slope_kernel(SlopeArgs g) {
  constexpr int V = 8;
  __shared__ float s[kSlopeRows][kSlopeCols * V];
  const int tc = threadIdx.x & (kSlopeCols - 1), tr = threadIdx.x / kSlopeCols;
  const int j = (blockIdx.x * kSlopeCols + tc) * V, have = g.N - j;
  float sum[V] = {}, scale = 1.0f;
  if (T::kType == kF16 && g.dz) {
    uint32_t top = 0;
    for (int i = threadIdx.x; i < g.tops; i += 256) {
      const uint32_t b = __float_as_uint(g.top[i]);
      top = b > top ? b : top;
    }
    top = workgroup_max(top);
    int s = 14 + 127 - (int)(top >> 23);
    if (s > 126) s = 126;  // 2^-s stays a normal number
    scale = __uint_as_float((uint32_t)(127 + s) << 23);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *g.factor = __uint_as_float((uint32_t)(127 - s) << 23);
  }
  if (have > 0)
    for (int64_t i = (int64_t)blockIdx.y * kSlopeRows + tr; i < g.M; i += (int64_t)gridDim.y * kSlopeRows) {
      float d[V];
      load_dz<T, TD>(g, i, j, have, d);
#pragma unroll
      for (int r = 0; r < V; ++r)
        if (r < have) sum[r] += d[r];
      if (g.dz) {
        if constexpr (T::kType == kF16)
#pragma unroll
          for (int r = 0; r < V; ++r) d[r] *= scale;
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

hipError_t launch_slope(SlopeArgs a, hipStream_t stream) {
  const dim3 grid((a.N + kSlopeCols * 8 - 1) / (kSlopeCols * 8), slope_blocks(a.M));
  if (a.type == kF16 && a.dz) {
    const unsigned most = kSlopeTops / grid.x;  // four at least: kMaxWidth / 256 <= kSlopeTops / 4
    const dim3 few(grid.x, grid.y < most ? grid.y : most);
    a.tops = (int)(few.x * few.y);
    if (a.dy_type == kF32) hipLaunchKernelGGL((slope_top_kernel<F16, F32>), few, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((slope_top_kernel<F16, F16>), few, dim3(256), 0, stream, a);
  }
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
