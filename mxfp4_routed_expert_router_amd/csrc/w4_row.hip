// The product of one or two rows with 4-bit weights: a stream of the weights.
//
// A workgroup takes R columns (R weight rows) whole; its threads split the sum, thread
// i taking the groups of 32 inputs i, i + threads, ....  A thread has 16 bytes of each of
// the R rows in flight, and the rows' x of its group in registers, which all R columns
// use.  A group's 32 products are added in fp32 (v_dot2), then times the scale; for int4,
// sum (q - z) x = sum q x - z sum x, the latter once for all columns.  The waves' sums
// meet in LDS and are added in wave order.
//
// One row of 9216 x 5120, MX: 8.0 us for 25.2 MB; of 65536 x 5120 33.8 us (5.3 TB/s), bound by the
// bytes; of 288 x 5120 2.8 us, a launch and one load's latency.  int4 takes half as long
// again (50 us at 65536 x 5120) with 1.44 times the vector instructions, which keep their units 49 %
// busy (MX 52 %): neither they nor the bytes (3.4 TB/s) bound it; a workgroup's waves wait for their
// loads, of half as many columns at a time.
#include "w4_device.h"

namespace moe_fp4 {
namespace {

template <typename T, int Code, int M, int R>
__global__ void __launch_bounds__(1024) w4_row_kernel(W4Args g, int shift) {
  __shared__ float sums[16][R * M];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * R, m0 = blockIdx.y * M, groups = g.K / 32;
  float acc[R][M] = {};
  for (int i = threadIdx.x; i < groups; i += blockDim.x) {
    u32x4 codes[R];
    float scale[R], zero[R];
    u32x4 x[M][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {  // columns past the end read the last one's weights
      const int64_t n = n0 + r < g.N ? n0 + r : g.N - 1;
      codes[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g.codes + n * g.ldw) + i);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {  // rows past the end read the first one
      const uint16_t* const p = g.x + (int64_t)(m0 + m < g.M ? m0 + m : m0) * g.ldx + i * 32;
#pragma unroll
      for (int d = 0; d < 4; ++d) x[m][d] = *reinterpret_cast<const u32x4_any*>(p + d * 8);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = n0 + r < g.N ? n0 + r : g.N - 1, at = n * g.groups + (i >> shift);
      scale[r] = scale_of<Code>(g, at);
      if constexpr (Code == kInt4) zero[r] = g.zeros ? (float)g.zeros[at] : 8.0f;
    }
    float sx[M] = {};
    if constexpr (Code == kInt4) {
      const uint32_t one = T::kType == kBf16 ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int d = 0; d < 16; ++d) sx[m] = dot2<T>(one, x[m][d / 4][d % 4], sx[m]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float dot[M] = {};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const u32x4 w = decode8<T, Code>(codes[r][d]);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int h = 0; h < 4; ++h) dot[m] = dot2<T>(w[h], x[m][d][h], dot[m]);
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if constexpr (Code == kInt4) dot[m] -= zero[r] * sx[m];
        acc[r][m] += scale[r] * dot[m];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float v = wave_sum_f32(acc[r][m]);
      if (lane == 0) sums[wave][r * M + m] = v;
    }
  __syncthreads();
  if (threadIdx.x >= R * M) return;
  const int waves = blockDim.x >> 6, r = threadIdx.x / M, m = threadIdx.x % M;
  float v = sums[0][threadIdx.x];
  for (int w = 1; w < waves; ++w) v += sums[w][threadIdx.x];
  if (n0 + r < g.N && m0 + m < g.M) finish_w4<T>(g, m0 + m, n0 + r, v);
}

template <typename T, int Code, int M, int R>
void launch_columns(const W4Args& a, int waves, hipStream_t stream) {
  const dim3 grid((a.N + R - 1) / R, (a.M + M - 1) / M);
  int shift = 0;  // groups of 32 in a scale's
  while (32 << shift < a.group) ++shift;
  hipLaunchKernelGGL((w4_row_kernel<T, Code, M, R>), grid, dim3(waves * 64), 0, stream, a, shift);
}
// Columns of a workgroup by time (one MI355X, weights cold, us; R = 1, 2, 4, 8):
//   one row, bf16, MX   N = 288, K = 5120: 2.8, 2.9, 3.2, 3.9; 5120 x 2304: 5.4, 4.6, 4.7, 5.3;
//                       9216 x 5120: 9.8, 7.7, 8.1, 8.8; 65536 x 5120: 53.9, 37.8, 36.6, 33.8
//   int4, groups of 128 9216 x 5120: 10.1, 10.2, 10.2, 11.9; 65536 x 5120: 54.4, 50.9, 51.7, 55.1
//   two rows, MX        9216 x 5120: 15.2, 11.7, 11.5, 11.9; 65536 x 5120: 89.4, 62.5, 57.0, 51.9
template <typename T, int Code, int M>
void launch_rows(const W4Args& a, hipStream_t stream) {
  const int need = (a.K / 32 + 63) / 64, waves = need < 16 ? need : 16;
  const int64_t all = (int64_t)a.N * waves;
  if (all < 8192) launch_columns<T, Code, M, 1>(a, waves, stream);
  else if (all < 16384) launch_columns<T, Code, M, 2>(a, waves, stream);
  else if (Code == kInt4 || all < 65536) launch_columns<T, Code, M, 4>(a, waves, stream);
  else launch_columns<T, Code, M, Code == kMx ? 8 : 4>(a, waves, stream);
}
template <typename T, int Code>
void launch(const W4Args& a, hipStream_t stream) {
  if (a.M == 1) launch_rows<T, Code, 1>(a, stream);
  else launch_rows<T, Code, 2>(a, stream);
}

}  // namespace

void launch_w4_row(const W4Args& a, hipStream_t stream) {
  if (a.type == kBf16) a.code == kMx ? launch<Bf16, kMx>(a, stream) : launch<Bf16, kInt4>(a, stream);
  else a.code == kMx ? launch<F16, kMx>(a, stream) : launch<F16, kInt4>(a, stream);
}

}  // namespace moe_fp4
