// The forward product of one to four rows an expert: a stream of the weights.
//
// A wave takes R columns (R weight rows) whole: lane l holds elements 8 l .. 8 l
// + 7 of every 512 of the sum, so each load is 1 KB of one weight row and R x U
// of them are in flight.  Pairs of products are added in fp32 (v_dot2), and
// the lanes' sums at the end in a fixed tree.  x comes from the caches.
#include "block_device.h"

namespace moe_fp4 {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <typename T>
__device__ __forceinline__ float dot8(const u32x4& a, const u32x4& b, float c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t ai = a[i], bi = b[i];
    if constexpr (T::kType == kBf16)
      c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, ai), __builtin_bit_cast(bf16x2, bi), c, false);
    else
      c = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, ai), __builtin_bit_cast(f16x2, bi), c, false);
  }
  return c;
}

template <typename T, int M, int R, int U>
__global__ void __launch_bounds__(256) product_row_kernel(ProductArgs g) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int e, row0, nrows;
  if (!row_tile(g.offsets, g.E, g.P, M, blockIdx.y, e, row0, nrows)) return;
  const int j0 = (blockIdx.x * 4 + wave) * R;
  if (j0 >= g.J) return;
  const uint16_t* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r)  // columns past the end read the last one's weights
    w[r] = g.b + (int64_t)e * g.w_stride + (int64_t)(j0 + r < g.J ? j0 + r : g.J - 1) * g.ldb + lane * 8;
  const uint16_t* x[M];
  bool has[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int s = m < nrows ? __builtin_amdgcn_readfirstlane(source_row(g, row0 + m)) : -1;
    has[m] = s >= 0;
    x[m] = g.a + (int64_t)(has[m] ? s : 0) * g.lda + lane * 8;
  }
  float acc[R][M] = {};
  int k = 0;
  for (; k + 512 * U <= g.K; k += 512 * U) {
    u32x4 fw[R][U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
        fw[r][u] = load8_once(w[r] + k + u * 512);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const u32x4 fx = has[m] ? load8(x[m] + k + u * 512, 8) : zero4();
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][m] = dot8<T>(fw[r][u], fx, acc[r][m]);
      }
  }
  for (; k < g.K; k += 512) {
    const int have = g.K - k - lane * 8;
    if (have <= 0) break;
    u32x4 fw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) fw[r] = load8(w[r] + k, have);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const u32x4 fx = has[m] ? load8(x[m] + k, have) : zero4();
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r][m] = dot8<T>(fw[r], fx, acc[r][m]);
    }
  }
  // lane m finishes row m's R columns
  f32x4 v = {};
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float s = wave_sum_f32(acc[r][m]);
      if (lane == m) v[r] = s;
    }
  if (lane < nrows) finish1<false>(g, g.c, row0 + lane, j0, R, v);
}

template <typename T, int M, int R, int U>
void launch_one(const ProductArgs& a, hipStream_t stream) {
  const dim3 grid((a.J + 4 * R - 1) / (4 * R), (unsigned)row_tiles_most(a, M));
  hipLaunchKernelGGL((product_row_kernel<T, M, R, U>), grid, dim3(256), 0, stream, a);
}
// Loads in flight and columns of a wave, by time (one MI355X, bf16, K = 5120,
// weights cold; a whole product of N columns in us):
//   one row    N = 5120: R1 U5 10.4, R2 U5 11.3, R4 U5 13.4; N = 288: 3.8, 4.9, 6.9
//   two rows   N = 5120: R1 U5 11.9, R2 U5 12.8; N = 288: 4.2, 5.4
//   four rows  N = 5120: R1 U5 15.6, R2 U2 15.3; N = 288: 5.0, 7.7; one to four
//              rows each of 30 experts, N = 2304: 145, 115
// A sum that is no multiple of 512 U ends in the loop with one load a column in
// flight.  One row, N = 5120: K = 4096 9.2 us, 2304 8.7 (5120: 10.9); one token's six
// of 138 experts: 2304 x 5120 24.4 us (5.8 TB/s), 2304 x 4096 22.2 (5.1), 5120 x 2304
// 32.6 (4.3).
template <typename T>
void launch(const ProductArgs& a, int m, hipStream_t stream) {
  if (m == 1) return launch_one<T, 1, 1, 5>(a, stream);
  if (m == 2) return launch_one<T, 2, 1, 5>(a, stream);
  if (a.J * row_tiles_most(a, 4) < 4096) return launch_one<T, 4, 1, 5>(a, stream);
  return launch_one<T, 4, 2, 2>(a, stream);
}

}  // namespace

void launch_product_row(const ProductArgs& a, int m, hipStream_t stream) {
  if (a.type == kBf16)
    launch<Bf16>(a, m, stream);
  else
    launch<F16>(a, m, stream);
}

}  // namespace moe_fp4
