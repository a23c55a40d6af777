// The dense forward product of 5 to 16 rows (a decode batch): bound by the weights'
// bytes.
//
// A workgroup takes 16 columns (16 weight rows) and all rows of the result; its
// NW waves split the sum, 64 of it a unit, wave w taking the units w,
// w + NW, ....  The weights go from memory to the registers as the matrix
// instruction's fragments, each element once and without a stop in LDS: a wave
// has U units of 2 KB in flight.  The rows of x come the same way, from the
// L2 that holds them.  The waves' sums meet in LDS and are added in wave order.
#include "block_device.h"

namespace moe_fp4 {
namespace {

template <typename T, int NW, int U>
__global__ void __launch_bounds__(NW * 64) product_few_kernel(ProductArgs g) {
  __shared__ f32x4 sums[NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quad = lane >> 4;
  const int j0 = blockIdx.x * 16;
  // columns past the end read the last one's weights: their results are not stored
  const int jr = j0 + l16 < g.J ? j0 + l16 : g.J - 1;
  const uint16_t* const w = g.b + (int64_t)jr * g.ldb + quad * 8;
  const bool live = l16 < g.P;
  const uint16_t* const x = g.a + (int64_t)(live ? l16 : 0) * g.lda + quad * 8;
  const int units = (g.K + 63) / 64;
  f32x4 acc = {};
  for (int u0 = wave; u0 < units; u0 += NW * U) {
    u32x4 fw[U][2], fx[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (u0 + u * NW) * 64 + h * 32;
        fw[u][h] = load8(w + k, g.K - k - quad * 8);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (u0 + u * NW) * 64 + h * 32;
        fx[u][h] = load8(x + k, live ? g.K - k - quad * 8 : 0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = T::mfma(fw[u][h], fx[u][h], acc);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
  f32x4 v = sums[0][lane];
#pragma unroll
  for (int i = 1; i < NW; ++i) v += sums[i][lane];
  const int j = j0 + quad * 4;
  if (live && j < g.J) finish1<false>(g, g.c, l16, j, 4, v);
}

// N = K = 5120, weights cold: 8 rows 20.0 us, 16 rows 23.7 (their bytes: 10.6).
// Sixteen waves where the workgroups would leave CUs with one (N = 2304, K = 5120,
// 16 rows: 14.2 us, 15.0 with eight).
template <typename T>
void launch(const ProductArgs& a, hipStream_t stream) {
  const dim3 grid((a.J + 15) / 16);
  if (grid.x <= 256)
    hipLaunchKernelGGL((product_few_kernel<T, 16, 5>), grid, dim3(1024), 0, stream, a);
  else
    hipLaunchKernelGGL((product_few_kernel<T, 8, 5>), grid, dim3(512), 0, stream, a);
}

}  // namespace

void launch_product_few(const ProductArgs& a, hipStream_t stream) {
  if (a.type == kBf16)
    launch<Bf16>(a, stream);
  else
    launch<F16>(a, stream);
}

}  // namespace moe_fp4
