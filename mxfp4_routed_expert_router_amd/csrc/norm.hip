// Layer norm and RMS norm, forward.
#include "norm.h"

namespace moe_fp4 {
namespace {

// TPR threads a row, up to CH chunks of eight elements a thread.
template <typename TX, typename TY, int TPR, int CH, bool Whole>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_kernel(NormArgs g) {
  constexpr int RPB = norm_threads(TPR) / TPR;
  __shared__ float slot[3 * (norm_threads(TPR) / 64)];
  const int lt = threadIdx.x % TPR, nc = (g.H + 7) / 8;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int64_t rr = row < g.T ? row : g.T - 1;  // a workgroup's threads stay together at its barriers
  const auto size = [&](int k) { return Whole ? 8 : g.H - 8 * k < 8 ? g.H - 8 * k : 8; };  // of chunk k
  Chunk<TX> raw[CH];
  float x[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lt + c * TPR;
    if (k < nc) raw[c].load(g.x, rr * g.ldx + 8 * k, size(k));
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) raw[c].values(x[c]);
  const float per = 1.0f / (float)g.H;
  float mean = 0.f;
  if (!g.rms) {
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lt + c * TPR < nc)
#pragma unroll
        for (int r = 0; r < 8; ++r) s[0] += x[c][r];  // zeros behind a chunk's end
    row_sums<(TPR > 64)>(s, slot);
    mean = s[0] * per;
  }
  // of the deviations: their squares' sum and their own, which is what rounding left
  // out of the mean.  It corrects the mean, the deviations and the squares.
  float ss[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (lt + c * TPR < nc)
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        x[c][r] -= mean;
        if (Whole || r < size(lt + c * TPR)) {
          ss[0] += x[c][r] * x[c][r];
          ss[1] += x[c][r];
        }
      }
  row_sums<(TPR > 64)>(ss, slot + norm_threads(TPR) / 64);
  const float off = g.rms ? 0.f : ss[1] * per;
  const float squares = ss[0] - ss[1] * off;
  mean += off;
  const float rstd = 1.0f / sqrtf((squares < 0.f ? 0.f : squares) * per + g.eps);  // NaN stays NaN
  if (row >= g.T) return;
  if (lt == 0) {
    if (g.mean) g.mean[row] = mean;
    if (g.rstd) g.rstd[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lt + c * TPR;
    if (k >= nc) break;
    float w[8], b[8];
    load_weight(g.gamma, g.w_type, 8 * k, size(k), 1.0f, w);
    load_weight(g.beta, g.w_type, 8 * k, size(k), 0.0f, b);
#pragma unroll
    for (int r = 0; r < 8; ++r) w[r] = (x[c][r] - off) * rstd * w[r] + b[r];
    store_chunk<TY, true>(g.y, row * g.ldy + 8 * k, size(k), w);
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  pick_types(a, [&](auto tx, auto ty) {
    pick_shape(a.H, [&](auto tpr, auto ch, auto whole) {
      constexpr int TPR = decltype(tpr)::value, threads = norm_threads(TPR), RPB = threads / TPR;
      hipLaunchKernelGGL((norm_kernel<decltype(tx), decltype(ty), TPR, decltype(ch)::value, decltype(whole)::value != 0>),
                         dim3((unsigned)((a.T + RPB - 1) / RPB)), dim3(threads), 0, stream, a);
    });
  });
  return hipGetLastError();
}

}  // namespace moe_fp4
