// Layer norm and RMS norm, backward.
#include "norm.h"

namespace moe_fp4 {
namespace {

// The workgroups walk the rows; a thread keeps its columns' gamma and the sums
// of dgamma and dbeta over the rows it has seen, and writes them once at the
// end to part[workgroup], which norm_columns_kernel adds up.  The next row's
// x and dy are on their way while a row is summed and written.
// RPB rows a workgroup: four, a wave each, or one by all its Threads threads.
template <typename TX, typename TY, int RPB, int Threads, int CH, bool Whole>
__global__ void __launch_bounds__(Threads) norm_backward_kernel(NormArgs g) {
  constexpr int TPR = RPB > 1 ? 64 : Threads;
  __shared__ float slot[2][2 * (Threads / 64)];
  // RPB > 1: [RPB][H], one gradient at a time; else gamma, which would take the
  // registers that let another workgroup run beside (5120 bf16: 164 with it there, 179 without):
  // [CH][2][threads] of four values, each thread's own
  extern __shared__ __align__(16) float sums[];
  const int lt = threadIdx.x % TPR, sub = threadIdx.x / TPR, nc = (g.H + 7) / 8;
  const float per = 1.0f / (float)g.H;
  const auto size = [&](int k) { return Whole ? 8 : g.H - 8 * k < 8 ? g.H - 8 * k : 8; };  // of chunk k
  float w[RPB > 1 ? CH : 1][8], dw[CH][8] = {}, db[CH][8] = {};
  f32x4* const ws = reinterpret_cast<f32x4*>(sums) + lt;
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (lt + c * TPR < nc) {
      float (&v)[8] = w[RPB > 1 ? c : 0];
      load_weight(g.gamma, g.w_type, 8 * (lt + c * TPR), size(lt + c * TPR), 1.0f, v);
      if constexpr (RPB == 1) {
        ws[2 * c * TPR] = f32x4{v[0], v[1], v[2], v[3]};
        ws[(2 * c + 1) * TPR] = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
  const int64_t stride = (int64_t)gridDim.x * RPB;
  Chunk<TX> rx[CH];
  Chunk<TY> rd[CH];
  float mean = 0.f, rstd = 0.f;
  auto send = [&](int64_t base) {  // for the row of this thread at `base`, or the last one
    const int64_t row = base + sub < g.T ? base + sub : g.T - 1;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = lt + c * TPR;
      if (k < nc) {
        rx[c].load(g.x, row * g.ldx + 8 * k, size(k));
        rd[c].load(g.dy, row * g.ldy + 8 * k, size(k));
      }
    }
    mean = g.rms ? 0.f : g.mean_in[row];
    rstd = g.rstd_in[row];
  };
  int64_t base = (int64_t)blockIdx.x * RPB;
  if (base < g.T) send(base);
  for (int turn = 0; base < g.T; base += stride, turn ^= 1) {
    const int64_t row = base + sub;
    const bool live = row < g.T;
    float x[CH][8], d[CH][8];
    const float m = mean, rs = rstd;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lt + c * TPR < nc) {
        rx[c].values(x[c]);
        rd[c].values(d[c]);
      }
    if (base + stride < g.T) send(base + stride);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lt + c * TPR < nc) {
        f32x4 v[2];
        if constexpr (RPB == 1) {
          v[0] = ws[2 * c * TPR];
          v[1] = ws[(2 * c + 1) * TPR];
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {  // dy is 0 behind a chunk's end, and so is every term
          x[c][r] = (x[c][r] - m) * rs;
          if (RPB == 1 || live) {
            dw[c][r] += d[c][r] * x[c][r];
            db[c][r] += d[c][r];
          }
          if constexpr (RPB == 1) d[c][r] *= v[r / 4][r % 4];
          else d[c][r] *= w[c][r];
          s[0] += d[c][r];
          s[1] += d[c][r] * x[c][r];
        }
      }
    row_sums<RPB == 1>(s, slot[turn]);
    const float mg = g.rms ? 0.f : s[0] * per, mgx = s[1] * per;
    if ((RPB == 1 || live) && g.dx)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = lt + c * TPR;
        if (k >= nc) break;
        float o[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) o[r] = rs * (d[c][r] - mg - x[c][r] * mgx);
        store_chunk<TX, false>(g.dx, row * g.lddx + 8 * k, size(k), o);
      }
  }
  if (!g.part) return;
  float* const part = g.part + (int64_t)blockIdx.x * 2 * g.H;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (lt + c * TPR < nc)
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (Whole || r < size(lt + c * TPR))
              sums[sub * g.H + (lt + c * TPR) * 8 + r] = which ? db[c][r] : dw[c][r];
      __syncthreads();
      for (int h = threadIdx.x; h < g.H; h += 256) {
        float s = sums[h];
#pragma unroll
        for (int i = 1; i < RPB; ++i) s += sums[i * g.H + h];
        part[which * g.H + h] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (lt + c * TPR < nc)
          store_chunk<F32, false>(part, which * g.H + (lt + c * TPR) * 8, size(lt + c * TPR), which ? db[c] : dw[c]);
    }
  }
}

// Column sums over the workgroups' parts: 32 columns a workgroup, eight
// threads each over every eighth part, joined in order.
__global__ void __launch_bounds__(256) norm_columns_kernel(const float* part, int parts, int H,
                                                           float* dgamma, float* dbeta, int accumulate) {
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), p0 = threadIdx.x >> 5;
  float v = 0.f;
  if (col < 2 * H)
    v = column_sum(part + col, 2 * H, p0, parts);
  s[p0][threadIdx.x & 31] = v;
  __syncthreads();
  if (p0 || col >= 2 * H) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x & 31];
  float* const out = col < H ? dgamma : dbeta;
  if (!out) return;
  const int h = col < H ? col : col - H;
  out[h] = accumulate ? out[h] + v : v;
}

__global__ void __launch_bounds__(256) norm_zero_kernel(float* a, float* b, int H) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= H) return;
  if (a) a[h] = 0.f;
  if (b) b[h] = 0.f;
}

}  // namespace

// As many workgroups as the CUs hold at once by their registers: more would only
// write more parts of the weight gradients, fewer leave the memory waiting
// (16384 x 5120 bf16: 512 workgroups 136 us, 768 112, 1024 144; 16384 x 4096
// fp32: 512 149, 768 156; 8192 x 16384 bf16: 256 157, 512 176).
int norm_blocks(const NormArgs& a) {
  const bool light = a.x_type != kF32 && a.H % 8 == 0;
  const int rows = a.H <= 1024 ? 4 : 1;
  const int most = a.H <= 1024   ? 768
                   : a.H <= 4096 ? (light ? 1024 : 512)
                   : a.H <= 6144 ? (light ? 768 : 512)
                   : a.H <= 8192 ? 512
                                 : 256;
  const int need = (a.T + rows - 1) / rows;
  return need < most ? need : most;
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream) {
  if (a.T == 0) {
    if (!a.accumulate && (a.dgamma || a.dbeta))
      hipLaunchKernelGGL(norm_zero_kernel, dim3((a.H + 255) / 256), dim3(256), 0, stream, a.dgamma,
                         a.dbeta, a.H);
    return hipGetLastError();
  }
  NormArgs b = a;
  if (!a.dgamma && !a.dbeta) b.part = nullptr;
  const int blocks = norm_blocks(a);
  const auto run = [&](auto rpb, auto threads_, auto ch) {
    constexpr int RPB = decltype(rpb)::value, Threads = decltype(threads_)::value, CH = decltype(ch)::value;
    const size_t lds = RPB > 1 ? (size_t)RPB * b.H * 4 : (size_t)Threads * CH * 32;
    pick_types(b, [&](auto tx, auto ty) {
      using X = decltype(tx);
      using Y = decltype(ty);
      if (b.H % 8 == 0)
        hipLaunchKernelGGL((norm_backward_kernel<X, Y, RPB, Threads, CH, true>), dim3((unsigned)blocks),
                           dim3(Threads), lds, stream, b);
      else
        hipLaunchKernelGGL((norm_backward_kernel<X, Y, RPB, Threads, CH, false>), dim3((unsigned)blocks),
                           dim3(Threads), lds, stream, b);
    });
  };
  // a wave a row up to 1024 elements, then four waves (five need more room than
  // they have work: 5120 in two chunks a thread 176 us, in three 133), then sixteen
  if (a.H <= 512) run(IntC<4>{}, IntC<256>{}, IntC<1>{});
  else if (a.H <= 1024) run(IntC<4>{}, IntC<256>{}, IntC<2>{});
  else if (a.H <= 4096) run(IntC<1>{}, IntC<256>{}, IntC<2>{});
  else if (a.H <= 6144) run(IntC<1>{}, IntC<256>{}, IntC<3>{});
  else if (a.H <= 8192) run(IntC<1>{}, IntC<256>{}, IntC<4>{});
  else run(IntC<1>{}, IntC<1024>{}, IntC<2>{});
  if (b.part)
    hipLaunchKernelGGL(norm_columns_kernel, dim3((2 * a.H + 31) / 32), dim3(256), 0, stream, b.part,
                       blocks, a.H, a.dgamma, a.dbeta, a.accumulate);
  return hipGetLastError();
}

}  // namespace moe_fp4
