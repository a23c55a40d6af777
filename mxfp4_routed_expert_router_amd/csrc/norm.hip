// Layer norm and RMS norm with weights, forward and backward.
//
//   mean = sum_h x / H (RMS: 0),  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   xhat = (x - mean) rstd,       y = xhat gamma + beta
//   g = dy gamma,  dx = rstd (g - mean_h(g) [RMS: not] - xhat mean_h(g xhat))
//   dgamma = sum_t dy xhat,  dbeta = sum_t dy
//
// Both passes are bound by memory: a row is read once into registers, its sums
// are taken from there (the variance from the centred values, so a mean far
// from zero costs no digits), and the result is written once.  All sums are
// fp32 in a fixed order: the same inputs give the same bits.
#include "block_device.h"

namespace moe_fp4 {
namespace {

// Chunks of V elements of a row, as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_chunk(const void* p, int64_t i, float (&v)[V]) {
  if constexpr (T::kType == kF32) {
    const float* q = static_cast<const float*>(p) + i;
    if constexpr (V == 8) {
      const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = q[0];
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if constexpr (V == 8) {
      const u32x4 a = ld16(q);
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = T::to_f32((uint16_t)(a[r / 2] >> (16 * (r & 1))));
    } else {
      v[0] = T::to_f32(q[0]);
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, const float (&v)[V]) {
  if constexpr (T::kType == kF32) {
    float* q = static_cast<float*>(p) + i;
    if constexpr (V == 8) {
      *reinterpret_cast<float4*>(q) = float4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<float4*>(q + 4) = float4{v[4], v[5], v[6], v[7]};
    } else {
      q[0] = v[0];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (V == 8) {
      u32x4 a;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        a[r] = (uint32_t)T::from_f32(v[2 * r]) | ((uint32_t)T::from_f32(v[2 * r + 1]) << 16);
      st16(q, a);
    } else {
      q[0] = T::from_f32(v[0]);
    }
  }
}
// The weights' type is a run-time choice (one load per workgroup and chunk).
template <int V>
__device__ __forceinline__ void load_weight(const void* p, int type, int i, float one, float (&v)[V]) {
  if (!p) {
#pragma unroll
    for (int r = 0; r < V; ++r) v[r] = one;
  } else if (type == kF32) {
    load_chunk<F32, V>(p, i, v);
  } else if (type == kBf16) {
    load_chunk<Bf16, V>(p, i, v);
  } else {
    load_chunk<F16, V>(p, i, v);
  }
}

// Sum over the TPR threads of a row, returned to all of them: within each wave
// by wave_sum_f32, then the waves' sums in wave order.  `slot`: one float per
// wave of the workgroup; barriers only where a row has several waves.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum_f32(v);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    lds_barrier();  // the previous sum's reads are done
    if ((threadIdx.x & 63) == 0) slot[wave] = v;
    lds_barrier();
    const int first = wave / W * W;
    v = slot[first];
#pragma unroll
    for (int i = 1; i < W; ++i) v += slot[first + i];
  }
  return v;
}

constexpr int norm_threads(int TPR) { return TPR < 256 ? 256 : TPR; }

// TPR threads a row, V elements a load, up to CH loads a thread.
template <typename TX, typename TY, int TPR, int V, int CH>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_kernel(NormArgs g) {
  constexpr int RPB = norm_threads(TPR) / TPR;
  __shared__ float slot[norm_threads(TPR) / 64];
  const int lt = threadIdx.x % TPR, nc = g.H / V;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int64_t rr = row < g.T ? row : g.T - 1;  // a workgroup's threads stay together at its barriers
  float x[CH][V];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lt + c * TPR;
    if (k < nc) load_chunk<TX, V>(g.x, rr * g.ldx + (int64_t)k * V, x[c]);
  }
  float mean = 0.f;
  if (!g.rms) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lt + c * TPR < nc)
#pragma unroll
        for (int r = 0; r < V; ++r) s += x[c][r];
    mean = row_sum<TPR>(s, slot) / (float)g.H;
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (lt + c * TPR < nc)
#pragma unroll
      for (int r = 0; r < V; ++r) {
        x[c][r] -= mean;
        ss += x[c][r] * x[c][r];
      }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(ss, slot) / (float)g.H + g.eps);
  if (row >= g.T) return;
  if (lt == 0) {
    if (g.mean) g.mean[row] = mean;
    if (g.rstd) g.rstd[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lt + c * TPR;
    if (k >= nc) break;
    float w[V], b[V];
    load_weight<V>(g.gamma, g.w_type, k * V, 1.0f, w);
    load_weight<V>(g.beta, g.w_type, k * V, 0.0f, b);
#pragma unroll
    for (int r = 0; r < V; ++r) w[r] = x[c][r] * rstd * w[r] + b[r];
    store_chunk<TY, V>(g.y, row * g.ldy + (int64_t)k * V, w);
  }
}

// The workgroups walk the rows; a thread keeps its columns' gamma and the sums
// of dgamma and dbeta over the rows it has seen, and writes them once at the
// end to part[workgroup], which norm_columns_kernel adds up.
template <typename TX, typename TY, int TPR, int V, int CH>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_backward_kernel(NormArgs g) {
  constexpr int RPB = norm_threads(TPR) / TPR;
  __shared__ float slot[norm_threads(TPR) / 64];
  extern __shared__ float sums[];  // RPB > 1: [RPB][H], one gradient at a time
  const int lt = threadIdx.x % TPR, sub = threadIdx.x / TPR, nc = g.H / V;
  float w[CH][V], dw[CH][V] = {}, db[CH][V] = {};
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (lt + c * TPR < nc) load_weight<V>(g.gamma, g.w_type, (lt + c * TPR) * V, 1.0f, w[c]);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < g.T; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + sub;
    const bool live = row < g.T;
    const int64_t rr = live ? row : g.T - 1;
    float x[CH][V], d[CH][V];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = lt + c * TPR;
      if (k < nc) {
        load_chunk<TX, V>(g.x, rr * g.ldx + (int64_t)k * V, x[c]);
        load_chunk<TY, V>(g.dy, rr * g.ldy + (int64_t)k * V, d[c]);
      }
    }
    const float mean = g.rms ? 0.f : g.mean_in[rr], rstd = g.rstd_in[rr];
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lt + c * TPR < nc)
#pragma unroll
        for (int r = 0; r < V; ++r) {
          x[c][r] = (x[c][r] - mean) * rstd;
          if (live) {
            dw[c][r] += d[c][r] * x[c][r];
            db[c][r] += d[c][r];
          }
          d[c][r] *= w[c][r];
          sg += d[c][r];
          sgx += d[c][r] * x[c][r];
        }
    const float mg = g.rms ? 0.f : row_sum<TPR>(sg, slot) / (float)g.H;
    const float mgx = row_sum<TPR>(sgx, slot) / (float)g.H;
    if (live && g.dx)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = lt + c * TPR;
        if (k >= nc) break;
        float o[V];
#pragma unroll
        for (int r = 0; r < V; ++r) o[r] = rstd * (d[c][r] - mg - x[c][r] * mgx);
        store_chunk<TX, V>(g.dx, row * g.lddx + (int64_t)k * V, o);
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
          for (int r = 0; r < V; ++r)
            sums[sub * g.H + (lt + c * TPR) * V + r] = which ? db[c][r] : dw[c][r];
      __syncthreads();
      for (int h = threadIdx.x; h < g.H; h += norm_threads(TPR)) {
        float s = sums[h];
#pragma unroll
        for (int i = 1; i < RPB; ++i) s += sums[i * g.H + h];
        part[which * g.H + h] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (lt + c * TPR < nc)
          store_chunk<F32, V>(part, which * g.H + (lt + c * TPR) * V, which ? db[c] : dw[c]);
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
    for (int p = p0; p < parts; p += 8) v += part[(int64_t)p * 2 * H + col];
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

bool wide_ok(const void* p, int64_t ld, int type) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * (type == kF32 ? 4 : 2)) % 16 == 0;
}

// Threads per row: a wave up to 2048 (wide) or 1024 elements, 256 up to 8192 or
// 4096, 1024 above; at most CH loads of V elements a thread.
template <bool BWD, typename TX, typename TY, int TPR, int V, int CH>
void launch_shape(const NormArgs& a, unsigned blocks, hipStream_t s) {
  constexpr int threads = norm_threads(TPR), RPB = threads / TPR;
  if constexpr (BWD)
    hipLaunchKernelGGL((norm_backward_kernel<TX, TY, TPR, V, CH>), dim3(blocks), dim3(threads),
                       RPB > 1 ? (size_t)RPB * a.H * 4 : 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<TX, TY, TPR, V, CH>), dim3((unsigned)((a.T + RPB - 1) / RPB)),
                       dim3(threads), 0, s, a);
}
template <bool BWD, typename TX, typename TY>
void launch_types(const NormArgs& a, bool wide, unsigned blocks, hipStream_t s) {
  if (wide) {
    if (a.H <= 2048) return launch_shape<BWD, TX, TY, 64, 8, 4>(a, blocks, s);
    if (a.H <= 8192) return launch_shape<BWD, TX, TY, 256, 8, 4>(a, blocks, s);
    return launch_shape<BWD, TX, TY, 1024, 8, 2>(a, blocks, s);
  }
  if (a.H <= 1024) return launch_shape<BWD, TX, TY, 64, 1, 16>(a, blocks, s);
  if (a.H <= 4096) return launch_shape<BWD, TX, TY, 256, 1, 16>(a, blocks, s);
  return launch_shape<BWD, TX, TY, 1024, 1, 16>(a, blocks, s);
}
template <bool BWD>
void launch_norm_any(const NormArgs& a, bool wide, unsigned blocks, hipStream_t s) {
  if (a.x_type == kBf16) return launch_types<BWD, Bf16, Bf16>(a, wide, blocks, s);
  if (a.x_type == kF16) return launch_types<BWD, F16, F16>(a, wide, blocks, s);
  if (a.y_type == kBf16) return launch_types<BWD, F32, Bf16>(a, wide, blocks, s);
  if (a.y_type == kF16) return launch_types<BWD, F32, F16>(a, wide, blocks, s);
  return launch_types<BWD, F32, F32>(a, wide, blocks, s);
}

}  // namespace

int norm_blocks(int T, int) { return T < 512 ? T : 512; }

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const bool wide = a.H % 8 == 0 && wide_ok(a.x, a.ldx, a.x_type) && wide_ok(a.y, a.ldy, a.y_type) &&
                    wide_ok(a.gamma, 0, a.w_type) && wide_ok(a.beta, 0, a.w_type);
  launch_norm_any<false>(a, wide, 0, stream);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream) {
  if (a.T == 0) {
    if (!a.accumulate && (a.dgamma || a.dbeta))
      hipLaunchKernelGGL(norm_zero_kernel, dim3((a.H + 255) / 256), dim3(256), 0, stream, a.dgamma,
                         a.dbeta, a.H);
    return hipGetLastError();
  }
  const bool wide = a.H % 8 == 0 && wide_ok(a.x, a.ldx, a.x_type) && wide_ok(a.dy, a.ldy, a.y_type) &&
                    wide_ok(a.dx, a.lddx, a.x_type) && wide_ok(a.gamma, 0, a.w_type);
  NormArgs b = a;
  if (!a.dgamma && !a.dbeta) b.part = nullptr;
  const int blocks = norm_blocks(a.T, a.H);
  launch_norm_any<true>(b, wide, (unsigned)blocks, stream);
  if (b.part)
    hipLaunchKernelGGL(norm_columns_kernel, dim3((2 * a.H + 31) / 32), dim3(256), 0, stream, b.part,
                       blocks, a.H, a.dgamma, a.dbeta, a.accumulate);
  return hipGetLastError();
}

}  // namespace moe_fp4
