// The global norm of many gradients, and clipping by it.
//
//   sumsq = sum over all elements of g^2,  norm = sqrt(sumsq)
//   factor = min(1, max_norm / (norm + eps)),  out = g factor
//
// Both passes are streams, bound by the bytes.  The tensors' addresses travel in
// the kernel's arguments (kTable of them a launch), so that a call needs no copy
// to the device and can be captured.  A workgroup takes chunks of kChunk bytes of
// one tensor each.  Squares are taken and summed in fp64: in fp32 those of values
// below 2^-75 would vanish and those above 2^64 overflow, and the 64-bit unit has
// the time (one conversion and one multiply-add an element, a third of what the
// memory leaves it).
#include "block_device.h"
#include "grad_clip.h"

namespace moe_fp4 {
namespace {

constexpr int kTable = 112, kChunk = 32768, kGradBlocks = 2048;

struct GradEntry {
  const void* in;
  void* out;
  int64_t n;
  int32_t first;  // the tensor's first chunk of the launch
  int16_t type, out_type;
};
struct GradTable {
  int32_t n, chunks;
  GradEntry e[kTable];
};
static_assert(sizeof(GradTable) <= 4096 - 64, "kernel arguments");

int64_t chunk_elements(int type) { return kChunk / (type == kF32 ? 4 : 2); }

// The tensors from *at on that fit one launch; false where none is left.
bool next_table(const moe_fp4_grad_tensor* t, int n, int* at, GradTable& g) {
  g.n = 0;
  g.chunks = 0;
  for (; *at < n && g.n < kTable; ++*at) {
    const moe_fp4_grad_tensor& v = t[*at];
    if (v.n == 0) continue;
    const int64_t c = (v.n + chunk_elements(v.type) - 1) / chunk_elements(v.type);  // 2^27 at most
    if (g.chunks > (1 << 30)) break;
    g.e[g.n++] = GradEntry{v.data, v.out ? v.out : v.data, v.n, g.chunks, (int16_t)v.type, (int16_t)v.out_type};
    g.chunks += (int32_t)c;
  }
  return g.n > 0;
}
unsigned table_blocks(const GradTable& g) { return g.chunks < kGradBlocks ? g.chunks : kGradBlocks; }

// The tensor of chunk c, and its elements [lo, lo + n) of it.
__device__ __forceinline__ const GradEntry& chunk_of(const GradTable& g, int c, int64_t& lo, int& n) {
  int a = 0, b = g.n - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (g.e[mid].first <= c) a = mid;
    else b = mid - 1;
  }
  const GradEntry& e = g.e[a];
  const int per = kChunk / (e.type == kF32 ? 4 : 2);
  lo = (int64_t)(c - e.first) * per;
  n = e.n - lo < per ? (int)(e.n - lo) : per;
  return e;
}

constexpr int kLoads = kChunk / 16 / 256;  // 16-byte loads of a thread and chunk

template <typename T>
__device__ __forceinline__ double squares_of_chunk(const void* p, int64_t lo, int n) {
  constexpr int V = T::kType == kF32 ? 4 : 8;
  double s[2] = {0., 0.};
  const int i0 = threadIdx.x * V;
  if (n == kLoads * 256 * V) {
    u32x4 v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      v[u] = *reinterpret_cast<const u32x4_any*>(static_cast<const char*>(p) + (lo + i0 + u * 256 * V) * (16 / V));
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll
      for (int r = 0; r < V; ++r) {
        float f;
        if constexpr (T::kType == kF32) f = __uint_as_float(v[u][r]);
        else f = T::to_f32((uint16_t)(v[u][r / 2] >> (16 * (r & 1))));
        const double d = f;
        s[r & 1] += d * d;
      }
  } else {
    for (int i = i0; i < n; i += 256 * V)
#pragma unroll
      for (int r = 0; r < V; ++r)
        if (i + r < n) {
          float f;
          if constexpr (T::kType == kF32) f = static_cast<const float*>(p)[lo + i + r];
          else f = T::to_f32(static_cast<const uint16_t*>(p)[lo + i + r]);
          const double d = f;
          s[r & 1] += d * d;
        }
  }
  return s[0] + s[1];
}

__global__ void __launch_bounds__(256) grad_sumsq_kernel(GradTable g, double* part) {
  __shared__ double of_wave[4];
  double s = 0.;
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    int64_t lo;
    int n;
    const GradEntry& e = chunk_of(g, c, lo, n);
    if (e.type == kF32) s += squares_of_chunk<F32>(e.in, lo, n);
    else if (e.type == kBf16) s += squares_of_chunk<Bf16>(e.in, lo, n);
    else s += squares_of_chunk<F16>(e.in, lo, n);
  }
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = ((of_wave[0] + of_wave[1]) + of_wave[2]) + of_wave[3];
}

__global__ void __launch_bounds__(1024) grad_sumsq_finish_kernel(const double* part, int parts, double* sumsq, int accumulate) {
  __shared__ double of_wave[16];
  double s = 0.;
  for (int i = threadIdx.x; i < parts; i += 1024) s += part[i];
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 16; ++w) s += of_wave[w];
  *sumsq = accumulate ? *sumsq + s : s;
}

// The product is rounded to fp32, and for a 16-bit result once more.
template <typename T, typename TO>
__device__ __forceinline__ void chunk_clip(const void* p, void* out, int64_t lo, int n, float factor) {
  constexpr int V = T::kType == kF32 ? 4 : 8;
  const int i0 = threadIdx.x * V;
  const auto one = [&](int i) {
    float f;
    if constexpr (T::kType == kF32) f = static_cast<const float*>(p)[lo + i];
    else f = T::to_f32(static_cast<const uint16_t*>(p)[lo + i]);
    f *= factor;
    if constexpr (TO::kType == kF32) static_cast<float*>(out)[lo + i] = f;
    else static_cast<uint16_t*>(out)[lo + i] = TO::from_f32(f);
  };
  if (n == kLoads * 256 * V) {
    u32x4 v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      v[u] = *reinterpret_cast<const u32x4_any*>(static_cast<const char*>(p) + (lo + i0 + u * 256 * V) * (16 / V));
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float f[V];
#pragma unroll
      for (int r = 0; r < V; ++r) {
        if constexpr (T::kType == kF32) f[r] = __uint_as_float(v[u][r]);
        else f[r] = T::to_f32((uint16_t)(v[u][r / 2] >> (16 * (r & 1))));
        f[r] *= factor;
      }
      const int64_t at = lo + i0 + u * 256 * V;
      if constexpr (TO::kType == kF32) {
        *reinterpret_cast<f32x4_word*>(static_cast<float*>(out) + at) = f32x4{f[0], f[1], f[2], f[3]};
      } else {
        uint32_t h[V / 2];
#pragma unroll
        for (int r = 0; r < V / 2; ++r)
          h[r] = (uint32_t)TO::from_f32(f[2 * r]) | ((uint32_t)TO::from_f32(f[2 * r + 1]) << 16);
        uint16_t* const q = static_cast<uint16_t*>(out) + at;
        if constexpr (V == 4) *reinterpret_cast<u32x2_any*>(q) = u32x2{h[0], h[1]};
        else *reinterpret_cast<u32x4_any*>(q) = u32x4{h[0], h[1], h[2], h[3]};
      }
    }
  } else {
    for (int i = i0; i < n; i += 256 * V)
#pragma unroll
      for (int r = 0; r < V; ++r)
        if (i + r < n) one(i + r);
  }
}

__global__ void __launch_bounds__(256) grad_clip_kernel(GradTable g, const double* sumsq, float max_norm, float eps,
                                                        float* norm) {
  const double root = sqrt(*sumsq), most = (double)max_norm / (root + (double)eps);
  const float factor = (float)(most > 1. ? 1. : most);  // NaN stays NaN
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    int64_t lo;
    int n;
    const GradEntry& e = chunk_of(g, c, lo, n);
    if (factor == 1.f && e.in == e.out) continue;
    if (e.type == kF32) {
      if (e.out_type == kF32) chunk_clip<F32, F32>(e.in, e.out, lo, n, factor);
      else if (e.out_type == kBf16) chunk_clip<F32, Bf16>(e.in, e.out, lo, n, factor);
      else chunk_clip<F32, F16>(e.in, e.out, lo, n, factor);
    } else if (e.type == kBf16) {
      chunk_clip<Bf16, Bf16>(e.in, e.out, lo, n, factor);
    } else {
      chunk_clip<F16, F16>(e.in, e.out, lo, n, factor);
    }
  }
}

}  // namespace

size_t grad_sumsq_workspace(const moe_fp4_grad_tensor* t, int n) {
  size_t blocks = 0;
  GradTable g;
  for (int at = 0; next_table(t, n, &at, g);) blocks += table_blocks(g);
  return blocks * sizeof(double);
}

hipError_t launch_grad_sumsq(const moe_fp4_grad_tensor* t, int n, double* sumsq, int accumulate, void* ws,
                             hipStream_t stream) {
  double* const part = static_cast<double*>(ws);
  int parts = 0;
  GradTable g;
  for (int at = 0; next_table(t, n, &at, g); parts += table_blocks(g))
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(table_blocks(g)), dim3(256), 0, stream, g, part + parts);
  hipLaunchKernelGGL(grad_sumsq_finish_kernel, dim3(1), dim3(1024), 0, stream, part, parts, sumsq, accumulate);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_fp4_grad_tensor* t, int n, const double* sumsq, float max_norm, float eps,
                            float* norm, hipStream_t stream) {
  GradTable g;
  bool first = true;
  for (int at = 0; next_table(t, n, &at, g); first = false)
    hipLaunchKernelGGL(grad_clip_kernel, dim3(table_blocks(g)), dim3(256), 0, stream, g, sumsq, max_norm, eps,
                       first ? norm : nullptr);
  if (first) {  // no elements: the norm alone
    g.n = g.chunks = 0;
    hipLaunchKernelGGL(grad_clip_kernel, dim3(1), dim3(256), 0, stream, g, sumsq, max_norm, eps, norm);
  }
  return hipGetLastError();
}

}  // namespace moe_fp4
