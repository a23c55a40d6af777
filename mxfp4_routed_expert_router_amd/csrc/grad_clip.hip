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
// the time (one conversion and one multiply-add an element: the vector units are busy 16 %).
//
// 2.26 GB of fp32 and 1.13 GB of bf16 gradients: the norm 552 us (6.1 TB/s), clipping into other
// tensors 1300 (5.2 TB/s); 150 tensors of 145 MB in two launches each: 38 and 59 us; seven small
// ones 4.4, 1.9 for the parts' sum, and 5.4.
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
    g.e[g.n++] = GradEntry{v.data, v.out ? v.out : v.data, v.n, g.chunks, (int16_t)v.type, (int16_t)(v.out ? v.out_type : v.type)};
    g.chunks += (int32_t)c;
  }
  return g.n > 0;
}
unsigned table_blocks(const GradTable& g) { return g.chunks < kGradBlocks ? g.chunks : kGradBlocks; }

constexpr int kThreads = 256, kLoads = kChunk / 16 / kThreads;  // 16-byte loads of a thread and chunk

// A workgroup takes every gridDim.x-th chunk (neighbouring ones took 8% longer: the memory
// then has 2048 places open at a time) and searches for the tensor of its first one only.
// A thread takes the 16 bytes at 16 (256 u + thread) of a chunk.
struct Chunk {
  const char* in;
  int64_t at;  // first element
  int n;       // elements
  int entry;
};
__device__ __forceinline__ int entry_of(const GradTable& g, int c) {
  int a = 0, b = g.n - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (g.e[mid].first <= c) a = mid;
    else b = mid - 1;
  }
  return a;
}
__device__ __forceinline__ Chunk chunk_at(const GradTable& g, int c, int entry) {
  const GradEntry& e = g.e[entry];
  const int size = e.type == kF32 ? 4 : 2, per = kChunk / size;
  Chunk o;
  o.at = (int64_t)(c - e.first) * per;
  o.n = e.n - o.at < per ? (int)(e.n - o.at) : per;
  o.in = static_cast<const char*>(e.in) + o.at * size;
  o.entry = entry;
  return o;
}
// The thread's bytes, zeros past the chunk's end.
__device__ __forceinline__ void load_chunk(const GradTable& g, const Chunk& c, u32x4 (&v)[kLoads]) {
  const bool wide = g.e[c.entry].type == kF32;
  const int bytes = c.n * (wide ? 4 : 2);
  if (bytes == kChunk) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) v[u] = *reinterpret_cast<const u32x4_any*>(c.in + (u * kThreads + threadIdx.x) * 16);
    return;
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int o = (u * kThreads + threadIdx.x) * 16;
    v[u] = zero4();
    if (o + 16 <= bytes) {
      v[u] = *reinterpret_cast<const u32x4_any*>(c.in + o);
    } else if (o < bytes) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (wide) {
          if (o + 4 * i < bytes) v[u][i] = *reinterpret_cast<const uint32_t*>(c.in + o + 4 * i);
        } else {
          const uint16_t* const q = reinterpret_cast<const uint16_t*>(c.in + o + 4 * i);
          if (o + 4 * i < bytes) v[u][i] = q[0];
          if (o + 4 * i + 2 < bytes) v[u][i] |= (uint32_t)q[1] << 16;
        }
    }
  }
}
// Element r of 16 bytes.
template <typename T>
__device__ __forceinline__ float element(const u32x4& v, int r) {
  if constexpr (T::kType == kF32) return __uint_as_float(v[r]);
  else return T::to_f32((uint16_t)(v[r / 2] >> (16 * (r & 1))));
}

template <typename T>
__device__ __forceinline__ void add_squares(const u32x4 (&v)[kLoads], double (&s)[2]) {
  constexpr int V = T::kType == kF32 ? 4 : 8;
#pragma unroll
  for (int u = 0; u < kLoads; ++u)
#pragma unroll
    for (int r = 0; r < V; ++r) {
      const double d = element<T>(v[u], r);
      s[r & 1] += d * d;
    }
}

__global__ void __launch_bounds__(kThreads, 6) grad_sumsq_kernel(GradTable g, double* part) {
  __shared__ double of_wave[kThreads / 64];
  double s[2] = {0., 0.};
  int entry = entry_of(g, blockIdx.x);
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    while (entry + 1 < g.n && g.e[entry + 1].first <= c) ++entry;
    const int type = g.e[entry].type;
    u32x4 v[kLoads];
    load_chunk(g, chunk_at(g, c, entry), v);
    if (type == kF32) add_squares<F32>(v, s);
    else if (type == kBf16) add_squares<Bf16>(v, s);
    else add_squares<F16>(v, s);
  }
  const double sum = wave_sum_f64(s[0] + s[1]);
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = sum;
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
__device__ __forceinline__ void scale_chunk(const GradTable& g, const Chunk& c, const u32x4 (&v)[kLoads], float factor) {
  constexpr int V = T::kType == kF32 ? 4 : 8;
  char* const out = static_cast<char*>(g.e[c.entry].out) + c.at * (TO::kType == kF32 ? 4 : 2);
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = (u * kThreads + threadIdx.x) * V;
    if (i >= c.n) break;
    float f[V];
#pragma unroll
    for (int r = 0; r < V; ++r) f[r] = element<T>(v[u], r) * factor;
    const bool whole = i + V <= c.n;
    if constexpr (TO::kType == kF32) {
      float* const q = reinterpret_cast<float*>(out) + i;
      if (whole) __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4_word*>(q));
      else
#pragma unroll
        for (int r = 0; r < V; ++r)
          if (i + r < c.n) q[r] = f[r];
    } else {
      uint32_t h[V / 2];
#pragma unroll
      for (int r = 0; r < V / 2; ++r)
        h[r] = (uint32_t)TO::from_f32(f[2 * r]) | ((uint32_t)TO::from_f32(f[2 * r + 1]) << 16);
      uint16_t* const q = reinterpret_cast<uint16_t*>(out) + i;
      if (!whole) {
#pragma unroll
        for (int r = 0; r < V; ++r)
          if (i + r < c.n) q[r] = (uint16_t)(h[r / 2] >> (16 * (r & 1)));
      } else if constexpr (V == 4) {
        __builtin_nontemporal_store(u32x2{h[0], h[1]}, reinterpret_cast<u32x2_any*>(q));
      } else {
        __builtin_nontemporal_store(u32x4{h[0], h[1], h[2], h[3]}, reinterpret_cast<u32x4_any*>(q));
      }
    }
  }
}

// The chunks go backwards: the last ones that the norm read are still in the 256 MB cache.
__global__ void __launch_bounds__(kThreads, 6) grad_clip_kernel(GradTable g, const double* sumsq, float max_norm, float eps,
                                                             float* norm) {
  const double root = sqrt(*sumsq), over = root + (double)eps;
  const double most = over == 0. ? 1. : over == INFINITY ? 0. : (double)max_norm / over;  // also where both are inf
  const float factor = (float)(most > 1. ? 1. : most);  // NaN stays NaN
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)root;
  int entry = g.n ? entry_of(g, g.chunks - 1 - (int)blockIdx.x) : 0;
  for (int c = g.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    while (g.e[entry].first > c) --entry;
    const GradEntry& e = g.e[entry];
    if (factor == 1.f && e.in == e.out) continue;
    const Chunk chunk = chunk_at(g, c, entry);
    u32x4 v[kLoads];
    load_chunk(g, chunk, v);
    if (e.type == kF32) {
      if (e.out_type == kF32) scale_chunk<F32, F32>(g, chunk, v, factor);
      else if (e.out_type == kBf16) scale_chunk<F32, Bf16>(g, chunk, v, factor);
      else scale_chunk<F32, F16>(g, chunk, v, factor);
    } else if (e.type == kBf16) {
      scale_chunk<Bf16, Bf16>(g, chunk, v, factor);
    } else {
      scale_chunk<F16, F16>(g, chunk, v, factor);
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
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(table_blocks(g)), dim3(kThreads), 0, stream, g, part + parts);
  hipLaunchKernelGGL(grad_sumsq_finish_kernel, dim3(1), dim3(1024), 0, stream, part, parts, sumsq, accumulate);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_fp4_grad_tensor* t, int n, const double* sumsq, float max_norm, float eps,
                            float* norm, hipStream_t stream) {
  GradTable g;
  bool first = true;
  for (int at = 0; next_table(t, n, &at, g); first = false)
    hipLaunchKernelGGL(grad_clip_kernel, dim3(table_blocks(g)), dim3(kThreads), 0, stream, g, sumsq, max_norm, eps,
                       first ? norm : nullptr);
  if (first) {  // no elements: the norm alone
    g.n = g.chunks = 0;
    hipLaunchKernelGGL(grad_clip_kernel, dim3(1), dim3(kThreads), 0, stream, g, sumsq, max_norm, eps, norm);
  }
  return hipGetLastError();
}

}  // namespace moe_fp4
