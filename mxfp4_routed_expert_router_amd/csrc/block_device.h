// Device helpers of the operators around the routed experts: the two 16-bit
// types, activations and their slopes, and where a tile of a ragged product lies.
#pragma once

#include "block.h"
#include "device_common.h"

namespace moe_fp4 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  static constexpr int kType = kBf16;
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);  // to nearest, ties to even
  }
};

struct F16 {
  static constexpr int kType = kF16;
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ float to_f32(uint16_t v) {
    return (float)__builtin_bit_cast(_Float16, v);
  }
  static __device__ __forceinline__ uint16_t from_f32(float v) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);  // to nearest, ties to even
  }
};

struct F32 {
  static constexpr int kType = kF32;
};

// Element i of an array of a type known at run time (uniform over the grid).
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int type) {
  if (type == kF32) return static_cast<const float*>(p)[i];
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return type == kBf16 ? Bf16::to_f32(v) : F16::to_f32(v);
}
__device__ __forceinline__ void store_from_f32(void* p, int64_t i, int type, float v) {
  if (type == kF32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = type == kBf16 ? Bf16::from_f32(v) : F16::from_f32(v);
}

// Activations in fp32.  gelu(z) = z Phi(z) with Phi from erfc, which keeps its
// relative accuracy where Phi is small; the tanh form is z sigmoid(2 u) with
// u = sqrt(2/pi) (z + 0.044715 z^3), which is 0.5 z (1 + tanh u) without its
// cancellation.
constexpr float kRsqrt2 = 0.70710678118654752f, kRsqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f, kGeluCubic = 0.044715f;

__device__ __forceinline__ float sigmoid_f32(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    case kActGelu: return z * (0.5f * erfcf(-z * kRsqrt2));
    case kActGeluTanh:
      return z * sigmoid_f32(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
    case kActSilu: return z * sigmoid_f32(z);
    default: return z;
  }
}
__device__ __forceinline__ float activate_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;  // 0 at 0; NaN stays NaN
    case kActGelu: return 0.5f * erfcf(-z * kRsqrt2) + z * (kRsqrt2Pi * expf(-0.5f * z * z));
    case kActGeluTanh: {
      const float p = sigmoid_f32(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
      return p + z * (p * (1.0f - p)) * (2.0f * kSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z * z));
    }
    case kActSilu: {
      const float p = sigmoid_f32(z);
      return p * (1.0f + z * (1.0f - p));
    }
    default: return 1.0f;
  }
}

// Expert e's rows [lo, lo + n).  The offsets are device data that the host has
// not seen: they are held to [0, P], so that no value makes an access leave an
// array (a result for offsets that are not ascending means nothing).
__device__ __forceinline__ void segment(const int32_t* offsets, int e, int P, int& lo, int& n) {
  if (!offsets) {
    lo = 0;
    n = P;
    return;
  }
  const int a = offsets[e], b = offsets[e + 1];
  lo = a < 0 ? 0 : a > P ? P : a;
  const int hi = b < lo ? lo : b > P ? P : b;
  n = hi - lo;
}

// The experts' row tiles laid end to end, ceil(rows / BM) of each: their number.
// Every wave finds it alone, 64 experts at a time; uniform over the wave.
__device__ __forceinline__ int row_tiles(const int32_t* offsets, int E, int P, int BM) {
  if (!offsets) return (P + BM - 1) / BM;
  const int lane = threadIdx.x & 63;
  int own = 0;
  for (int e = lane; e < E; e += 64) {
    int lo, n;
    segment(offsets, e, P, lo, n);
    own += (n + BM - 1) / BM;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) own += __shfl_xor(own, d, 64);
  return __builtin_amdgcn_readfirstlane(own);
}

// Row tile `t` of them: its expert, first row and row count.  False where t is
// past the last one.
__device__ __forceinline__ bool row_tile(const int32_t* offsets, int E, int P, int BM, int t,
                                         int& e, int& row0, int& nrows) {
  if (!offsets) {
    e = 0;
    row0 = t * BM;
    nrows = P - row0 < BM ? P - row0 : BM;
    return row0 < P;
  }
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int lo = 0, n = 0;
    if (e0 + lane < E) segment(offsets, e0 + lane, P, lo, n);
    const int own = (n + BM - 1) / BM;
    int upto = own;  // tiles of this group's experts up to and with this lane's
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (t < total) {
      const int src = __ffsll((unsigned long long)__ballot(upto > t)) - 1;
      const int first = __builtin_amdgcn_readlane(upto - own, src);
      e = e0 + src;
      row0 = __builtin_amdgcn_readlane(lo, src) + (t - first) * BM;
      const int left = __builtin_amdgcn_readlane(n, src) - (t - first) * BM;
      nrows = left < BM ? left : BM;
      return true;
    }
    t -= total;
  }
  return false;
}

// Eight elements at any element's address: p[0 .. n - 1], zeros behind (n <= 0:
// nothing is read).  The hardware takes 16-byte loads at any address.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 o = zero4();
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) o[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
  return o;
}

// All eight, of data read once (weights): the caches keep it at low priority.
__device__ __forceinline__ u32x4 load8_once(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}

// Row of x that row s of the ragged side reads, or -1 for a zero row.
__device__ __forceinline__ int source_row(const ProductArgs& g, int s) {
  if (!g.rows) return s;
  const int p = g.rows[s];
  if (p < 0) return -1;
  const int r = (int)((unsigned)p / (unsigned)g.row_div);
  return r < g.R ? r : -1;
}

// Four neighbouring elements at a multiple of four, of an aligned array.
__device__ __forceinline__ f32x4 load4_as_f32(const void* p, int64_t i, int type) {
  if (type == kF32) return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
  const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  const uint16_t h[4] = {(uint16_t)v.x, (uint16_t)(v.x >> 16), (uint16_t)v.y, (uint16_t)(v.y >> 16)};
  f32x4 o;
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = type == kBf16 ? Bf16::to_f32(h[r]) : F16::to_f32(h[r]);
  return o;
}
__device__ __forceinline__ void store4_from_f32(void* p, int64_t i, int type, const f32x4& v) {
  if (type == kF32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = v;
    return;
  }
  uint32_t h[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = type == kBf16 ? Bf16::from_f32(v[r]) : F16::from_f32(v[r]);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = uint2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
}

// What a product does with the sums of one row's columns j .. j + N - 1: bias,
// the kept pre-activation, activation, residual and accumulation in fp32, then
// one rounding to the result's type.  The activation takes the sum itself, not
// its rounded copy z.
template <int N>
__device__ __forceinline__ void finish_columns(const ProductArgs& g, void* c, int64_t i, int j,
                                               const f32x4& sum) {
#pragma unroll
  for (int r = 0; r < N; ++r) {
    if (j + r >= g.J) break;
    float v = sum[r];
    if (g.bias) v += load_as_f32(g.bias, j + r, g.bias_type);
    if (g.z) store_from_f32(g.z, i * g.ldz + j + r, g.type, v);
    v = activate(v, g.act);
    if (g.residual) v += load_as_f32(g.residual, i * g.ldr + j + r, g.c_type);
    if (g.accumulate) v += load_as_f32(c, i * g.ldc + j + r, g.c_type);
    store_from_f32(c, i * g.ldc + j + r, g.c_type, v);
  }
}
// The same for four columns, in one access of each array where they allow it (g.wide).
__device__ __forceinline__ void finish4(const ProductArgs& g, void* c, int64_t i, int j,
                                        const f32x4& sum) {
  if (g.wide) {
    f32x4 v = sum;
    if (g.bias) v += load4_as_f32(g.bias, j, g.bias_type);
    if (g.z) store4_from_f32(g.z, i * g.ldz + j, g.type, v);
    if (g.act != kActNone)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = activate(v[r], g.act);
    if (g.residual) v += load4_as_f32(g.residual, i * g.ldr + j, g.c_type);
    if (g.accumulate) v += load4_as_f32(c, i * g.ldc + j, g.c_type);
    store4_from_f32(c, i * g.ldc + j, g.c_type, v);
    return;
  }
finish_columns<4>(g, c, i, j, sum);
}
__device__ __forceinline__ void* result_of(const ProductArgs& g, int e) {
  return static_cast<char*>(g.c) + (int64_t)e * g.c_stride * (g.c_type == kF32 ? 4 : 2);
}

}  // namespace moe_fp4
