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

// Terms enter the matrix instruction's sum aligned by their exponent fields: a
// value below 2^-14 is exact in its product, but the sum's step is that of 2^-14.
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

// Activations in fp32, within a few steps of it: exp and the reciprocal are the
// hardware's (one step each), an exponent's rounding adds about |exponent| half
// steps.  A sigmoid below 2^-126 is 0: silu from z = -87.3 down and tanh gelu from
// -10 down, where both are under 1e-35.
//
// The tanh form of gelu is z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3): 0.5 z
// (1 + tanh u) without its cancellation.  The exact form needs the normal
// distribution Phi(z) = 1 - Phi(-z) and, for the slope, its density, which share
// q = exp(-z^2 / 2): Phi(-u) = q R(u) for u >= 0 with R(u) = exp(u^2/2)
// erfc(u / sqrt 2) / 2, a smooth function fitted as a polynomial of degree 8 in
// t = 1 / (1 + 0.3 u) (least largest relative error, 5.8e-8, for u <= 14.5, past
// which Phi(-u) is below fp32).  No cancellation on the small side; 2e-6
// relative up to u = 6, 8e-6 up to 13.
constexpr float kLog2e = 1.4426950408889634f, kRsqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f, kGeluCubic = 0.044715f;

__device__ __forceinline__ float exp_f32(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + exp_f32(-v));
}
__device__ __forceinline__ float normal_cdf(float z, float& q) {
  const float u = fabsf(z), t = __builtin_amdgcn_rcpf(1.0f + 0.3f * u);
  q = exp_f32(-0.5f * (z * z));
  float r = 0x1.3aa226p-5f;
  r = r * t - 0x1.5abde0p-3f;
  r = r * t + 0x1.d4e4aep-3f;
  r = r * t - 0x1.3abc3ep-4f;
  r = r * t + 0x1.246220p-3f;
  r = r * t + 0x1.836c76p-4f;
  r = r * t + 0x1.f37ce0p-4f;
  r = r * t + 0x1.e96846p-4f;
  r = r * t + 0x1.eec0b4p-18f;
  const float low = q * r;
  return z < 0.0f ? low : 1.0f - low;
}
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  return sigmoid_f32(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
}

__device__ __forceinline__ float activate(float z, int act) {
  float q;
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    case kActGelu: return z * normal_cdf(z, q);
    case kActGeluTanh: return z * gelu_tanh_gate(z);
    case kActSilu: return z * sigmoid_f32(z);
    default: return z;
  }
}
// The slopes are 1 and 0 in fp32 long before |z| = 1000.  There z is held, so that
// no 0 * inf follows where z^2 passes fp32 or z is infinite (a kept fp16 z may be).
__device__ __forceinline__ float activate_slope(float z, int act) {
  if (act == kActRelu) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;  // 0 at 0; NaN stays NaN
  z = fabsf(z) > 1000.0f ? copysignf(1000.0f, z) : z;
  switch (act) {
    case kActGelu: {
      float q;
      const float p = normal_cdf(z, q);
      return p + z * (kRsqrt2Pi * q);
    }
    case kActGeluTanh: {
      const float p = gelu_tanh_gate(z);
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

// The expert that owns row tile `t` of them, its first tile and its rows [lo,
// lo + n).  False where t is past the last tile.
__device__ __forceinline__ bool tile_owner(const int32_t* offsets, int E, int P, int BM, int t, int& e, int& first,
                                           int& lo, int& n) {
  const int lane = threadIdx.x & 63;
  int before = 0;  // tiles of the groups of experts passed
  for (int e0 = 0; e0 < E; e0 += 64) {
    int l = 0, m = 0;
    if (e0 + lane < E) segment(offsets, e0 + lane, P, l, m);
    const int own = (m + BM - 1) / BM;
    int upto = own;  // tiles of this group's experts up to and with this lane's
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (t - before < total) {
      const int src = __ffsll((unsigned long long)__ballot(upto > t - before)) - 1;
      e = e0 + src;
      first = before + __builtin_amdgcn_readlane(upto - own, src);
      lo = __builtin_amdgcn_readlane(l, src);
      n = __builtin_amdgcn_readlane(m, src);
      return true;
    }
    before += total;
  }
  return false;
}

// Row tile `t` of them: its expert, first row and row count.
__device__ __forceinline__ bool row_tile(const int32_t* offsets, int E, int P, int BM, int t,
                                         int& e, int& row0, int& nrows) {
  int first = 0, lo = 0, n = P;
  e = 0;
  if (offsets && !tile_owner(offsets, E, P, BM, t, e, first, lo, n)) return false;
  row0 = lo + (t - first) * BM;
  const int left = n - (t - first) * BM;
  nrows = left < BM ? left : BM;
  return left > 0;
}

// Eight elements at any element's address: p[0 .. n - 1], zeros behind (n <= 0:
// nothing is read).  The hardware takes 16-byte loads at any address.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_word;
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 o = zero4();
  if (n > 0) {  // all loads before the first use: one wait
    uint32_t v[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) v[i] = p[i < n ? i : 0];
#pragma unroll
    for (int i = 0; i < 7; ++i) o[i / 2] |= i < n ? v[i] << (16 * (i & 1)) : 0u;
  }
  return o;
}

// All eight, of data read once (weights): the caches keep it at low priority.
__device__ __forceinline__ u32x4 load8_once(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}

// Eight elements of type T (F32, Bf16 or F16) at any element's address as fp32,
// those from n on as zeros.
template <typename T>
__device__ __forceinline__ void load8_as_f32(const void* p, int64_t i, int n, float (&v)[8]) {
  if constexpr (T::kType == kF32) {
    const float* const q = static_cast<const float*>(p) + i;
    if (n >= 8) {
      const f32x4 a = *reinterpret_cast<const f32x4_word*>(q), b = *reinterpret_cast<const f32x4_word*>(q + 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[r] = a[r];
        v[4 + r] = b[r];
      }
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = r < n ? q[r] : 0.f;
    }
  } else {
    const u32x4 a = load8(static_cast<const uint16_t*>(p) + i, n);
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = T::to_f32((uint16_t)(a[r / 2] >> (16 * (r & 1))));
  }
}

// Row of x that row s of the ragged side reads, or -1 for a zero row.
__device__ __forceinline__ int source_row(const ProductArgs& g, int s) {
  if (!g.rows) return s;
  const int p = g.rows[s];
  if (p < 0) return -1;
  const int r = (int)((unsigned)p / (unsigned)g.row_div);
  return r < g.R ? r : -1;
}

// The elements i .. i + 3 of an array, at any element's address, of which n exist:
// at once where all do (`wide`), else one by one, all loads before the first use.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
__device__ __forceinline__ f32x4 load4_as_f32(const void* p, int64_t i, int n, int type, bool wide) {
  f32x4 o;
  if (type == kF32) {
    const float* const q = static_cast<const float*>(p) + i;
    if (wide) return *reinterpret_cast<const f32x4_word*>(q);
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = q[r < n ? r : 0];
    return o;
  }
  const uint16_t* const q = static_cast<const uint16_t*>(p) + i;
  uint16_t h[4];
  if (wide) {
    const u32x2 v = *reinterpret_cast<const u32x2_any*>(q);
    h[0] = (uint16_t)v[0], h[1] = (uint16_t)(v[0] >> 16), h[2] = (uint16_t)v[1], h[3] = (uint16_t)(v[1] >> 16);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = q[r < n ? r : 0];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = type == kBf16 ? Bf16::to_f32(h[r]) : F16::to_f32(h[r]);
  return o;
}
__device__ __forceinline__ void store4_from_f32(void* p, int64_t i, int n, int type, bool wide, const f32x4& v) {
  if (type == kF32) {
    float* const q = static_cast<float*>(p) + i;
    if (wide) {
      *reinterpret_cast<f32x4_word*>(q) = v;
      return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < n) q[r] = v[r];
    return;
  }
  uint16_t* const q = static_cast<uint16_t*>(p) + i;
  uint32_t h[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = type == kBf16 ? Bf16::from_f32(v[r]) : F16::from_f32(v[r]);
  if (wide) {
    *reinterpret_cast<u32x2_any*>(q) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (r < n) q[r] = (uint16_t)h[r];
}

// What a product does with the sums of the columns j .. j + 3 of U rows (none
// where row[u] is negative; `most` columns at most): the factor, bias, the kept
// pre-activation, activation, residual and accumulation in fp32, then one
// rounding to the result's type.  The activation takes the sum itself, not its
// rounded copy z.  The rows' reads go out together, before any store.  Factor:
// whether a call may have one (compiled in where none does, it cost the bf16 rows'
// gradient of 12288 rows on 48 experts 3 of 366 us).
template <int U, bool Factor>
__device__ __forceinline__ void finish(const ProductArgs& g, void* c, const int64_t (&row)[U], int j, int most,
                                       const f32x4 (&sum)[U]) {
  const int n = g.J - j < most ? g.J - j : most;
  // of the whole wave, so that no condition stands between the reads
  const bool wide = __builtin_amdgcn_ballot_w64(n != 4) == 0;
  const f32x4 bias = g.bias ? load4_as_f32(g.bias, j, n, g.bias_type, wide) : f32x4{};
  const float factor = Factor && g.factor ? *g.factor : 1.0f;
  f32x4 more[U], old[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = row[u];
    more[u] = g.residual && i >= 0 ? load4_as_f32(g.residual, i * g.ldr + j, n, g.c_type, wide) : f32x4{};
    old[u] = g.accumulate && i >= 0 ? load4_as_f32(c, i * g.ldc + j, n, g.c_type, wide) : f32x4{};
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = row[u];
    f32x4 v = sum[u];
    if constexpr (Factor) v *= factor;
    if (g.bias) v += bias;
    if (g.z && i >= 0) store4_from_f32(g.z, i * g.ldz + j, n, g.type, wide, v);
    if (g.act != kActNone)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = activate(v[r], g.act);
    if (g.residual) v += more[u];
    if (g.accumulate) v += old[u];
    if (i >= 0) store4_from_f32(c, i * g.ldc + j, n, g.c_type, wide, v);
  }
}
template <bool Factor>
__device__ __forceinline__ void finish1(const ProductArgs& g, void* c, int64_t i, int j, int most, const f32x4& sum) {
  const int64_t row[1] = {i};
  const f32x4 sums[1] = {sum};
  finish<1, Factor>(g, c, row, j, most, sums);
}
// Sum of every eighth of a column's `parts` values from the p0-th on, `width`
// apart: eight loads in flight, added in order.
__device__ __forceinline__ float column_sum(const float* part, int64_t width, int p0, int parts) {
  float v = 0.f;
  int p = p0;
  for (; p + 56 < parts; p += 64) {
    float a[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) a[u] = part[(p + 8 * u) * width];
#pragma unroll
    for (int u = 0; u < 8; ++u) v += a[u];
  }
  for (; p < parts; p += 8) v += part[p * width];
  return v;
}
__device__ __forceinline__ void* result_of(const ProductArgs& g, int e) {
  return static_cast<char*>(g.c) + (int64_t)e * g.c_stride * (g.c_type == kF32 ? 4 : 2);
}

}  // namespace moe_fp4
