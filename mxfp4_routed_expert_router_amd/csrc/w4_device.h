// Decoding of 4-bit weights in registers, and the end of a product with them.
#pragma once

#include "block_device.h"
#include "w4.h"

namespace moe_fp4 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t __attribute__((aligned(1))) u32_byte;
typedef u32x4 __attribute__((aligned(1))) u32x4_byte;

// The two codes of byte `byte` (a constant where the call is unrolled) as 16-bit values.
template <typename T>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t v, int byte) {
  if constexpr (T::kType == kBf16) {
    switch (byte) {
      case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0));
      case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1));
      case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2));
      default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3));
    }
  } else {
    switch (byte) {
      case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 0));
      case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 1));
      case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 2));
      default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 3));
    }
  }
}
// int4 codes 0 .. 15 read as E4M3 bytes are exactly code * 2^-9 (0 to 7 as subnormals,
// 8 to 15 in the first binade): the conversion from fp8 with the factor 2^9 gives them.
template <typename T>
__device__ __forceinline__ uint32_t fp8_pair(uint32_t v, bool high) {
  if constexpr (T::kType == kBf16)
    return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.0f, true))
                : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.0f, false));
  else
    return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.0f, true))
                : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.0f, false));
}
// Eight codes, low nibble first, unscaled.
template <typename T, int Code>
__device__ __forceinline__ u32x4 decode8(uint32_t v) {
  if constexpr (Code == kMx) {
    return u32x4{fp4_pair<T>(v, 0), fp4_pair<T>(v, 1), fp4_pair<T>(v, 2), fp4_pair<T>(v, 3)};
  } else {
    const uint32_t even = v & 0x0F0F0F0Fu, odd = (v >> 4) & 0x0F0F0F0Fu;
    const uint32_t a = __builtin_amdgcn_perm(odd, even, 0x05010400u);  // codes 0 1 2 3
    const uint32_t b = __builtin_amdgcn_perm(odd, even, 0x07030602u);  // codes 4 5 6 7
    return u32x4{fp8_pair<T>(a, false), fp8_pair<T>(a, true), fp8_pair<T>(b, false), fp8_pair<T>(b, true)};
  }
}

// Two products added in fp32.
template <typename T>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  if constexpr (T::kType == kBf16)
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
  else
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
}

__device__ __forceinline__ float scalar_as_f32(const void* p, int64_t i, int type) {
  if (type == kF32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return type == kBf16 ? Bf16::to_f32(h) : F16::to_f32(h);
}
template <int Code>
__device__ __forceinline__ float scale_of(const W4Args& g, int64_t i) {
  if constexpr (Code == kMx) return ue8m0_to_f32(static_cast<const uint8_t*>(g.scales)[i]);
  else return scalar_as_f32(g.scales, i, g.scale_type);
}

// The sum of row m, column n: bias, activation, residual and accumulation in fp32, one
// rounding.
template <typename T>
__device__ __forceinline__ void finish_w4(const W4Args& g, int m, int n, float v) {
  if (g.bias) v += scalar_as_f32(g.bias, n, g.bias_type);
  v = activate(v, g.act);
  if (g.residual) v += scalar_as_f32(g.residual, m * g.ldr + n, g.out_type);
  const int64_t y = m * g.ldy + n;
  if (g.accumulate) v += scalar_as_f32(g.y, y, g.out_type);
  if (g.out_type == kF32) static_cast<float*>(g.y)[y] = v;
  else static_cast<uint16_t*>(g.y)[y] = T::from_f32(v);
}

}  // namespace moe_fp4
