// Layer norm and RMS norm with weights, forward and backward.
//
//   mean = sum_h x / H (RMS: 0),  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   xhat = (x - mean) rstd,       y = xhat gamma + beta
//   g = dy gamma,  dx = rstd (g - mean_h(g) [RMS: not] - xhat mean_h(g xhat))
//   dgamma = sum_t dy xhat,  dbeta = sum_t dy
//
// Both passes are bound by memory: a row is read once into registers, its sums
// are taken from there, and the result is written once.  The forward pass takes the
// deviations from a first mean, and their own mean corrects them, the mean and the
// variance: the first mean is off by a few steps of itself, up to 0.25 in a row
// of 1e6, which would be all the deviation that a row of one value shows (y = 1
// where it is 0).  16384 x 5120 bf16 takes 64.5 us with that, 63.8 without.  All
// sums are fp32 in a fixed order: the same inputs give the same bits.
#pragma once

#include "block_device.h"

namespace moe_fp4 {
namespace {

// Eight elements of a row at any element's address, n of them in it (zeros
// behind): as loaded, for values that arrive later, and as fp32.
template <typename T>
struct Chunk {
  u32x4 a[T::kType == kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    if constexpr (T::kType == kF32) {
      typedef u32x4 __attribute__((aligned(4))) u32x4_word;
      const uint32_t* const q = static_cast<const uint32_t*>(p) + i;
      if (n >= 8) {
        a[0] = *reinterpret_cast<const u32x4_word*>(q);
        a[1] = *reinterpret_cast<const u32x4_word*>(q + 4);
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint32_t v = q[r < n ? r : 0];
          a[r / 4][r % 4] = r < n ? v : 0u;
        }
      }
    } else {
      a[0] = load8(static_cast<const uint16_t*>(p) + i, n);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if constexpr (T::kType == kF32) {
        const uint32_t w = a[r / 4][r % 4];
        v[r] = __uint_as_float(w);
      } else {
        v[r] = T::to_f32((uint16_t)(a[0][r / 2] >> (16 * (r & 1))));
      }
    }
  }
};
// kPast: the store passes the L2 (non-temporal).  It pays where a row is read and
// written once: 16384 x 5120 bf16 forward 65.1 us, 67.2 without (x 2304 37.4 either
// way).  In the backward pass it does not: f32 rows of 4096 147 -> 158 us.
template <typename T, bool kPast>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, int n, const float (&v)[8]) {
  if constexpr (T::kType == kF32) {
    float* const q = static_cast<float*>(p) + i;
    if (n >= 8) {
      const f32x4 a{v[0], v[1], v[2], v[3]}, b{v[4], v[5], v[6], v[7]};
      if constexpr (kPast) {
        __builtin_nontemporal_store(a, reinterpret_cast<f32x4_word*>(q));
        __builtin_nontemporal_store(b, reinterpret_cast<f32x4_word*>(q + 4));
      } else {
        *reinterpret_cast<f32x4_word*>(q) = a;
        *reinterpret_cast<f32x4_word*>(q + 4) = b;
      }
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < n) q[r] = v[r];
    }
  } else {
    uint16_t* const q = static_cast<uint16_t*>(p) + i;
    if (n >= 8) {
      u32x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        o[r] = (uint32_t)T::from_f32(v[2 * r]) | ((uint32_t)T::from_f32(v[2 * r + 1]) << 16);
      if constexpr (kPast) __builtin_nontemporal_store(o, reinterpret_cast<u32x4_any*>(q));
      else *reinterpret_cast<u32x4_any*>(q) = o;
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < n) q[r] = T::from_f32(v[r]);
    }
  }
}
// The weights' type is a run-time choice (one load per workgroup and chunk).
__device__ __forceinline__ void load_weight(const void* p, int type, int i, int n, float one, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = one;
  } else if (type == kF32) {
    load8_as_f32<F32>(p, i, n, v);
  } else if (type == kBf16) {
    load8_as_f32<Bf16>(p, i, n, v);
  } else {
    load8_as_f32<F16>(p, i, n, v);
  }
}

// Sums of N values over a wave, or with Block over the workgroup's waves in wave
// order (two at least), returned to all threads.  `slot`: N floats a wave, used
// once between two barriers; one barrier inside.
template <bool Block, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slot) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum_f32(v[n]);
  if constexpr (Block) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) slot[(threadIdx.x >> 6) * N + n] = v[n];
    lds_barrier();
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = slot[n];
    for (int i = 1; i < waves; ++i)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += slot[i * N + n];
  }
}

constexpr int norm_threads(int TPR) { return TPR < 256 ? 256 : TPR; }

// Threads and loads a row: the fewest threads, a wave at least, that hold it in
// registers.  Whole: the width is a multiple of eight, so no chunk ends early.
template <typename F>
void pick_shape(int H, F&& f) {
  const auto whole = [&](auto tpr, auto ch) {
    if (H % 8 == 0) return f(tpr, ch, IntC<1>{});
    return f(tpr, ch, IntC<0>{});
  };
  if (H <= 512) return whole(IntC<64>{}, IntC<1>{});
  if (H <= 1024) return whole(IntC<64>{}, IntC<2>{});
  if (H <= 2048) return whole(IntC<64>{}, IntC<4>{});
  if (H <= 4096) return whole(IntC<256>{}, IntC<2>{});
  if (H <= 6144) return whole(IntC<256>{}, IntC<3>{});
  if (H <= 8192) return whole(IntC<256>{}, IntC<4>{});
  return whole(IntC<1024>{}, IntC<2>{});
}
template <typename F>
void pick_types(const NormArgs& a, F&& f) {
  if (a.x_type == kBf16) return f(Bf16{}, Bf16{});
  if (a.x_type == kF16) return f(F16{}, F16{});
  if (a.y_type == kBf16) return f(F32{}, Bf16{});
  if (a.y_type == kF16) return f(F32{}, F16{});
  return f(F32{}, F32{});
}

}  // namespace
}  // namespace moe_fp4
