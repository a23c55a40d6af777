// The dense product of a few rows with 4-bit weights and group scales: bound by the
// weights' bytes.
//
// A workgroup takes 16 NT columns (weight rows) and 16 MT rows of x; its waves split
// the sum, 128 inputs (four groups of 32) a unit, wave w taking the units w, w + NW,
// ....  Lane l loads 16 bytes of codes of column l % 16 for group l / 16 of the unit,
// decodes them in registers and feeds them to the matrix cores as the B operand of
// 16x16x32 products, x being A: a lane then holds sums of one column, whose scale
// it can apply.  The waves' sums meet in LDS and are added in wave order.
//
// MX with bf16 x: the conversion from E2M1 takes the scale and its result is exact in
// bf16, so that the products of all groups run into one sum.  Elsewhere (fp16 does not
// hold all scales, a scaled int4 is not exact in 16 bits) a group has a sum of its own,
// which the fp32 scale multiplies; its 32 inputs must then lie in one product, and
// the four lanes of a column exchange their dwords (a 4 x 4 transposition).
// int4 codes 0 .. 15 read as E4M3 bytes are exactly code * 2^-9 (0 to 7 as subnormals,
// 8 to 15 in the first binade): the conversion from fp8 with the factor 2^9 gives them.
// The zero point is taken off the sum: sum (q - z) x = sum q x - z sum x, where sum x comes
// from a product with ones.
#include "block_device.h"
#include "w4.h"

namespace moe_fp4 {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The bytes of a row of x in one product: eight values from k on, zeros past the end.
__device__ __forceinline__ u32x4 load_x(const uint16_t* x, int k, int K, bool live) {
  return live && k < K ? *reinterpret_cast<const u32x4_any*>(x + k) : zero4();
}

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

// Dword d of the lane with quad q becomes dword q of the lane with quad d (quad: l / 16).
__device__ __forceinline__ u32x4 transpose_quads(u32x4 v) {
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float scalar_as_f32(const void* p, int64_t i, int type) {
  if (type == kF32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return type == kBf16 ? Bf16::to_f32(h) : F16::to_f32(h);
}

// Group is the inputs of a scale within a unit (32, 64 or 128; 256 takes 128's).
template <typename T, int Code, int Group, int NT, int MT, int NW, int U>
__global__ void __launch_bounds__(NW * 64) w4_kernel(W4Args g) {
  constexpr bool kScaled = Code == kMx && T::kType == kBf16;  // scales go into the conversion
  constexpr int kSums = 128 / Group;                          // scaled sums of a unit
  extern __shared__ f32x4 sums[];                             // [NW][NT][MT][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const uint8_t* w[NT];
  int64_t sc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {  // columns past the end read the last one's weights: their results are not stored
    const int n = n0 + i * 16 + l16 < g.N ? n0 + i * 16 + l16 : g.N - 1;
    w[i] = g.codes + n * g.ldw;
    sc[i] = (int64_t)n * g.groups;
  }
  const uint16_t* x[MT];
  bool live[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    live[j] = m0 + j * 16 + l16 < g.M;
    x[j] = g.x + (int64_t)(live[j] ? m0 + j * 16 + l16 : 0) * g.ldx;
  }
  f32x4 acc[NT][MT] = {};
  const int units = (g.K + 127) / 128;
  for (int u0 = wave; u0 < units; u0 += NW * U) {
    u32x4 codes[U][NT];
    float scale[U][NT][kScaled ? 1 : kSums], zero[U][NT][kSums];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (u0 + u * NW) * 128 + quad * 32;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        codes[u][i] = k < g.K ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w[i] + k / 2)) : zero4();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (u0 + u * NW) * 128;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if constexpr (kScaled) {
          const int at = k / 32 + quad < g.groups ? k / 32 + quad : 0;
          scale[u][i][0] = ue8m0_to_f32(static_cast<const uint8_t*>(g.scales)[sc[i] + at]);
        } else {
#pragma unroll
          for (int s = 0; s < kSums; ++s) {
            const int of = (k + s * Group) / g.group, at = of < g.groups ? of : 0;
            if constexpr (Code == kMx) {
              scale[u][i][s] = ue8m0_to_f32(static_cast<const uint8_t*>(g.scales)[sc[i] + at]);
            } else {
              scale[u][i][s] = scalar_as_f32(g.scales, sc[i] + at, g.scale_type);
              zero[u][i][s] = g.zeros ? (float)g.zeros[sc[i] + at] : 8.0f;
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = (u0 + u * NW) * 128;
      if (k0 >= g.K) break;
      if constexpr (kScaled) {
        // product d takes dword d of every lane: inputs k0 + 32 quad + 8 d ..
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          u32x4 fx[MT];
#pragma unroll
          for (int j = 0; j < MT; ++j) fx[j] = load_x(x[j], k0 + quad * 32 + d * 8, g.K, live[j]);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const u32x4 b = __builtin_bit_cast(u32x4, fp4x8_to_bf16x8(codes[u][i][d], scale[u][i][0]));
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = T::mfma(fx[j], b, acc[i][j]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) codes[u][i] = transpose_quads(codes[u][i]);
#pragma unroll
        for (int s = 0; s < kSums; ++s) {
          f32x4 part[NT][MT] = {}, sx[MT] = {};
#pragma unroll
          for (int d = s * Group / 32; d < (s + 1) * Group / 32; ++d) {  // product d: inputs k0 + 32 d + 8 quad ..
            u32x4 fx[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) fx[j] = load_x(x[j], k0 + d * 32 + quad * 8, g.K, live[j]);
            if constexpr (Code == kInt4) {
              const uint32_t one = T::kType == kBf16 ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
              for (int j = 0; j < MT; ++j) sx[j] = T::mfma(fx[j], u32x4{one, one, one, one}, sx[j]);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const u32x4 b = decode8<T, Code>(codes[u][i][d]);
#pragma unroll
              for (int j = 0; j < MT; ++j) part[i][j] = T::mfma(fx[j], b, part[i][j]);
            }
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              f32x4 v = part[i][j];
              if constexpr (Code == kInt4) v -= zero[u][i][s] * sx[j];
              acc[i][j] += scale[u][i][s] * v;
            }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) sums[((wave * NT + i) * MT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // thread -> column n0 + 16 i + c, row m0 + 16 j + r; lane 16 (r / 4) + c held it in component r % 4
  const float* const f = reinterpret_cast<const float*>(sums);
  for (int o = threadIdx.x; o < NT * MT * 256; o += NW * 64) {
    const int c = o & 15, i = (o >> 4) % NT, r16 = (o >> 4) / NT, r = r16 & 15, j = r16 >> 4;
    const int m = m0 + j * 16 + r, n = n0 + i * 16 + c;
    if (m >= g.M || n >= g.N) continue;
    const int at = ((i * MT + j) * 64 + 16 * (r >> 2) + c) * 4 + (r & 3);
    float v = f[at];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += f[at + q * NT * MT * 256];
    if (g.bias) v += scalar_as_f32(g.bias, n, g.bias_type);
    v = activate(v, g.act);
    if (g.residual) v += scalar_as_f32(g.residual, m * g.ldr + n, g.out_type);
    const int64_t y = m * g.ldy + n;
    if (g.accumulate) v += scalar_as_f32(g.y, y, g.out_type);
    if (g.out_type == kF32) static_cast<float*>(g.y)[y] = v;
    else static_cast<uint16_t*>(g.y)[y] = T::from_f32(v);
  }
}

template <typename T, int Code, int Group, int NT, int MT, int NW, int U>
void launch_tiles(const W4Args& a, hipStream_t stream) {
  const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * MT - 1) / (16 * MT));
  hipLaunchKernelGGL((w4_kernel<T, Code, Group, NT, MT, NW, U>), grid, dim3(NW * 64), NW * NT * MT * 1024, stream, a);
}

template <typename T, int Code, int Group>
void launch_rows(const W4Args& a, hipStream_t stream) {
  if (a.M <= 16) launch_tiles<T, Code, Group, 1, 1, 8, 2>(a, stream);
  else launch_tiles<T, Code, Group, 2, 4, 8, 1>(a, stream);
}

template <typename T>
void launch_type(const W4Args& a, hipStream_t stream) {
  if (a.code == kMx) launch_rows<T, kMx, 32>(a, stream);
  else if (a.group == 32) launch_rows<T, kInt4, 32>(a, stream);
  else if (a.group == 64) launch_rows<T, kInt4, 64>(a, stream);
  else launch_rows<T, kInt4, 128>(a, stream);
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t stream) {
  if (a.type == kBf16) launch_type<Bf16>(a, stream);
  else launch_type<F16>(a, stream);
  return hipGetLastError();
}

}  // namespace moe_fp4
