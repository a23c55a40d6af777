// The dense product of a few rows with 4-bit weights and group scales: bound by the
// weights' bytes.
//
// A workgroup takes 16 NT columns (weight rows) and 16 MT rows of x; its waves split
// the sum, each taking neighbouring units of 128 inputs (four groups of 32).  Loads go
// out as memory lies: four lanes read 64 bytes of codes of a column, sixteen 256 bytes of a
// row of x (in the matrix instruction's own order, neighbouring lanes in different
// rows, a load took four times as long).  They pass through the wave's own corner of
// LDS into 16x16x32 products, x as A and the codes, decoded in registers, as B: a lane
// then holds sums of one column, whose scale it can apply, and a product takes one group.
// The next unit's loads are on their way while one is computed.  The waves' sums meet in
// LDS and are added in wave order.
//
// 16 rows of 5120 x 9216, int4: 16.5 us where the weights' 24 MB take 5: 160 workgroups read
// 47 MB of x from the L2 besides, and a wave's nine units follow one another.
//
// MX with bf16 x: the conversion from E2M1 takes the scale and its result is exact in
// bf16, so that the products of all groups run into one sum.  Elsewhere (fp16 does not
// hold all scales, a scaled int4 is not exact in 16 bits) a scale's inputs have a sum of
// their own, which the fp32 scale multiplies.  The zero point is taken off that sum:
// sum (q - z) x = sum q x - z sum x, where sum x comes from a product with ones.
#include "w4_device.h"

namespace moe_fp4 {
namespace {

// A wave's corner of LDS, bytes: the codes (64 a column, the 16-byte chunk c of column r
// at chunk c ^ (r / 4) % 4), the rows of x (256 each, chunk c of row r at c ^ r), scales
// and zeros as fp32 (16 a column).  Neither writes nor reads meet in a bank.
template <int NT, int MT>
struct Corner {
  static constexpr int kCodes = 0, kX = NT * 1024, kScale = kX + MT * 4096, kZero = kScale + NT * 256,
                       kBytes = kZero + NT * 256;
};

// Group is the inputs of a scale within a unit (32, 64 or 128; 256 takes 128's).
template <typename T, int Code, int Group, int NT, int MT>
struct Unit {
  static constexpr bool kScaled = Code == kMx && T::kType == kBf16;  // scales go into the conversion
  using C = Corner<NT, MT>;
  u32x4 codes[NT], x[MT][4];
  uint32_t scale[NT], zero[NT];  // of column lane / 4, group lane % 4, as loaded: whatever waits for a load stands in add

  // Unit u (held to the last one: the loads of none past it are used).
  __device__ __forceinline__ void load(const W4Args& g, const int (&n)[NT], const int (&m)[MT][4], int u, int units, int lane,
                                       int shift) {
    const int k0 = (u < units ? u : units - 1) * 128;
    // lanes past the row's end load its first bytes, which add drops
    const int kc = k0 + (lane & 3) * 32 < g.K ? k0 + (lane & 3) * 32 : 0;
    const int kx = k0 + (lane & 15) * 8 < g.K ? k0 + (lane & 15) * 8 : 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      codes[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g.codes + n[i] * g.ldw + kc / 2));
      const int64_t at = (int64_t)n[i] * g.groups + (kc >> shift);
      if constexpr (Code == kMx) {
        scale[i] = static_cast<const uint8_t*>(g.scales)[at];
      } else {
        if (g.scale_type == kF32) scale[i] = static_cast<const uint32_t*>(g.scales)[at];
        else scale[i] = static_cast<const uint16_t*>(g.scales)[at];
        if (g.zeros) zero[i] = g.zeros[at];
      }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int d = 0; d < 4; ++d) x[j][d] = *reinterpret_cast<const u32x4_any*>(g.x + m[j][d] * g.ldx + kx);
  }

  __device__ __forceinline__ void add(const W4Args& g, char* lds, f32x4 (&acc)[NT][MT], int u, int lane) {
    const int k0 = u * 128, l16 = lane & 15, quad = lane >> 4;
    if (k0 + 128 > g.K) {
#pragma unroll
      for (int i = 0; i < NT; ++i) codes[i] = sel4(k0 + (lane & 3) * 32 < g.K, codes[i]);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) x[j][d] = sel4(k0 + l16 * 8 < g.K, x[j][d]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      st16(lds + C::kCodes + i * 1024 + (lane >> 2) * 64 + (((lane & 3) ^ quad) << 4), codes[i]);
      float f;
      if constexpr (Code == kMx) f = ue8m0_to_f32(scale[i]);
      else f = g.scale_type == kF32 ? __uint_as_float(scale[i])
                                    : g.scale_type == kBf16 ? Bf16::to_f32((uint16_t)scale[i]) : F16::to_f32((uint16_t)scale[i]);
      *reinterpret_cast<float*>(lds + C::kScale + i * 256 + lane * 4) = f;
      if constexpr (Code == kInt4)
        *reinterpret_cast<float*>(lds + C::kZero + i * 256 + lane * 4) = g.zeros ? (float)zero[i] : 8.0f;
    }
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int r = 4 * d + quad;
        st16(lds + C::kX + j * 4096 + r * 256 + ((l16 ^ r) << 4), x[j][d]);
      }
    f32x4 s[NT], z[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      s[i] = *reinterpret_cast<const f32x4*>(lds + C::kScale + i * 256 + l16 * 16);
      if constexpr (Code == kInt4) z[i] = *reinterpret_cast<const f32x4*>(lds + C::kZero + i * 256 + l16 * 16);
    }
    f32x4 part[NT][MT], sx[MT];
#pragma unroll
    for (int d = 0; d < 4; ++d) {  // a product: group d of the unit, lane: eight inputs from 8 quad on
      u32x4 fx[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) fx[j] = ld16(lds + C::kX + j * 4096 + l16 * 256 + (((d * 4 + quad) ^ l16) << 4));
      if (!kScaled && d % (Group / 32) == 0) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          sx[j] = f32x4{};
#pragma unroll
          for (int i = 0; i < NT; ++i) part[i][j] = f32x4{};
        }
      }
      if constexpr (Code == kInt4) {
        const uint32_t one = T::kType == kBf16 ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
        for (int j = 0; j < MT; ++j) sx[j] = T::mfma(fx[j], u32x4{one, one, one, one}, sx[j]);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(lds + C::kCodes + i * 1024 + l16 * 64 + ((d ^ (l16 >> 2)) << 4) +
                                                              quad * 4);
        if constexpr (kScaled) {
          const u32x4 b = __builtin_bit_cast(u32x4, fp4x8_to_bf16x8(c, s[i][d]));
#pragma unroll
          for (int j = 0; j < MT; ++j) acc[i][j] = T::mfma(fx[j], b, acc[i][j]);
        } else {
          const u32x4 b = decode8<T, Code>(c);
#pragma unroll
          for (int j = 0; j < MT; ++j) part[i][j] = T::mfma(fx[j], b, part[i][j]);
        }
      }
      if (!kScaled && (d + 1) % (Group / 32) == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            const int first = d + 1 - Group / 32;  // past the row's end only the scale's first group is sure
            f32x4 v = part[i][j];
            if constexpr (Code == kInt4) v -= z[i][first] * sx[j];
            acc[i][j] += s[i][first] * v;
          }
      }
    }
  }
};

template <typename T, int Code, int Group, int NT, int MT, int NW>
__global__ void __launch_bounds__(NW * 64) w4_kernel(W4Args g, int shift) {
  using C = Corner<NT, MT>;
  constexpr int kSums = NW * NT * MT * 1024, kCorners = NW * C::kBytes;
  __shared__ char lds[kSums > kCorners ? kSums : kCorners];  // the corners, then the waves' sums [NW][NT][MT][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  // columns and rows past the end read the last one's: their results are not stored
  int n[NT], m[MT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) n[i] = n0 + i * 16 + (lane >> 2) < g.N ? n0 + i * 16 + (lane >> 2) : g.N - 1;
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int r = m0 + j * 16 + d * 4 + (lane >> 4);
      m[j][d] = r < g.M ? r : g.M - 1;
    }
  f32x4 acc[NT][MT] = {};
  const int units = (g.K + 127) / 128, per = (units + NW - 1) / NW;
  const int u0 = wave * per, u1 = u0 + per < units ? u0 + per : units;
  char* const corner = lds + wave * C::kBytes;
  Unit<T, Code, Group, NT, MT> a, b;
  if (u0 < u1) a.load(g, n, m, u0, units, lane, shift);
  for (int u = u0; u < u1; u += 2) {
    b.load(g, n, m, u + 1, units, lane, shift);
    a.add(g, corner, acc, u, lane);
    if (u + 1 >= u1) break;
    a.load(g, n, m, u + 2, units, lane, shift);
    b.add(g, corner, acc, u + 1, lane);
  }
  __syncthreads();
  f32x4* const sums = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) sums[((wave * NT + i) * MT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // thread -> column n0 + 16 i + c, row m0 + 16 j + r; lane 16 (r / 4) + c held it in component r % 4
  const float* const f = reinterpret_cast<const float*>(lds);
  for (int o = threadIdx.x; o < NT * MT * 256; o += NW * 64) {
    const int c = o & 15, i = (o >> 4) % NT, r16 = (o >> 4) / NT, r = r16 & 15, j = r16 >> 4;
    const int row = m0 + j * 16 + r, col = n0 + i * 16 + c;
    if (row >= g.M || col >= g.N) continue;
    const int at = ((i * MT + j) * 64 + 16 * (r >> 2) + c) * 4 + (r & 3);
    float v = f[at];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += f[at + q * NT * MT * 256];
    finish_w4<T>(g, row, col, v);
  }
}

template <typename T, int Code, int Group, int NT, int MT, int NW>
void launch_tiles(const W4Args& a, hipStream_t stream) {
  const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * MT - 1) / (16 * MT));
  int shift = 5;  // of inputs to scales
  while (1 << shift < a.group) ++shift;
  hipLaunchKernelGGL((w4_kernel<T, Code, Group, NT, MT, NW>), grid, dim3(NW * 64), 0, stream, a, shift);
}

// Tiles by time (one MI355X, bf16 x, MX, weights cold, us; NT MT NW):
//   16 rows   N = 288: 1 1 8 6.8, 2 1 8 9.2; 5120 x 9216: 20.9, 17.2; 9216 x 5120: 19.5, 20.0
//   24 rows   2304 x 5120: 1 1 8 11.2, 2 1 8 9.8, 2 2 4 12.5; 9216 x 5120: 27.6, 26.5, 23.2; 4 4 4 28.7
//   64 rows   N = 288: 1 1 8 8.5, 2 2 4 12.8; 5120 x 5120: 30.4, 22.5, 4 4 4 30.4; 9216 x 5120: 54.0, 34.9, 31.4
template <typename T, int Code, int Group>
void launch_rows(const W4Args& a, hipStream_t stream) {
  if (a.N <= 512 && a.M <= 16384) launch_tiles<T, Code, Group, 1, 1, 8>(a, stream);  // (a grid's rows end at 65535)
  else if (a.M <= 16) {
    // two columns' tiles where that fills the CUs about once, or many times
    if ((a.N > 4096 && a.N <= 8192) || a.N >= 16384) launch_tiles<T, Code, Group, 2, 1, 8>(a, stream);
    else launch_tiles<T, Code, Group, 1, 1, 8>(a, stream);
  } else if (a.M <= 32 || a.N <= 8192) launch_tiles<T, Code, Group, 2, 2, 4>(a, stream);
  else launch_tiles<T, Code, Group, 4, 4, 4>(a, stream);
}

template <typename T>
void launch_type(const W4Args& a, hipStream_t stream) {
  if (a.code == kMx) launch_rows<T, kMx, 32>(a, stream);
  else if (a.group == 32) launch_rows<T, kInt4, 32>(a, stream);
  else if (a.group == 64) launch_rows<T, kInt4, 64>(a, stream);
  else launch_rows<T, kInt4, 128>(a, stream);
}

}  // namespace

// Where each kernel is taken, by time (one MI355X, bf16 x, weights cold, us):
//   rows as a stream of the weights, one and two from K = 1024 on: one row of 9216 x 5120 8.0, on
//     the matrix cores 13.2; two 11.4, 13.2; four 17.0, 13.4; one of 5120 x 512 3.7, 3.1
//   up to 16 rows of many columns held in registers, where a wave's scales fit beside them (tiles,
//     held): 16 rows, MX, 9216 x 5120: 19.4, 15.3; 3 rows 13.4, 14.6; 8192 x 8192: 16.8 by tiles,
//     whose workgroups are 256 there; 16384 x 5120: 19.0 held; 65536 x 5120: 74, 54
//   shared through LDS (tiles, shared): 8 rows, int4 groups of 64, 32768 x 5120: 38, 47; 65536 x
//     5120: 75, 54; 32 rows, MX, 24576 x 5120: 40, 45; 65536 x 5120: 101, 56; 64 rows, 16384 x 5120:
//     34, 50; 24576 x 5120: 61, 52; 65536 x 5120: 127, 60
// All of these are at K = 5120 or near it, most with MX and bf16: at other K the crossings may lie
// elsewhere, since a workgroup's work grows with K.
hipError_t launch_w4(const W4Args& a, hipStream_t stream) {
  const bool hold = a.code == kMx || a.group >= 128;
  const int wide = a.M > 32 ? 20480 : a.M > 16 ? 32768 : 49152;  // columns from which rows are shared
  if (a.M <= 2 && a.K >= 1024) launch_w4_row(a, stream);
  else if (a.M <= 16 && hold && a.N >= (a.M > 8 ? 8193 : 16384)) launch_w4_hold(a, stream);
  else if (a.N >= wide && w4_row_bytes(a) <= kWideRowBytes) launch_w4_wide(a, stream);
  else if (a.type == kBf16) launch_type<Bf16>(a, stream);
  else launch_type<F16>(a, stream);
  return hipGetLastError();
}

}  // namespace moe_fp4
