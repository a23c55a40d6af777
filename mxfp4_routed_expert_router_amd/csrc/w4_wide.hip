// The product with 4-bit weights on many columns: rows of x shared through LDS.
//
// A workgroup takes 256 columns and 16 MT rows and goes along the sum 128 inputs (a unit)
// at a time.  A wave of its own (two for 64 rows) brings x into one of two buffers of LDS, which eight others read:
// a wave's loads return in order, and one that waited for rows of x from the L2 would wait
// for all codes asked for before them.  Each of the eight has 32 columns, whose codes go
// from memory straight into its ring in LDS, four or five units ahead, as memory lies (four lanes:
// 64 bytes of a column), from where the lanes take them in the order of the matrix
// instruction: x is A, the codes, decoded in registers, are B, a lane's sums are of one
// column, a product takes one group.  The columns' scales, one piece of memory, are copied
// to LDS at the start.  No sums are split.
//
// 64 rows of 65536 x 5120, MX: 60 us, 184 MB read where 178 are needed (291 with loads that
// the L2 keeps at low priority: a line's two halves are taken a unit apart), matrix cores 28 %
// busy; 256 workgroups, one a CU, whose LDS holds 64 KB of codes on their way: bound by their
// latency and the decoding between two barriers, 1.3 us a unit.  The same through the
// tiles of w4.hip, whose every wave reads x for itself: 127 us.
#include "lds_dma.h"
#include "w4_device.h"

namespace moe_fp4 {
namespace {

constexpr int kWideWaves = 8, kWideTiles = 2, kWideColumns = kWideWaves * kWideTiles * 16;
// Waves that bring x, threads, and units in a wave's ring: what 160 KB of LDS hold.
template <int MT>
struct Wide {
  static constexpr int kXWaves = MT == 4 ? 2 : 1, kThreads = (kWideWaves + kXWaves) * 64, kRing = MT == 4 ? 5 : 6;
};
constexpr int kWideUnit = kWideTiles * 1024;  // bytes of codes of a wave's unit

template <typename T, int Code, int Group, int MT>
__global__ void __launch_bounds__(Wide<MT>::kThreads) w4_wide_kernel(W4Args g, int shift) {
  constexpr bool kScaled = Code == kMx && T::kType == kBf16;  // scales go into the conversion
  constexpr int NT = kWideTiles, kXWaves = Wide<MT>::kXWaves, kRing = Wide<MT>::kRing;
  constexpr int kLoads = MT * 4 / kXWaves;  // 16-byte loads of x a lane and unit
  __shared__ __align__(1024) char ring[kWideWaves][kRing][kWideUnit];  // column c: 64 bytes, chunk k at k ^ c / 4 % 4
  __shared__ __align__(1024) char xs[2][MT * 4096];                        // row r: 256 bytes, chunk c at c ^ r % 16
  __shared__ __align__(16) char scales[kWideColumns * kWideRowBytes];      // then the zeros
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  int tile;
  if (!xcd_tile((g.N + kWideColumns - 1) / kWideColumns, tile)) return;
  const int m0 = blockIdx.y * 16 * MT, units = (g.K + 127) / 128, c0 = tile * kWideColumns;
  const int size = Code == kMx ? 1 : g.scale_type == kF32 ? 4 : 2;
  const int columns = g.N - c0 < kWideColumns ? g.N - c0 : kWideColumns, some = columns * g.groups;
  const auto copy = [&](const void* from, int bytes, char* to) {
    const char* const p = static_cast<const char*>(from);
    for (int i = threadIdx.x * 16; i < bytes; i += Wide<MT>::kThreads * 16) {
      if (i + 16 <= bytes) {
        const u32x4 v = *reinterpret_cast<const u32x4_byte*>(p + i);
        st16(to + i, v);
      } else {
        for (int j = i; j < bytes; ++j) to[j] = p[j];
      }
    }
  };
  char* const zeros = scales + (columns * g.groups * size + 15) / 16 * 16;
  copy(static_cast<const char*>(g.scales) + (int64_t)c0 * g.groups * size, some * size, scales);
  if (Code == kInt4 && g.zeros) copy(g.zeros + (int64_t)c0 * g.groups, some, zeros);
  if (wave >= kWideWaves) {  // rows of x: load j takes rows row_of(j), chunk lane % 16
    const auto row_of = [&](int j) { return 4 * (j * kXWaves + wave - kWideWaves) + quad; };
    const uint16_t* px[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int r = m0 + row_of(j);
      px[j] = g.x + (r < g.M ? r : g.M - 1) * g.ldx + l16 * 8;  // rows past the end: not stored
    }
    constexpr int kAhead = MT == 1 ? 4 : 3;  // units of x in registers
    u32x4 x[kAhead][kLoads];
    const auto load = [&](int u, u32x4 (&o)[kLoads]) {  // held to the last unit; inputs past the end take the row's first
      const int k0 = (u < units ? u : units - 1) * 128, at = k0 + l16 * 8 < g.K ? k0 : -l16 * 8;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) o[j] = *reinterpret_cast<const u32x4_any*>(px[j] + at);
    };
    const auto store = [&](int u, const u32x4 (&o)[kLoads]) {  // zeros past the end: no code counts there
      const bool in = u * 128 + l16 * 8 < g.K;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = row_of(j);
        st16(xs[u & 1] + r * 256 + ((l16 ^ (r & 15)) << 4), sel4(in, o[j]));
      }
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) load(a, x[a]);
    store(0, x[0]);
    for (int u = 0; u < units;) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        lds_barrier();  // unit u is there, and unit u - 1's buffer free
        load(u + kAhead, x[a]);
        if (u + 1 < units) store(u + 1, x[(a + 1) % kAhead]);
        if (++u >= units) break;
      }
    }
    return;
  }
  const int n0 = c0 + wave * NT * 16;
  // the lane's chunk of a unit of column lane / 4; columns past the end read the last one's
  const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
  const uint8_t* w[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int n = n0 + i * 16 + (lane >> 2) < g.N ? n0 + i * 16 + (lane >> 2) : g.N - 1;
    w[i] = g.codes + n * g.ldw + chunk * 16;
  }
  const uint32_t ring0 = lds_addr(ring[wave][0]);
  const auto load = [&](int u, int slot) {  // held to the last unit; inputs past the end take the row's first
    const int k0 = (u < units ? u : units - 1) * 128, at = k0 + chunk * 32 < g.K ? k0 / 2 : -chunk * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) lds_load16(ring0 + slot * kWideUnit + i * 1024, w[i] + at);
  };
  int col[NT];  // of the copied scales
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int c = wave * NT * 16 + i * 16 + l16;
    col[i] = (c < columns ? c : columns - 1) * g.groups;
  }
  f32x4 acc[NT][MT] = {};
  const auto unit = [&](int u, int slot) {
    const char* const xu = xs[u & 1];
    const char* const cu = ring[wave][slot];
    constexpr int kSums = 128 / Group;
    float s[NT][kSums], z[NT][kSums];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if constexpr (Code == kMx) {
        if ((g.groups & 3) == 0) {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(scales + col[i] + u * 4);
#pragma unroll
          for (int d = 0; d < 4; ++d) s[i][d] = ue8m0_to_f32((v >> (8 * d)) & 255u);
        } else {
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int at = u * 4 + d < g.groups ? u * 4 + d : g.groups - 1;
            s[i][d] = ue8m0_to_f32(static_cast<uint8_t>(scales[col[i] + at]));
          }
        }
      } else {
#pragma unroll
        for (int d = 0; d < kSums; ++d) {
          const int of = (u * 128 + d * Group) >> shift, at = col[i] + (of < g.groups ? of : g.groups - 1);
          s[i][d] = scalar_as_f32(scales, at, g.scale_type);
          z[i][d] = g.zeros ? (float)static_cast<uint8_t>(zeros[at]) : 8.0f;
        }
      }
    }
    f32x4 part[NT][MT], sx[MT];
#pragma unroll
    for (int d = 0; d < 4; ++d) {  // a product: group d of the unit, lane: eight inputs from 8 quad on
      u32x4 fx[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) fx[j] = ld16(xu + j * 4096 + l16 * 256 + (((d * 4 + quad) ^ l16) << 4));
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
        const uint32_t c = *reinterpret_cast<const uint32_t*>(cu + i * 1024 + l16 * 64 + ((d ^ (l16 >> 2)) << 4) + quad * 4);
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
        const int of = d / (Group / 32);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            f32x4 v = part[i][j];
            if constexpr (Code == kInt4) v -= z[i][of] * sx[j];
            acc[i][j] += s[i][of] * v;
          }
      }
    }
  };
  // No other loads of this wave are under way from here to the end of the loop: the copy's
  // were waited for by its stores.
#pragma unroll
  for (int a = 0; a < kRing - 1; ++a) load(a, a);
  for (int u = 0, slot = 0; u < units; ++u) {
    // unit u's codes (two loads) are there, those of the units behind may be under way; the
    // lanes' reads of unit u - 1 are done, whose part of the ring is filled next
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(NT * (kRing - 2)) : "memory");
    load(u + kRing - 1, slot ? slot - 1 : kRing - 1);
    unit(u, slot);
    slot = slot + 1 < kRing ? slot + 1 : 0;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // none may land in another workgroup's LDS
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = m0 + j * 16 + quad * 4 + r, n = n0 + i * 16 + l16;
        if (m < g.M && n < g.N) finish_w4<T>(g, m, n, acc[i][j][r]);
      }
}

template <typename T, int Code, int Group>
void launch_group(const W4Args& a, hipStream_t stream) {
  int shift = 5;  // of inputs to scales
  while (1 << shift < a.group) ++shift;
  const auto run = [&](auto k, int mt, int threads) {
    hipLaunchKernelGGL(k, dim3(xcd_grid((a.N + kWideColumns - 1) / kWideColumns), (a.M + 16 * mt - 1) / (16 * mt)),
                       dim3(threads), 0, stream, a, shift);
  };
  if (a.M <= 16) run(w4_wide_kernel<T, Code, Group, 1>, 1, Wide<1>::kThreads);
  else if (a.M <= 32) run(w4_wide_kernel<T, Code, Group, 2>, 2, Wide<2>::kThreads);
  else run(w4_wide_kernel<T, Code, Group, 4>, 4, Wide<4>::kThreads);
}
template <typename T>
void launch(const W4Args& a, hipStream_t stream) {
  if (a.code == kMx) launch_group<T, kMx, 32>(a, stream);
  else if (a.group == 32) launch_group<T, kInt4, 32>(a, stream);
  else if (a.group == 64) launch_group<T, kInt4, 64>(a, stream);
  else launch_group<T, kInt4, 128>(a, stream);
}

}  // namespace

void launch_w4_wide(const W4Args& a, hipStream_t stream) {
  if (a.type == kBf16) launch<Bf16>(a, stream);
  else launch<F16>(a, stream);
}

}  // namespace moe_fp4
