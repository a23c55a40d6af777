// The product of up to 16 rows with 4-bit weights on many columns: rows of x held in
// registers.
//
// A workgroup's eight waves split the sum, and each keeps its part of 16 rows of x, UW
// units of 128 inputs, in registers as the A operands of 16x16x32 products.  The
// workgroup then goes over tiles of 16 columns, blockIdx.x, blockIdx.x + gridDim.x, ...,
// of whose codes a wave loads 1 KB a unit, two tiles ahead.  Loads go out as memory lies
// (four lanes: 64 bytes of codes of a column; sixteen: 256 bytes of a row of x) and pass
// through the wave's own corner of LDS into the order of the matrix instruction, in which
// a lane's sums are of one column, whose scale it can apply, and a product takes one
// group.  The waves' sums of a tile meet in LDS and are added in wave order.  A sum longer
// than the eight waves hold is taken in chunks, the tiles' totals kept in LDS between them.
//
// 16 rows of 65536 x 5120, MX: 53 us for 178 MB.  A CU has one workgroup, 80 KB of codes on
// their way; its tiles wait for one another at their barriers.
#include "w4_device.h"

namespace moe_fp4 {
namespace {

constexpr int kHoldWaves = 8, kHoldAhead = 3;  // tiles in registers: one computed, two on their way
constexpr int kHoldBlocks = 256, kHoldTiles = (kMaxWidth / 16 + kHoldBlocks - 1) / kHoldBlocks;  // tiles of a workgroup

// A column's scales in a wave's units: MX one dword a unit, int4 one value a Group.
template <int Code, int Group, int UW>
struct HoldScales {
  static constexpr int kCount = Code == kMx ? UW : UW * 128 / Group;
  static constexpr int kRegs = (kCount + 3) / 4;  // lane l loads those of column l / 4: l % 4, l % 4 + 4, ...
  static constexpr int kPitch = (kRegs * 4) | 1;
};

template <typename T, int Code, int Group, int UW>
__global__ void __launch_bounds__(kHoldWaves * 64) w4_hold_kernel(W4Args g, int chunk_units, int shift) {
  constexpr bool kScaled = Code == kMx && T::kType == kBf16;  // scales go into the conversion
  using S = HoldScales<Code, Group, UW>;
  __shared__ char corners[kHoldWaves][UW * 1024 < 4096 ? 4096 : UW * 1024];
  __shared__ uint32_t scale_lds[kHoldWaves][16 * S::kPitch], zero_lds[kHoldWaves][Code == kInt4 ? 16 * S::kPitch : 1];
  __shared__ f32x4 sums[2][kHoldWaves][64];
  __shared__ float totals[kHoldTiles][256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4, row4 = lane >> 2, m0 = blockIdx.y * 16;
  char* const corner = corners[wave];
  const int units = (g.K + 127) / 128, tiles = (g.N + 15) / 16;
  const int mine = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // tiles of this workgroup
  const int chunks = (units + chunk_units - 1) / chunk_units;
  // this wave's units of chunk c: [first, last)
  const auto range = [&](int c, int& first, int& last) {
    const int end = units - c * chunk_units < chunk_units ? units : (c + 1) * chunk_units;
    const int per = (end - c * chunk_units + kHoldWaves - 1) / kHoldWaves;
    first = c * chunk_units + wave * per;
    last = first + per < end ? first + per : end;
  };
  u32x4 codes[kHoldAhead][UW];
  uint32_t scale[kHoldAhead][S::kRegs], zero[kHoldAhead][S::kRegs];
  // The loads of the i-th piece of work: tile i % mine of chunk i / mine (none past the last
  // piece is used).  The last tile starts early where it is short; its columns of the tile
  // before are not stored.  Inputs past the wave's take its first: what x holds there is 0.
  const auto tile_start = [&](int i, int& c) {
    const int at = i < chunks * mine ? i : chunks * mine - 1;
    c = at / mine;
    const int n0 = (blockIdx.x + (at - c * mine) * gridDim.x) * 16;
    return n0 + 16 <= g.N ? n0 : g.N > 16 ? g.N - 16 : 0;
  };
  const int row = row4 < g.N ? row4 : g.N - 1;
  const auto load = [&](int i, u32x4 (&cd)[UW], uint32_t (&sc)[S::kRegs], uint32_t (&ze)[S::kRegs]) {
    int c, first, last;
    const int n0 = tile_start(i, c);
    range(c, first, last);
    const int start = first < units ? first * 128 : 0, count = (last < units ? last * 128 : g.K) - start;
    const uint8_t* const w = g.codes + (int64_t)n0 * g.ldw + start / 2;
    const uint32_t r = (uint32_t)row * (uint32_t)g.ldw;
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      const int k = u * 128 + (lane & 3) * 32;
      cd[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + (r + (k < count ? k / 2 : 0))));
    }
    const int64_t s0 = (int64_t)n0 * g.groups + (start >> shift);
    const int have = g.groups - (start >> shift);  // scales of a row from there on
#pragma unroll
    for (int v = 0; v < S::kRegs; ++v) {
      if constexpr (Code == kMx) {  // four bytes, the row's last four where fewer are left
        const uint8_t* const p = static_cast<const uint8_t*>(g.scales) + s0;
        const int j = (v * 4 + (lane & 3)) * 4, at = row * g.groups;
        if (g.groups >= 4) sc[v] = *reinterpret_cast<const u32_byte*>(p + at + (j < have - 4 ? j : have - 4));
        else sc[v] = p[at] | p[at + (have > 1 ? 1 : 0)] << 8 | p[at + (have > 2 ? 2 : 0)] << 16;
      } else {
        const int j = v * 4 + (lane & 3), of = Group == 128 && g.group == 256 ? ((start + j * 128) >> 8) - (start >> 8) : j;
        const int at = row * g.groups + (of < have ? of : 0);
        if (g.scale_type == kF32) sc[v] = (static_cast<const uint32_t*>(g.scales) + s0)[at];
        else sc[v] = (static_cast<const uint16_t*>(g.scales) + s0)[at];
        if (g.zeros) ze[v] = (g.zeros + s0)[at];
      }
    }
  };
  u32x4 x[UW][4];
  const auto load_x = [&](int c) {
    int first, last;
    range(c, first, last);
    const int end = last * 128 < g.K ? last * 128 : g.K;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int m = m0 + 4 * d + quad < g.M ? m0 + 4 * d + quad : g.M - 1;  // rows past the end: not stored
      const uint16_t* const p = g.x + m * g.ldx;
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        const int k = (first + u) * 128 + l16 * 8;
        x[u][d] = *reinterpret_cast<const u32x4_any*>(p + (k < end ? k : 0));
      }
    }
  };
  const auto turn_x = [&](int c) {  // row 4 d + quad, chunk l16 -> row l16, chunk 4 d + quad (a chunk: eight inputs)
    int first, last;
    range(c, first, last);
    const int end = last * 128 < g.K ? last * 128 : g.K;
#pragma unroll
    for (int u = 0; u < UW; ++u) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int r = 4 * d + quad;
        st16(corner + r * 256 + ((l16 ^ r) << 4), sel4((first + u) * 128 + l16 * 8 < end, x[u][d]));
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) x[u][d] = ld16(corner + l16 * 256 + (((d * 4 + quad) ^ l16) << 4));
    }
  };
  const auto tile = [&](int i, u32x4 (&cd)[UW], uint32_t (&sc)[S::kRegs], uint32_t (&ze)[S::kRegs]) {
    int c, first, last;
    const int n0 = tile_start(i, c);
    range(c, first, last);
    const int left = g.groups - (first < units ? first * 4 : 0);  // MX: scales of the row from the wave's first on
#pragma unroll
    for (int u = 0; u < UW; ++u) st16(corner + u * 1024 + row4 * 64 + (((lane & 3) ^ quad) << 4), cd[u]);
#pragma unroll
    for (int v = 0; v < S::kRegs; ++v) {
      const int j = v * 4 + (lane & 3), at = row4 * S::kPitch + j;
      if constexpr (Code == kMx) {
        const int more = j * 4 + 4 - left;  // bytes of it that lie before the unit's
        scale_lds[wave][at] = sc[v] >> (g.groups >= 4 && more > 0 && more < 4 ? 8 * more : 0);
      } else {
        scale_lds[wave][at] = g.scale_type == kF32 ? sc[v]
                                                   : __float_as_uint(g.scale_type == kBf16 ? Bf16::to_f32((uint16_t)sc[v])
                                                                                           : F16::to_f32((uint16_t)sc[v]));
        if (g.zeros) zero_lds[wave][at] = __float_as_uint((float)ze[v]);
      }
    }
    f32x4 acc = {};
#pragma unroll
    for (int u = 0; u < UW; ++u) {
      uint32_t cw[4];
#pragma unroll
      for (int d = 0; d < 4; ++d)
        cw[d] = *reinterpret_cast<const uint32_t*>(corner + u * 1024 + l16 * 64 + ((d ^ (l16 >> 2)) << 4) + quad * 4);
      if constexpr (Code == kMx) {
        const uint32_t s4 = scale_lds[wave][l16 * S::kPitch + u];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float s = ue8m0_to_f32((s4 >> (8 * d)) & 255u);
          if constexpr (kScaled)
            acc = T::mfma(x[u][d], __builtin_bit_cast(u32x4, fp4x8_to_bf16x8(cw[d], s)), acc);
          else
            acc += s * T::mfma(x[u][d], decode8<T, Code>(cw[d]), f32x4{});
        }
      } else {
#pragma unroll
        for (int s = 0; s < 128 / Group; ++s) {
          f32x4 part = {}, sx = {};
#pragma unroll
          for (int d = s * Group / 32; d < (s + 1) * Group / 32; ++d) {
            const uint32_t one = T::kType == kBf16 ? 0x3F803F80u : 0x3C003C00u;
            sx = T::mfma(x[u][d], u32x4{one, one, one, one}, sx);
            part = T::mfma(x[u][d], decode8<T, Code>(cw[d]), part);
          }
          const int at = l16 * S::kPitch + u * (128 / Group) + s;
          part -= (g.zeros ? __uint_as_float(zero_lds[wave][at]) : 8.0f) * sx;
          acc += __uint_as_float(scale_lds[wave][at]) * part;
        }
      }
    }
    const int parity = i & 1;
    sums[parity][wave][lane] = acc;
    lds_barrier();  // the buffer of this parity is written again two tiles on, behind the next tile's barrier
    if ((wave >> 2) == parity) {  // four waves finish a tile, the others the next one
      // thread -> column o % 16, row o / 16 of the tile; lane 16 (r / 4) + column held it in component r % 4
      const int o = (wave & 3) * 64 + lane, col = o & 15, r = o >> 4, m = m0 + r;
      const int t = i - c * mine, n = n0 + col;
      const float* const f = reinterpret_cast<const float*>(sums[parity]) + (16 * (r >> 2) + col) * 4 + (r & 3);
      float total = f[0];
#pragma unroll
      for (int q = 1; q < kHoldWaves; ++q) total += f[q * 256];
      // A tile's totals are kept and taken up by different threads where `mine` is odd: a
      // barrier lies between (of the tiles between, or of the one tile's next chunk).
      if (c) total += totals[t][o];
      if (c + 1 < chunks) totals[t][o] = total;
      else if (m < g.M && n < g.N && n >= (blockIdx.x + t * gridDim.x) * 16) finish_w4<T>(g, m, n, total);
    }
  };
  load_x(0);
#pragma unroll
  for (int a = 0; a < kHoldAhead - 1; ++a) load(a, codes[a], scale[a], zero[a]);
  turn_x(0);
  const int all = chunks * mine;
  for (int i = 0;;) {
#pragma unroll
    for (int a = 0; a < kHoldAhead; ++a) {
      constexpr int last = kHoldAhead - 1;
      load(i + last, codes[(a + last) % kHoldAhead], scale[(a + last) % kHoldAhead], zero[(a + last) % kHoldAhead]);
      tile(i, codes[a], scale[a], zero[a]);
      if (++i >= all) return;
      if (i % mine == 0) {
        load_x(i / mine);
        turn_x(i / mine);
      }
    }
  }
}

template <typename T, int Code, int Group>
void launch_group(const W4Args& a, hipStream_t stream) {
  const int tiles = (a.N + 15) / 16, blocks = tiles < kHoldBlocks ? tiles : kHoldBlocks;
  const dim3 grid(blocks, (a.M + 15) / 16);
  const int units = (a.K + 127) / 128;
  // chunks of at most 40 units, alike long; a wave's four units run as five, one of zeros (16 rows of
  // 16384 x 4096 17.4 us, x 5120 19.0)
  const int chunks = (units + 39) / 40, per = (units + chunks - 1) / chunks, uw = (per + kHoldWaves - 1) / kHoldWaves;
  int shift = 5;  // of inputs to scales
  while (1 << shift < a.group) ++shift;
  const auto run = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(kHoldWaves * 64), 0, stream, a, uw * kHoldWaves, shift); };
  if (uw <= 1) run(w4_hold_kernel<T, Code, Group, 1>);
  else if (uw <= 2) run(w4_hold_kernel<T, Code, Group, 2>);
  else if (uw <= 3) run(w4_hold_kernel<T, Code, Group, 3>);
  else run(w4_hold_kernel<T, Code, Group, 5>);
}
template <typename T>
void launch(const W4Args& a, hipStream_t stream) {
  if (a.code == kMx) launch_group<T, kMx, 32>(a, stream);
  else launch_group<T, kInt4, 128>(a, stream);
}

}  // namespace

void launch_w4_hold(const W4Args& a, hipStream_t stream) {
  if (a.type == kBf16) launch<Bf16>(a, stream);
  else launch<F16>(a, stream);
}

}  // namespace moe_fp4
