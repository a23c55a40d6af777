// 16-bit products through LDS tiles filled straight from memory.
//
// A workgroup computes BI x BJ results (i: rows of the result, j: its columns),
// 64 of the sum a step.  global_load_lds_dwordx4 fills the operands' stages in
// LDS without passing through registers; the two halves of a step are read into
// registers half a step ahead of the matrix instructions, and one barrier a
// step keeps the waves together.  A has two stages, B two or three: B's rows
// (the weights, in forward and dgrad) come from HBM and are sent for two steps
// ahead with three.
//
// LDS layout.  An operand that is contiguous along the sum (x, dy as the row
// side, w of forward) is held as [index][64]: a load brings whole 128-byte lines
// (with 64 bytes a row, twice the requests reach the L2), and the 16-byte chunk
// c of row r lies at c ^ (r % 8), so that a fragment's 16 rows are read without
// bank conflicts (4 cycles a wave; measured 8 with c ^ (r % 8) ^ (r / 8)).  An
// operand that is contiguous along its own index (w of dgrad; both of wgrad) is
// held as it lies, [64][index], and ds_read_b64_tr_b16 turns 4 x 16 blocks on the
// way to the registers: within 16 lanes, lane i receives column i of the four
// rows that lanes 4 r .. 4 r + 3 address.  Its 32-byte units (16 indexes) of row
// r sit at unit ^ unit_swizzle(r).
//
// Bound by the matrix cores and LDS together where the rows are many: 4096^3 bf16
// 95 - 98 us forward, 95 - 97 rows' gradient, 98 - 101 weights' gradient (1.4
// PFLOP/s; a step of 256 x 256 takes 1.5 us).  By the weights' bytes where an expert
// has few rows: 48 experts of 2304 x 5120, 32 rows each, 205 us (5.5 TB/s).
#pragma once

#include "block_device.h"
#include "lds_dma.h"

namespace moe_fp4 {
namespace {

constexpr int kStepK = 64;
constexpr int kIndexCache = 1024;  // row indexes of a gathered sum held in LDS

__device__ const __align__(16) uint32_t zero_chunk[4] = {0u, 0u, 0u, 0u};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) char lds_char;

// Units of rows r of which 8 (rows 0-3 and 8-11, say) are read together: they
// take 8 different 32-byte bank groups.
template <int BX>
__device__ __forceinline__ int unit_swizzle(int r) {
  if constexpr (BX >= 128) return (r & 3) | ((r >> 1) & 4);
  return ((r >> 1) & 1) | ((r >> 2) & 2);
}

// 16 bytes at a + off, off known when compiling: the instruction's offset.
__device__ __forceinline__ u32x4 lds_read16(uint32_t a, int off) {
  return *reinterpret_cast<const lds_u32x4*>(reinterpret_cast<lds_char*>(a) + off);
}
// 8 k-values of 16 indexes: two turned 4 x 16 blocks, 4 rows apart.
template <int BX>
__device__ __forceinline__ u32x4 lds_read_turned(uint32_t a, int off) {
  lds_char* const p = reinterpret_cast<lds_char*>(a) + off;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(p));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(p + 4 * BX * 2));
  const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
  return u32x4{l.x, l.y, h.x, h.y};
}

// An address that is the same in all lanes, into scalar registers.
__device__ __forceinline__ const char* uniform(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}

// BI x BJ results, WI x WJ waves, SB stages of B; OCC waves per SIMD.
template <int BI_, int BJ_, int WI_, int WJ_, int SB_, int OCC_>
struct Shape {
  static constexpr int BI = BI_, BJ = BJ_, WI = WI_, WJ = WJ_, SB = SB_, OCC = OCC_;
  static constexpr int W = WI * WJ, Threads = 64 * W;
  static constexpr int FI = BI / WI / 16, FJ = BJ / WJ / 16;  // fragments of a wave
  static constexpr int StageA = BI * 128, StageB = BJ * 128, Lds = 2 * StageA + SB * StageB;
  static constexpr int LA = BI / 8 / W, LB = BJ / 8 / W;      // 1 KB loads of a wave and stage
  // the epilogue's passes: up to four fragments of columns by as many of rows as fit the stages
  static constexpr int JC = FJ < 4 ? FJ : 4, Fit = Lds / (W * 16 * JC * 64), IC = FI <= Fit ? FI : FI / 2;
  static_assert(BI % (8 * W) == 0 && BJ % (8 * W) == 0 && BI >= 64 && BJ >= 64, "whole loads");
  static_assert(FJ % JC == 0 && FI % IC == 0 && IC <= Fit, "the epilogue's parts fit the stages");
};

// REG: for rows that are not 16-byte aligned or not a multiple of eight long, the
// stages (two of each operand) are filled through registers, a step ahead.
template <typename T, int OP, bool GATHER, bool REG, typename S>
__global__ void __launch_bounds__(S::Threads, S::OCC) product_lds_kernel(ProductArgs g, int col_tiles) {
  constexpr bool KA = OP != kWgrad, KB = OP == kFwd;  // contiguous along the sum
  constexpr bool RowsA = GATHER && OP == kFwd, RowsB = GATHER && OP == kWgrad;
  static_assert(!REG || S::SB == 2, "a step ahead");
  // behind the stages: row indexes of a gathered sum
  __shared__ __align__(1024) uint8_t smem[S::Lds + (RowsB ? kIndexCache * 4 : 0)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // ---- which tile: workgroups are dealt to the 8 XCDs round robin; each XCD
  // takes a contiguous run of tiles, one expert's after another's, up to four row
  // tiles of each column tile in turn, so that a run shares rows and weights in
  // its L2 (24576 rows on 64 experts 630 us; 667 with bands of four row tiles that
  // pass an expert's end)
  const int each = (g.I + S::BI - 1) / S::BI;  // row tiles of an expert's weights
  const int rt_all = OP == kWgrad ? g.E * each : row_tiles(g.offsets, g.E, g.P, S::BI);
  const int64_t total = (int64_t)rt_all * col_tiles;
  const int64_t per = (total + 7) / 8, slot = blockIdx.x >> 3, tile = (blockIdx.x & 7) * per + slot;
  if (slot >= per || tile >= total) return;
  int rt = (int)(tile / col_tiles), e = 0, first_tile = 0, lo = 0, rows = g.I;  // the tile's expert, and its rows
  if (OP == kWgrad) {
    e = rt / each;
    first_tile = e * each;
  } else if (g.offsets && !tile_owner(g.offsets, g.E, g.P, S::BI, rt, e, first_tile, lo, rows)) {
    return;
  }
  const int nt = (rows + S::BI - 1) / S::BI, bands = (nt + 3) / 4, high0 = (nt + bands - 1) / bands;
  int64_t in = tile - (int64_t)first_tile * col_tiles;
  const int band = (int)(in / ((int64_t)high0 * col_tiles)) * high0;  // its first row tile
  in -= (int64_t)band * col_tiles;
  const int high = nt - band < high0 ? nt - band : high0;
  rt = band + (int)in % high;
  const int j0 = (int)in / high * S::BJ, i0 = lo + rt * S::BI;
  const int ni = rows - rt * S::BI < S::BI ? rows - rt * S::BI : S::BI;
  int row0 = 0, klen = g.K;  // of the sum: wgrad's first row, and the length
  const uint16_t* b = g.b;
  if (OP == kWgrad)
    segment(g.offsets, e, g.P, row0, klen);
  else
    b += (int64_t)e * g.w_stride;
  int k0 = 0;
  if (g.splits > 1) {
    const int share = ((klen + g.splits - 1) / g.splits + kStepK - 1) / kStepK * kStepK;
    k0 = (int)blockIdx.y * share;
    klen = klen - k0 < share ? klen - k0 : share;
    if (klen < 0) klen = 0;
  }
  const int nsteps = (klen + kStepK - 1) / kStepK, full = klen / kStepK;

  // ---- this wave's loads: each fills 1 KB of a stage from its lanes'
  // addresses, a uniform base that advances with the steps and the lane's
  // offset.  Indexes past an edge read the last one's data: their results are
  // not stored.  Gathered rows have 64-bit addresses of their own.
  const int first = OP == kWgrad ? row0 + k0 : k0;
  const char* const abase = uniform(
      KA ? g.a + (RowsA ? 0 : (int64_t)i0 * g.lda) + k0 : g.a + (int64_t)first * g.lda + i0);
  const char* const bbase = uniform(
      KB ? b + (int64_t)j0 * g.ldb + k0 : b + (RowsB ? 0 : (int64_t)first * g.ldb) + j0);
  const int64_t astep = KA ? kStepK * 2 : kStepK * 2 * g.lda, bstep = KB ? kStepK * 2 : kStepK * 2 * g.ldb;
  const char* const zero = reinterpret_cast<const char*>(zero_chunk);
  const int kchunk = ((lane & 7) ^ (lane >> 3)) * 8;  // a lane's place along the sum
  // operands that lie along their index: the place along the sum of load u
  auto krow = [&](int u, int BX) { return u * (512 / BX) + lane / (BX / 8); };
  uint32_t offa[S::LA], offb[S::LB];
  const char* rowp[RowsA ? S::LA : 1];  // gathered x of forward: the lane's row, or null
  int src[RowsB ? S::LB : 1];           // gathered x of wgrad: the lane's row of the step to come, or -1
#pragma unroll
  for (int n = 0; n < S::LA; ++n) {
    const int u = n * S::W + wave;
    if constexpr (KA) {
      const int r = u * 8 + (lane >> 3), rr = r < ni ? r : ni - 1;
      offa[n] = (uint32_t)(rr * g.lda + kchunk) * 2;
      if constexpr (RowsA) {
        const int row = source_row(g, i0 + rr);
        rowp[n] = row < 0 ? nullptr : abase + ((int64_t)row * g.lda + kchunk) * 2;
      }
    } else {
      const int k = krow(u, S::BI), s = lane % (S::BI / 8);
      const int col = ((s >> 1) ^ unit_swizzle<S::BI>(k)) * 16 + (s & 1) * 8;
      offa[n] = (uint32_t)(k * g.lda + (col < ni ? col : REG ? 0 : ni - 8)) * 2;
    }
  }
#pragma unroll
  for (int n = 0; n < S::LB; ++n) {
    const int u = n * S::W + wave, nj = g.J - j0;
    if constexpr (KB) {
      const int r = u * 8 + (lane >> 3);
      offb[n] = (uint32_t)((r < nj ? r : nj - 1) * g.ldb + kchunk) * 2;
    } else {
      const int k = krow(u, S::BJ), s = lane % (S::BJ / 8);
      const int col = ((s >> 1) ^ unit_swizzle<S::BJ>(k)) * 16 + (s & 1) * 8;
      offb[n] = (uint32_t)((RowsB ? 0 : k * g.ldb) + (col < nj ? col : REG ? 0 : nj - 8)) * 2;
    }
  }
  const uint32_t lds0 = lds_addr(smem);
  // Load n of step s of A or B into the stage at `to`.  TAIL: the step may end
  // or lie past the end of the sum, where zeros are brought in.
  auto issue_a = [&](int n, int s, uint32_t to, auto tail_) {
    constexpr bool tail = decltype(tail_)::value != 0;
    const int u = n * S::W + wave;
    const bool past = tail && s * kStepK + (KA ? kchunk : krow(u, S::BI)) >= klen;
    const char* const base = abase + s * astep;
    if constexpr (RowsA) {
      const char* const p = rowp[n];
      lds_load16(to + u * 1024, past || !p ? zero : p + s * astep);
    } else if constexpr (!tail) {
      lds_load16_at(to + u * 1024, base, offa[n]);
    } else {
      lds_load16(to + u * 1024, past ? zero : base + offa[n]);
    }
  };
  auto issue_b = [&](int n, int s, uint32_t to, auto tail_) {
    constexpr bool tail = decltype(tail_)::value != 0;
    const int u = n * S::W + wave;
    const bool past = tail && s * kStepK + (KB ? kchunk : krow(u, S::BJ)) >= klen;
    const char* const base = bbase + s * bstep;
    if constexpr (RowsB) {
      const int row = src[n];  // -1 past the end
      lds_load16(to + u * 1024, row < 0 ? zero : bbase + (int64_t)row * g.ldb * 2 + offb[n]);
    } else if constexpr (!tail) {
      lds_load16_at(to + u * 1024, base, offb[n]);
    } else {
      lds_load16(to + u * 1024, past ? zero : base + offb[n]);
    }
  };
  // REG: step s's loads, waiting in registers for their stage.  At an edge, where
  // `have` of a chunk's eight elements are left, the eight that end there are read
  // instead and moved down on their way to the stage: the loads of a step are under
  // way together, behind no condition (gradients of 2047 x 2303 x 5119: rows 160 -> 117
  // us, weights 194 -> 138; 333 x 1001 x 515: 33 -> 22, 18 -> 14).  Only rows
  // of fewer than eight elements are read one by one.  Inlined by request: called,
  // they would keep the registers in memory.
  u32x4 rega[REG ? S::LA : 1], regb[REG ? S::LB : 1];
  const bool eight = (KA ? g.K : g.I) >= 8 && (KB ? g.K : g.J) >= 8;
  auto left = [&](int n, int s, auto b_) __attribute__((always_inline)) {  // of load n of A or B
    constexpr bool B = decltype(b_)::value != 0;
    if constexpr (B ? KB : KA) {
      return klen - s * kStepK - kchunk;
    } else {
      constexpr int BX = B ? S::BJ : S::BI;
      const int k = krow(n * S::W + wave, BX), c = lane % (BX / 8);
      return s * kStepK + k < klen ? (B ? g.J - j0 : ni) - (((c >> 1) ^ unit_swizzle<BX>(k)) * 16 + (c & 1) * 8) : 0;
    }
  };
  auto fetch = [&](int s, auto la_) __attribute__((always_inline)) {
    if constexpr (REG) {
      auto from_a = [&](int n) { return RowsA ? rowp[RowsA ? n : 0] + s * astep : abase + s * astep + offa[n]; };
      auto from_b = [&](int n) {
        return RowsB ? bbase + (int64_t)src[RowsB ? n : 0] * g.ldb * 2 + offb[n] : bbase + s * bstep + offb[n];
      };
      auto have_a = [&](int n) { return RowsA && !rowp[RowsA ? n : 0] ? 0 : left(n, s, IntC<0>{}); };
      auto have_b = [&](int n) { return RowsB && src[RowsB ? n : 0] < 0 ? 0 : left(n, s, IntC<1>{}); };
      auto at = [&](const char* p, int have) {
        return reinterpret_cast<const u32x4_any*>(have >= 8 ? p : have > 0 ? p - 2 * (8 - have) : zero);
      };
      if (OP == kFwd && s < full) {  // 2047 x 2303 x 5119, f16: 122 us, 125 without
#pragma unroll
        for (int n = 0; n < decltype(la_)::value; ++n)
          rega[n] = *at(from_a(n), !RowsA || rowp[RowsA ? n : 0] ? 8 : 0);
#pragma unroll
        for (int n = 0; n < S::LB; ++n) regb[n] = *at(from_b(n), 8);
      } else if (eight) {
#pragma unroll
        for (int n = 0; n < decltype(la_)::value; ++n) rega[n] = *at(from_a(n), have_a(n));
#pragma unroll
        for (int n = 0; n < S::LB; ++n) regb[n] = *at(from_b(n), have_b(n));
      } else {
#pragma unroll
        for (int n = 0; n < decltype(la_)::value; ++n)
          rega[n] = load8(reinterpret_cast<const uint16_t*>(from_a(n)), have_a(n));
#pragma unroll
        for (int n = 0; n < S::LB; ++n) regb[n] = load8(reinterpret_cast<const uint16_t*>(from_b(n)), have_b(n));
      }
    }
  };
  // step s, into the stages at sa, sb
  auto put = [&](int s, uint32_t sa, uint32_t sb, auto la_) __attribute__((always_inline)) {
    if constexpr (REG) {
      auto down = [&](u32x4& v, int have) __attribute__((always_inline)) {
        const int back = have > 0 && have < 8 ? 8 - have : 0;
        uint32_t w0 = v[0], w1 = v[1], w2 = v[2], w3 = v[3];
        const bool four = back & 4, two = back & 2, one = back & 1;
        w0 = four ? w2 : w0, w1 = four ? w3 : w1, w2 = four ? 0 : w2, w3 = four ? 0 : w3;
        w0 = two ? w1 : w0, w1 = two ? w2 : w1, w2 = two ? w3 : w2, w3 = two ? 0 : w3;
        const uint32_t sh = one ? 16 : 0;
        v = u32x4{__builtin_amdgcn_alignbit(w1, w0, sh), __builtin_amdgcn_alignbit(w2, w1, sh),
                  __builtin_amdgcn_alignbit(w3, w2, sh), w3 >> sh};
      };
      const bool whole = (s < full || !(KA || KB)) && (KA || ni == S::BI) && (KB || g.J - j0 >= S::BJ);
      if (eight && !whole) {
#pragma unroll
        for (int n = 0; n < decltype(la_)::value; ++n) down(rega[n], left(n, s, IntC<0>{}));
#pragma unroll
        for (int n = 0; n < S::LB; ++n) down(regb[n], left(n, s, IntC<1>{}));
      }
#pragma unroll
      for (int n = 0; n < decltype(la_)::value; ++n)
        *reinterpret_cast<lds_u32x4*>(lds0 + sa + (n * S::W + wave) * 1024 + lane * 16) = rega[n];
#pragma unroll
      for (int n = 0; n < S::LB; ++n)
        *reinterpret_cast<lds_u32x4*>(lds0 + 2 * S::StageA + sb + (n * S::W + wave) * 1024 + lane * 16) = regb[n];
    }
  };
  // Gathered sums: the rows of step s.  A block of row indexes is put into LDS
  // every kIndexCache rows.
  auto next_rows = [&](int s) {
    if constexpr (RowsB) {
      int32_t* const index_cache = reinterpret_cast<int32_t*>(smem + S::Lds);
      if (s * kStepK % kIndexCache == 0) {
        __syncthreads();  // the last block's entries are read
        for (int i = threadIdx.x; i < kIndexCache; i += S::Threads) {
          const int k = s * kStepK + i;
          index_cache[i] = k < klen ? source_row(g, row0 + k0 + k) : -1;
        }
        __syncthreads();
      }
#pragma unroll
      for (int n = 0; n < S::LB; ++n)
        src[n] = index_cache[(s * kStepK + krow(n * S::W + wave, S::BJ)) % kIndexCache];
    }
  };

  // ---- this wave's fragments.  Ragged rows: the waves take row blocks of 16 in
  // turn, so that the blocks of a tile's valid rows are spread over them.
  const int wi = wave % S::WI, wj = wave / S::WI, l16 = lane & 15, quad = lane >> 4;
  const int tr = quad * 8 + (l16 >> 2);  // a lane's row of a turned block
  const uint32_t chunk0 = (uint32_t)(quad ^ (l16 & 7)) << 4;
  const uint32_t fa0 = lds0 + (KA ? (wi * 16 + l16) * 128 + chunk0
                                  : tr * S::BI * 2 + (((wi * S::FI) ^ unit_swizzle<S::BI>(tr)) << 5) + (l16 & 3) * 8);
  const uint32_t fb0 = lds0 + 2 * S::StageA +
                       (KB ? (wj * S::FJ * 16 + l16) * 128 + chunk0
                           : tr * S::BJ * 2 + (((wj * S::FJ) ^ unit_swizzle<S::BJ>(tr)) << 5) + (l16 & 3) * 8);
  // fragment f of half h of a step; `stage`: bytes to its stage
  auto read_a = [&](int f, int h, uint32_t stage) {
    if constexpr (KA) return lds_read16((fa0 + stage) ^ (uint32_t)(h << 6), f * S::WI * 2048);
    else return lds_read_turned<S::BI>((fa0 + stage) ^ (uint32_t)(f << 5), h * 32 * S::BI * 2);
  };
  auto read_b = [&](int f, int h, uint32_t stage) {
    if constexpr (KB) return lds_read16((fb0 + stage) ^ (uint32_t)(h << 6), f * 2048);
    else return lds_read_turned<S::BJ>((fb0 + stage) ^ (uint32_t)(f << 5), h * 32 * S::BJ * 2);
  };

  f32x4 acc[S::FJ][S::FI] = {};
  u32x4 ra[2][S::FI], rb[2][S::FJ];

  // The sum with the first FA row fragments of each wave, LA loads of A a wave.
  auto sum = [&](auto fa_, auto la_) {
    constexpr int FA = decltype(fa_)::value, LA = decltype(la_)::value, F = FA + S::FJ;
    uint32_t sa = 0, sb = 0;  // bytes to the current step's stages
    // One step; its first half is in registers when it starts, or on the way.
    auto step = [&](int t, auto tail_) {
      const uint32_t sa1 = sa ^ S::StageA, sb1 = sb == (S::SB - 1) * S::StageB ? 0 : sb + S::StageB;
#pragma unroll
      for (int j = 0; j < S::FJ; ++j) {
#pragma unroll
        for (int f = j * F / S::FJ; f < (j + 1) * F / S::FJ; ++f) {
          if (f < S::FJ) rb[1][f] = read_b(f, 1, sb);
          else ra[1][f - S::FJ] = read_a(f - S::FJ, 1, sa);
        }
#pragma unroll
        for (int i = 0; i < FA; ++i) acc[j][i] = T::mfma(rb[0][j], ra[0][i], acc[j][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // step t + 1 has landed in LDS everywhere, and every wave has read step t:
      // its stages are free
      if constexpr (REG) {
        put(t + 1, sa1, sb1, la_);
        __syncthreads();
      } else {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S::SB - 2) * S::LB) : "memory");
      }
      next_rows(t + S::SB);
      fetch(t + 2, la_);
#pragma unroll
      for (int j = 0; j < S::FJ; ++j) {
        constexpr int L = REG ? 0 : LA + S::LB;
#pragma unroll
        for (int n = j * L / S::FJ; n < (j + 1) * L / S::FJ; ++n) {
          if (n < LA) issue_a(n, t + 2, lds0 + sa, tail_);
          else issue_b(n - LA, t + S::SB, lds0 + 2 * S::StageA + sb, tail_);
        }
#pragma unroll
        for (int f = j * F / S::FJ; f < (j + 1) * F / S::FJ; ++f) {
          if (f < S::FJ) rb[0][f] = read_b(f, 0, sb1);
          else ra[0][f - S::FJ] = read_a(f - S::FJ, 0, sa1);
        }
#pragma unroll
        for (int i = 0; i < FA; ++i) acc[j][i] = T::mfma(rb[1][j], ra[1][i], acc[j][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
      sa = sa1;
      sb = sb1;
    };
    if constexpr (REG) {
      next_rows(0);
      fetch(0, la_);
      put(0, 0, 0, la_);
      next_rows(1);
      fetch(1, la_);
      __syncthreads();
    } else {
#pragma unroll
      for (int s = 0; s < S::SB; ++s) {
        if (s < 2)
#pragma unroll
          for (int n = 0; n < LA; ++n) issue_a(n, s, lds0 + s * S::StageA, IntC<1>{});
        next_rows(s);
#pragma unroll
        for (int n = 0; n < S::LB; ++n) issue_b(n, s, lds0 + 2 * S::StageA + s * S::StageB, IntC<1>{});
      }
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LA + (S::SB - 1) * S::LB) : "memory");
    }
#pragma unroll
    for (int f = 0; f < S::FJ; ++f) rb[0][f] = read_b(f, 0, 0);
#pragma unroll
    for (int f = 0; f < FA; ++f) ra[0][f] = read_a(f, 0, 0);
    int t = 0;
    if constexpr (!REG)
      for (; t + S::SB < full; ++t) step(t, IntC<0>{});
    for (; t < nsteps; ++t) step(t, IntC<1>{});
  };
  // A tile with few valid rows does without the fragments of the others.
  constexpr int FI = S::FI, LA = S::LA;
  const int fa = ((ni + 15) / 16 + S::WI - 1) / S::WI;
  if (!KA || fa > FI * 3 / 4) {
    sum(IntC<FI>{}, IntC<LA>{});
  } else if constexpr (KA && FI >= 8) {
    if (fa > FI / 2) sum(IntC<FI * 3 / 4>{}, IntC<(LA * 3 + 3) / 4>{});
    else if (fa > FI / 4) sum(IntC<FI / 2>{}, IntC<(LA + 1) / 2>{});
    else sum(IntC<FI / 4>{}, IntC<(LA + 3) / 4>{});
  } else if constexpr (KA) {
    if (fa > FI / 2) sum(IntC<FI>{}, IntC<LA>{});
    else sum(IntC<FI / 2>{}, IntC<(LA + 1) / 2>{});
  }
  // loads past the end still write zeros to LDS: they end here, and every wave
  // has read its last fragments
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // ---- results: through LDS, 64 columns at a time, so that 16 lanes store one
  // row's 64 neighbouring columns, whole lines.  B's fragments are the matrix
  // instruction's A operand: a lane holds four neighbouring columns of one row.
  // Each wave uses its own part; the 16-byte chunk c of row r lies at c ^ (r % CH).
  // Plain results leave 16 bytes a lane at a scalar address and a lane's 32-bit
  // offset, four or eight rows' reads from LDS ahead of their stores: a weight
  // gradient of few rows an expert is bound by this part.  They pass the L2 (non-
  // temporal): other XCDs read them after the launch, whose end writes the L2
  // back anyway, and 2.3 GB of weight gradients take 611 us against 695.  Parts of
  // a split sum stay in it for the kernel that joins them (512 x 512 x 16384: 27.3
  // us against 29.1).
  constexpr int JC = S::JC, IC = S::IC, CH = JC * 4, Rows = IC * 16, RowBytes = JC * 64, At = 64 / CH, Q = 16 / At;
  const uint32_t own = lds0 + wave * Rows * RowBytes;
  void* const c = OP == kWgrad ? result_of(g, e) : g.c;
  const int64_t slice = g.splits > 1 ? (int64_t)blockIdx.y * (OP == kWgrad ? g.E : 1) + (OP == kWgrad ? e : 0) : 0;
  float* const part = g.splits > 1 ? g.part + (slice * g.I + i0) * g.J : nullptr;
  constexpr bool Factor = T::kType == kF16 && OP != kFwd;  // only a dense backward pass in fp16 has one
  const float factor = Factor && g.factor ? *g.factor : 1.0f;
  const int ch = lane % CH, lr = lane / CH;  // a lane's chunk and its first row of a part
  // row r0 + lr of the wave's part at x0: r0 of the tile, in scalar registers
  auto place = [&](int x0, int r0) {
    return KA ? ((x0 + r0 / 16) * S::WI + wi) * 16 + r0 % 16 : (wi * S::FI + x0) * 16 + r0;
  };
  auto value = [&](int x, int q) {  // row 16 x + At q + lr of the part
    return *reinterpret_cast<const lds_f32x4*>(
        reinterpret_cast<lds_char*>(own + (q * At + lr) * RowBytes + ((ch ^ ((q * At + lr) % CH)) << 4)) + x * 16 * RowBytes);
  };
#pragma unroll
  for (int y0 = 0; y0 < S::FJ; y0 += JC)
#pragma unroll
    for (int x0 = 0; x0 < S::FI; x0 += IC) {
#pragma unroll
      for (int y = 0; y < JC; ++y)
#pragma unroll
        for (int x = 0; x < IC; ++x)
          *reinterpret_cast<lds_f32x4*>(own + (x * 16 + l16) * RowBytes + (((y * 4 + quad) ^ (l16 % CH)) << 4)) =
              acc[y0 + y][x0 + x];
      const int jw = j0 + (wj * S::FJ + y0) * 16, j = jw + ch * 4;
      // E columns a lane: a part's rows of the wave, read from LDS together, then
      // stored; `all`: every row of the tile is valid; `past`: past the L2
      auto leave = [&](auto e_, auto all_, auto past_, const char* to, int64_t ld) {
        constexpr int E = decltype(e_)::value, Size = E == 8 ? 2 : 4, L = JC * 16 / E, A = 64 / L, N = 16 / A;
        const int c0 = lane % L * (E / 4), r0 = lane / L;
        if (jw + c0 * 4 >= g.J) return;
        const uint32_t off = (uint32_t)(r0 * ld + c0 * 4) * Size;
#pragma unroll
        for (int x = 0; x < IC; ++x) {
          f32x4 v[N][E / 4];
#pragma unroll
          for (int q = 0; q < N; ++q)
#pragma unroll
            for (int h = 0; h < E / 4; ++h)
              v[q][h] = *reinterpret_cast<const lds_f32x4*>(
                  reinterpret_cast<lds_char*>(own + (q * A + r0) * RowBytes + (((c0 + h) ^ ((q * A + r0) % CH)) << 4)) +
                  x * 16 * RowBytes);
          if constexpr (Factor && decltype(past_)::value)
#pragma unroll
            for (int q = 0; q < N; ++q)
#pragma unroll
              for (int h = 0; h < E / 4; ++h) v[q][h] *= factor;
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const int di = place(x0, x * 16 + q * A);
            if (!decltype(all_)::value && di + r0 >= ni) continue;
            char* const p = const_cast<char*>(uniform(to + di * ld * Size)) + off;
            if constexpr (E == 4) {
              if constexpr (decltype(past_)::value) __builtin_nontemporal_store(v[q][0], reinterpret_cast<f32x4_word*>(p));
              else *reinterpret_cast<f32x4*>(p) = v[q][0];
            } else {
              u32x4 o;
#pragma unroll
              for (int r = 0; r < 4; ++r)
                o[r] = (uint32_t)T::from_f32(v[q][r / 2][r % 2 * 2]) |
                       ((uint32_t)T::from_f32(v[q][r / 2][r % 2 * 2 + 1]) << 16);
              __builtin_nontemporal_store(o, reinterpret_cast<u32x4_any*>(p));
            }
          }
        }
      };
      if (part && g.J % 4 == 0) {
        leave(IntC<4>{}, IntC<0>{}, IntC<0>{}, reinterpret_cast<const char*>(part + jw), g.J);
      } else if (g.plain && !part) {
        const char* const to = static_cast<const char*>(c) + ((int64_t)i0 * g.ldc + jw) * (g.c_type == kF32 ? 4 : 2);
        if (g.c_type == kF32)
          ni == S::BI ? leave(IntC<4>{}, IntC<1>{}, IntC<1>{}, to, g.ldc) : leave(IntC<4>{}, IntC<0>{}, IntC<1>{}, to, g.ldc);
        else  // of the operands' type
          ni == S::BI ? leave(IntC<8>{}, IntC<1>{}, IntC<1>{}, to, g.ldc) : leave(IntC<8>{}, IntC<0>{}, IntC<1>{}, to, g.ldc);
      } else if (j < g.J) {
#pragma unroll 1
        for (int x = 0; x < IC; ++x) {
          f32x4 v[Q];
          int64_t row[Q];
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            v[q] = value(x, q);
            const int di = place(x0, x * 16 + q * At) + lr;
            row[q] = di < ni ? i0 + di : -1;
          }
          if (!part) {
            finish<Q, Factor>(g, c, row, j, 4, v);
          } else {
            const bool wide = __builtin_amdgcn_ballot_w64(g.J - j < 4) == 0;
#pragma unroll
            for (int q = 0; q < Q; ++q)
              if (row[q] >= 0) store4_from_f32(part, (row[q] - i0) * g.J + j, g.J - j, kF32, wide, v[q]);
          }
        }
      }
    }
}

template <typename T, int OP, bool REG, typename S>
void launch_shape(const ProductArgs& a, hipStream_t stream) {
  const int ct = (a.J + S::BJ - 1) / S::BJ;
  const int64_t rt = OP == kWgrad ? (int64_t)a.E * ((a.I + S::BI - 1) / S::BI) : row_tiles_most(a, S::BI);
  const dim3 grid((unsigned)((rt * ct + 7) / 8 * 8), (unsigned)a.splits);
  if (OP != kDgrad && a.rows)
    hipLaunchKernelGGL((product_lds_kernel<T, OP, OP != kDgrad, REG, S>), grid, dim3(S::Threads), 0, stream, a, ct);
  else
    hipLaunchKernelGGL((product_lds_kernel<T, OP, false, REG, S>), grid, dim3(S::Threads), 0, stream, a, ct);
}

template <typename T, int OP, int SB>
void launch_tiles(const ProductArgs& a, int shape, hipStream_t stream) {
  switch (shape) {
    case kBig: return launch_shape<T, OP, false, Shape<256, 256, 2, 4, SB, 2>>(a, stream);
    case kMid: return launch_shape<T, OP, false, Shape<128, 128, 2, 2, SB, 2>>(a, stream);
    case kLow: return launch_shape<T, OP, false, Shape<64, 128, 1, 4, 2, 3>>(a, stream);
    default: return launch_shape<T, OP, true, Shape<64, 128, 1, 4, 2, 3>>(a, stream);
  }
}

}  // namespace
}  // namespace moe_fp4
