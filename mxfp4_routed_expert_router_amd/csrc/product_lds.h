// 16-bit products through LDS tiles filled straight from memory.
//
// A workgroup computes BI x BJ results (i: rows of the result, j: its columns),
// 32 of the sum a step.  A ring of stages in LDS holds the next steps' operand
// tiles; global_load_lds_dwordx4 fills them without passing through registers,
// and the fragments of step t + 1 are read from LDS while the matrix
// instructions of step t run, so the matrix cores wait only at one barrier a
// step.
//
// LDS layout.  An operand that is contiguous along the sum (x, dy as the row
// side, w of forward) is held as [index][32]: 64-byte rows, the 16-byte chunk
// c of row r at slot c ^ chunk_swizzle(r), so that the 16 rows of a fragment
// read spread over all banks.  An operand that is contiguous along its own
// index (w of dgrad; both of wgrad) is held as it lies, [32][index], and
// ds_read_b64_tr_b16 turns 4 x 16 blocks on the way to the registers: within 16
// lanes, lane i receives column i of the four rows that lanes 4 r .. 4 r + 3
// address.  Its 32-byte units (16 indexes) of row r sit at unit ^ unit_swizzle(r).
#pragma once

#include "block_device.h"
#include "lds_dma.h"

namespace moe_fp4 {
namespace {

constexpr int kStepK = 32;
constexpr int kIndexCache = 1024;  // row indexes of a gathered sum held in LDS

__device__ const __align__(16) uint32_t zero_chunk[4] = {0u, 0u, 0u, 0u};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

__device__ __forceinline__ int chunk_swizzle(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }
// Units of rows r of which 8 (rows 0-3 and 8-11, say) are read together: they
// take 8 different 32-byte bank groups.
template <int BX>
__device__ __forceinline__ int unit_swizzle(int r) {
  if constexpr (BX >= 128) return (r & 3) | ((r >> 1) & 4);
  if constexpr (BX == 64) return ((r >> 1) & 1) | ((r >> 2) & 2);
  return (r >> 3) & 1;
}

__device__ __forceinline__ u32x4 lds_read16(uint32_t a) {
  return *reinterpret_cast<const lds_u32x4*>(a);
}
// 8 k-values of 16 indexes: two turned 4 x 16 blocks, 4 rows apart.
template <int BX>
__device__ __forceinline__ u32x4 lds_read_turned(uint32_t a) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(a));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(a + 4 * BX * 2));
  const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
  return u32x4{l.x, l.y, h.x, h.y};
}

// BI x BJ results, WI x WJ waves, ST stages; OCC waves per SIMD.
template <int BI_, int BJ_, int WI_, int WJ_, int ST_, int OCC_>
struct Shape {
  static constexpr int BI = BI_, BJ = BJ_, WI = WI_, WJ = WJ_, ST = ST_, OCC = OCC_;
  static constexpr int W = WI * WJ, Threads = 64 * W;
  static constexpr int FI = BI / WI / 16, FJ = BJ / WJ / 16;   // fragments of a wave
  static constexpr int NI = BI / 16, NJ = BJ / 16;             // 1 KB loads of a stage
  static constexpr int LPW = (NI + NJ) / W;                    // loads of a wave
  static constexpr int Stage = (BI + BJ) * 64;
  // fragments of columns of a pass of the epilogue: at most four, as fit the stages
  static constexpr int Fit = ST * Stage / (W * FI * 16 * 64);
  static constexpr int JC = FJ >= 4 && Fit >= 4 ? 4 : FJ >= 2 && Fit >= 2 ? 2 : 1;
  static_assert((NI + NJ) % W == 0 && ST >= 3, "every wave issues the same number of loads");
};

template <typename T, int OP, bool GATHER, typename S>
__global__ void __launch_bounds__(S::Threads, S::OCC) product_lds_kernel(ProductArgs g, int col_tiles) {
  constexpr bool KA = OP != kWgrad, KB = OP == kFwd;  // contiguous along the sum
  __shared__ __align__(1024) uint8_t smem[S::ST * S::Stage];
  __shared__ int32_t index_cache[GATHER && OP == kWgrad ? kIndexCache : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // ---- which tile: workgroups are dealt to the 8 XCDs round robin; each XCD
  // takes a contiguous run of tiles, four row tiles of each column tile in turn,
  // so that a run shares rows and weights in its L2
  const int rt_all = OP == kWgrad ? g.E * ((g.I + S::BI - 1) / S::BI) : row_tiles(g.offsets, g.E, g.P, S::BI);
  const int64_t total = (int64_t)rt_all * col_tiles;
  const int64_t per = (total + 7) / 8, slot = blockIdx.x >> 3, tile = (blockIdx.x & 7) * per + slot;
  if (slot >= per || tile >= total) return;
  constexpr int GR = 4;
  const int band = (int)(tile / (GR * col_tiles)), in = (int)(tile - (int64_t)band * GR * col_tiles);
  const int high = rt_all - band * GR < GR ? rt_all - band * GR : GR;
  const int rt = band * GR + in % high, j0 = in / high * S::BJ;
  int e, row0, nrows, i0, ni, klen;
  const uint16_t* b = g.b;
  if (OP == kWgrad) {
    const int it = (g.I + S::BI - 1) / S::BI;
    e = rt / it;
    i0 = (rt - e * it) * S::BI;
    ni = g.I - i0 < S::BI ? g.I - i0 : S::BI;
    segment(g.offsets, e, g.P, row0, klen);
  } else {
    if (!row_tile(g.offsets, g.E, g.P, S::BI, rt, e, row0, nrows)) return;
    i0 = row0;
    ni = nrows;
    klen = g.K;
    b += (int64_t)e * g.w_stride;
  }
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
  constexpr bool RowsA = GATHER && OP == kFwd, RowsB = GATHER && OP == kWgrad;
  const int first = OP == kWgrad ? row0 + k0 : k0;
  const char* const abase = reinterpret_cast<const char*>(
      KA ? g.a + (RowsA ? 0 : (int64_t)i0 * g.lda) + k0 : g.a + (int64_t)first * g.lda + i0);
  const char* const bbase = reinterpret_cast<const char*>(
      KB ? b + (int64_t)j0 * g.ldb + k0 : b + (RowsB ? 0 : (int64_t)first * g.ldb) + j0);
  const int64_t astep = KA ? kStepK * 2 : kStepK * 2 * g.lda, bstep = KB ? kStepK * 2 : kStepK * 2 * g.ldb;
  const char* const zero = reinterpret_cast<const char*>(zero_chunk);
  const int kchunk = ((lane & 3) ^ chunk_swizzle(lane >> 2)) * 8;  // a lane's place along the sum
  // turned operands: place along the sum of load u
  auto krow = [&](int u, int BX) { return u * (512 / BX) + lane / (BX / 8); };
  uint32_t off[S::LPW];
  const char* rowp[RowsA ? S::LPW : 1];  // gathered x of forward: the lane's row, or null
  int src[RowsB ? S::LPW : 1];           // gathered x of wgrad: the lane's row of the step to come, or -1
#pragma unroll
  for (int n = 0; n < S::LPW; ++n) {
    const int q = n * S::W + wave;
    const bool isa = q < S::NI;
    const int u = isa ? q : q - S::NI;
    if (isa ? KA : KB) {
      const int r = u * 16 + (lane >> 2), most = isa ? ni : g.J - j0;
      const int rr = r < most ? r : most - 1;
      off[n] = (uint32_t)(rr * (isa ? g.lda : g.ldb) + kchunk) * 2;
      if constexpr (RowsA)
        if (isa) {
          const int row = source_row(g, i0 + rr);
          rowp[n] = row < 0 ? nullptr : abase + ((int64_t)row * g.lda + kchunk) * 2;
        }
    } else {
      const int BX = isa ? S::BI : S::BJ, k = krow(u, BX), s = lane % (BX / 8);
      const int unit = (s >> 1) ^ (isa ? unit_swizzle<S::BI>(k) : unit_swizzle<S::BJ>(k));
      const int col = unit * 16 + (s & 1) * 8, most = isa ? g.I - i0 : g.J - j0;
      off[n] = (uint32_t)((RowsB && !isa ? 0 : k * (isa ? g.lda : g.ldb)) + (col < most ? col : most - 8)) * 2;
    }
  }
  const uint32_t lds0 = lds_addr(smem);
  // Load n of step s.  Past the end of the sum it brings zeros, so that every
  // step issues the same number of loads and the waits below are exact.
  auto issue = [&](int n, int s) {
    const int q = n * S::W + wave;
    const bool isa = q < S::NI;
    const uint32_t to = lds0 + (uint32_t)((s % S::ST) * S::Stage + q * 1024);
    const char* const base = isa ? abase + s * astep : bbase + s * bstep;
    const int u = isa ? q : q - S::NI;
    const int k = (isa ? KA : KB) ? kchunk : krow(u, isa ? S::BI : S::BJ);
    const bool past = s >= full && s * kStepK + k >= klen;
    if (RowsA && isa) {
      lds_load16(to, past || !rowp[RowsA ? n : 0] ? zero : rowp[RowsA ? n : 0] + s * astep);
    } else if (RowsB && !isa) {
      const int row = src[RowsB ? n : 0];  // -1 past the end
      lds_load16(to, row < 0 ? zero : bbase + (int64_t)row * g.ldb * 2 + off[n]);
    } else if (s < full) {
      lds_load16_at(to, base, off[n]);
    } else {
      lds_load16(to, past ? zero : base + off[n]);
    }
  };
  // Gathered sums: a block of row indexes is put into LDS every kIndexCache rows.
  auto fetch_indexes = [&](int s) {  // before step s's, s * 32 a multiple of kIndexCache
    for (int i = threadIdx.x; i < kIndexCache; i += S::Threads) {
      const int k = s * kStepK + i;
      index_cache[i] = k < klen ? source_row(g, row0 + k0 + k) : -1;
    }
    __syncthreads();
  };
  auto next_rows = [&](int s) {
#pragma unroll
    for (int n = 0; n < S::LPW; ++n)
      if (n * S::W + wave >= S::NI)
        src[RowsB ? n : 0] = index_cache[(s * kStepK + krow(n * S::W + wave - S::NI, S::BJ)) % kIndexCache];
  };
  auto issue_all = [&](int s) {
    if constexpr (RowsB) {
      if (s * kStepK % kIndexCache == 0) {
        __syncthreads();  // the last block's entries are read
        fetch_indexes(s);
      }
      next_rows(s);
    }
#pragma unroll
    for (int n = 0; n < S::LPW; ++n) issue(n, s);
  };

  // ---- this wave's fragments
  const int wi = wave % S::WI, wj = wave / S::WI, l16 = lane & 15, quad = lane >> 4;
  uint32_t fa0, fb0;
  if constexpr (KA)
    fa0 = wi * S::FI * 1024 + l16 * 64 + ((quad ^ chunk_swizzle(l16)) << 4);
  else {
    const int r = quad * 8 + (l16 >> 2);
    fa0 = r * S::BI * 2 + (((wi * S::FI) ^ unit_swizzle<S::BI>(r)) << 5) + (l16 & 3) * 8;
  }
  if constexpr (KB)
    fb0 = S::BI * 64 + wj * S::FJ * 1024 + l16 * 64 + ((quad ^ chunk_swizzle(l16)) << 4);
  else {
    const int r = quad * 8 + (l16 >> 2);
    fb0 = S::BI * 64 + r * S::BJ * 2 + (((wj * S::FJ) ^ unit_swizzle<S::BJ>(r)) << 5) + (l16 & 3) * 8;
  }
  fa0 += lds0;
  fb0 += lds0;
  auto read_a = [&](int f, uint32_t stage) {
    if constexpr (KA) return lds_read16(fa0 + stage + f * 1024);
    else return lds_read_turned<S::BI>((fa0 + stage) ^ (uint32_t)(f << 5));
  };
  auto read_b = [&](int f, uint32_t stage) {
    if constexpr (KB) return lds_read16(fb0 + stage + f * 1024);
    else return lds_read_turned<S::BJ>((fb0 + stage) ^ (uint32_t)(f << 5));
  };

  f32x4 acc[S::FJ][S::FI] = {};
  u32x4 ra[2][S::FI], rb[2][S::FJ];

  // One step: when it starts, its fragments are in registers (`cur`) or on
  // their way there.
  auto step = [&](int t, auto cur_) {
    constexpr int cur = decltype(cur_)::value, nxt = cur ^ 1;
    // step t + 1 has landed in LDS everywhere, and every wave has read step t
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S::ST - 2) * S::LPW) : "memory");
    const uint32_t stage = (uint32_t)((t + 1) % S::ST) * S::Stage;
    if constexpr (RowsB) issue_all(t + S::ST);
#pragma unroll
    for (int j = 0; j < S::FJ; ++j) {
      if constexpr (!RowsB)
#pragma unroll
        for (int n = j * S::LPW / S::FJ; n < (j + 1) * S::LPW / S::FJ; ++n) issue(n, t + S::ST);
      constexpr int F = S::FI + S::FJ;
#pragma unroll
      for (int f = j * F / S::FJ; f < (j + 1) * F / S::FJ; ++f) {
        if (f < S::FJ) rb[nxt][f] = read_b(f, stage);
        else ra[nxt][f - S::FJ] = read_a(f - S::FJ, stage);
      }
#pragma unroll
      for (int i = 0; i < S::FI; ++i) acc[j][i] = T::mfma(rb[cur][j], ra[cur][i], acc[j][i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int s = 0; s < S::ST; ++s) issue_all(s);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S::ST - 1) * S::LPW) : "memory");
#pragma unroll
  for (int f = 0; f < S::FJ; ++f) rb[0][f] = read_b(f, 0);
#pragma unroll
  for (int f = 0; f < S::FI; ++f) ra[0][f] = read_a(f, 0);
  for (int t = 0; t < nsteps; t += 2) {  // an odd last step is followed by one of zeros
    step(t, IntC<0>{});
    step(t + 1, IntC<1>{});
  }
  // loads past the end still write zeros to LDS: they end here, and every wave
  // has read its last fragments
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // ---- results: through LDS, 64 columns at a time, so that 16 lanes store one
  // row's 64 neighbouring columns.  B's fragments are the matrix instruction's
  // A operand: a lane holds four neighbouring columns of one row.  Each wave
  // uses its own part; the 16-byte chunk c of row r lies at c ^ (r % 16).
  constexpr int JC = S::JC, CH = JC * 4, Rows = S::FI * 16, RowBytes = JC * 64;
  static_assert(S::W * Rows * RowBytes <= S::ST * S::Stage && S::FJ % JC == 0, "the parts fit the stages");
  const uint32_t own = lds0 + wave * Rows * RowBytes;
  void* const c = OP == kWgrad ? result_of(g, e) : g.c;
  const int64_t slice = g.splits > 1 ? (int64_t)blockIdx.y * (OP == kWgrad ? g.E : 1) + (OP == kWgrad ? e : 0) : 0;
  float* const part = g.splits > 1 ? g.part + (slice * g.I + i0) * g.J : nullptr;
#pragma unroll
  for (int y0 = 0; y0 < S::FJ; y0 += JC) {
#pragma unroll
    for (int y = 0; y < JC; ++y)
#pragma unroll
      for (int x = 0; x < S::FI; ++x)
        *reinterpret_cast<lds_f32x4*>(own + (x * 16 + l16) * RowBytes + (((y * 4 + quad) ^ (l16 % CH)) << 4)) =
            acc[y0 + y][x];
    const int ch = lane % CH, j = j0 + (wj * S::FJ + y0) * 16 + ch * 4;
#pragma unroll 1
    for (int r = lane / CH; r < Rows; r += 64 / CH) {
      const int di = wi * Rows + r;
      if (di >= ni || j >= g.J) continue;
      const f32x4 v = *reinterpret_cast<const lds_f32x4*>(own + r * RowBytes + ((ch ^ (r % 16 % CH)) << 4));
      if (!part) {
        finish4(g, c, i0 + di, j, v);
        continue;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k < g.J) part[(int64_t)di * g.J + j + k] = v[k];
    }
  }
}

template <typename T, int OP, typename S>
void launch_shape(const ProductArgs& a, hipStream_t stream) {
  const int ct = (a.J + S::BJ - 1) / S::BJ;
  const int64_t rt = OP == kWgrad ? (int64_t)a.E * ((a.I + S::BI - 1) / S::BI) : row_tiles_most(a, S::BI);
  const dim3 grid((unsigned)((rt * ct + 7) / 8 * 8), (unsigned)a.splits);
  if (OP != kDgrad && a.rows)
    hipLaunchKernelGGL((product_lds_kernel<T, OP, OP != kDgrad, S>), grid, dim3(S::Threads), 0, stream, a, ct);
  else
    hipLaunchKernelGGL((product_lds_kernel<T, OP, false, S>), grid, dim3(S::Threads), 0, stream, a, ct);
}


using Big = Shape<256, 256, 2, 4, 4, 2>;
using Mid = Shape<128, 128, 2, 2, 4, 2>;
using Low = Shape<64, 128, 1, 4, 4, 3>;
enum { kBig, kMid, kLow };

// The tile shape of a product.  Rates of the three at 4096^3 (bf16, forward /
// dgrad / wgrad): Big 1161 / 1193 / 1218 TFLOP/s, Mid 848 / 940 / 993, Low 640 /
// 756 / 806; so the larger where its tiles occupy most of the 256 CUs and the
// experts' rows fill most of a tile.  With 32 rows an expert (48 experts, 2304 x
// 5120) Low takes 264 / 241 us for forward / dgrad, Mid 276 / 244, Big 330 /
// 289, while wgrad, bound by its writes, takes 589, 574 and 513.
inline int product_shape(const ProductArgs& a, int op) {
  const int64_t live = !a.offsets ? 1 : a.E < a.P ? a.E : a.P;
  const int64_t groups = op == kWgrad ? a.E : live ? live : 1;   // experts with results
  const int64_t rows = op == kWgrad ? a.I : (a.P + groups - 1) / groups;  // of one, on average
  const auto tiles = [&](int bi, int bj) { return groups * ((rows + bi - 1) / bi) * ((a.J + bj - 1) / bj); };
  constexpr int kBusy = 200;
  if (rows > 128 && tiles(256, 256) >= kBusy) return kBig;
  if (rows > 64 && tiles(128, 128) >= kBusy) return kMid;
  return kLow;
}

}  // namespace
}  // namespace moe_fp4
