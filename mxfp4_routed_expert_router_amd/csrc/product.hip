// 16-bit products grouped by expert (and dense, as one expert) on the matrix cores.
#include "block_device.h"

namespace moe_fp4 {
namespace {

// ---------------------------------------------------------------- any sizes, any alignment
// 64 x 64 results a workgroup of four waves (32 x 32 each), 32 of the sum at a
// time through LDS as [index][k].  Elements are loaded one by one where a row
// is not 16-byte aligned or ends inside a chunk, so every size and stride runs
// here.
constexpr int kAnyTile = 64, kAnyK = 32, kAnyPad = 40;

// Eight elements p[0..7], those from n on as zeros.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n, bool wide) {
  if (n >= 8 && wide) return ld16(p);
  uint16_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0;
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)v[2 * i] | ((uint32_t)v[2 * i + 1] << 16);
  return o;
}

template <typename T, int OP>
__global__ void __launch_bounds__(256) product_any_kernel(ProductArgs g, int row_tiles, int col_tiles) {
  __shared__ __align__(16) uint16_t sa[kAnyTile * kAnyPad], sb[kAnyTile * kAnyPad];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
  int e, row0 = 0, nrows = 0, i0, j0 = ct * kAnyTile, ni, klen;
  const uint16_t* b = g.b;
  if (OP == kWgrad) {
    e = rt / row_tiles;
    i0 = (rt % row_tiles) * kAnyTile;
    ni = g.I - i0;
    segment(g.offsets, e, g.P, row0, klen);
  } else {
    if (!row_tile(g.offsets, g.E, g.P, kAnyTile, rt, e, row0, nrows)) return;
    i0 = row0;
    ni = nrows;
    klen = g.K;
    b += (int64_t)e * g.w_stride;
  }
  // this workgroup's part of the sum
  int k0 = 0, k1 = klen;
  if (g.splits > 1) {
    const int per = ((klen + g.splits - 1) / g.splits + kAnyK - 1) / kAnyK * kAnyK;
    k0 = (int)blockIdx.y * per;
    k1 = k0 + per < klen ? k0 + per : klen;
  }
  const bool wa = (((uintptr_t)g.a | (uintptr_t)(g.lda * 2)) & 15) == 0;
  const bool wb = (((uintptr_t)b | (uintptr_t)(g.ldb * 2)) & 15) == 0;
  // along k: thread t loads index t / 4, k chunk t % 4; along the index: k t / 8, index chunk t % 8
  const int kr = t >> 2, kc = (t & 3) * 8, sr = t >> 3, sc = (t & 7) * 8;
  int64_t arow = -1;
  if (OP == kFwd && kr < ni) {
    const int s = source_row(g, i0 + kr);
    if (s >= 0) arow = (int64_t)s * g.lda;
  }
  if (OP == kDgrad && kr < ni) arow = (int64_t)(i0 + kr) * g.lda;
  f32x4 acc[2][2] = {};
  for (int k = k0; k < k1; k += kAnyK) {
    u32x4 va = zero4(), vb = zero4();
    if (OP != kWgrad) {
      if (arow >= 0) va = load8(g.a + arow + k + kc, k1 - k - kc, wa);
    } else if (k + sr < k1) {
      va = load8(g.a + (int64_t)(row0 + k + sr) * g.lda + i0 + sc, g.I - i0 - sc, wa);
    }
    if (OP == kFwd) {
      if (j0 + kr < g.J) vb = load8(b + (int64_t)(j0 + kr) * g.ldb + k + kc, k1 - k - kc, wb);
    } else if (k + sr < k1) {
      const int s = OP == kWgrad ? source_row(g, row0 + k + sr) : k + sr;
      if (s >= 0) vb = load8(b + (int64_t)s * g.ldb + j0 + sc, g.J - j0 - sc, wb);
    }
    __syncthreads();  // the previous step's reads are done
    if (OP != kWgrad) {
      st16(sa + kr * kAnyPad + kc, va);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) sa[(sc + i) * kAnyPad + sr] = (uint16_t)(va[i / 2] >> (16 * (i & 1)));
    }
    if (OP == kFwd) {
      st16(sb + kr * kAnyPad + kc, vb);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) sb[(sc + i) * kAnyPad + sr] = (uint16_t)(vb[i / 2] >> (16 * (i & 1)));
    }
    __syncthreads();
    u32x4 fa[2], fb[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      fa[x] = ld16(sa + ((wave & 1) * 32 + x * 16 + (lane & 15)) * kAnyPad + (lane >> 4) * 8);
      fb[x] = ld16(sb + ((wave >> 1) * 32 + x * 16 + (lane & 15)) * kAnyPad + (lane >> 4) * 8);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x) acc[y][x] = T::mfma(fb[y], fa[x], acc[y][x]);
  }
  // B's rows are the matrix instruction's A operand: a lane holds four
  // neighbouring columns of one result row
  void* c = OP == kWgrad ? result_of(g, e) : g.c;
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int di = (wave & 1) * 32 + x * 16 + (lane & 15);
      const int j = j0 + (wave >> 1) * 32 + y * 16 + (lane >> 4) * 4;
      if (di >= ni || j >= g.J) continue;
      if (g.splits > 1) {
        const int64_t slice = (int64_t)blockIdx.y * (OP == kWgrad ? g.E : 1) + (OP == kWgrad ? e : 0);
        float* p = g.part + (slice * g.I + i0 + di) * g.J + j;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j + r < g.J) p[r] = acc[y][x][r];
      } else {
        finish4(g, c, i0 + di, j, acc[y][x]);
      }
    }
}

// The parts of a split sum, added in order, then the epilogue.  Four columns a
// thread.  Rows that no expert owns are left alone.
template <int OP>
__global__ void __launch_bounds__(256) product_join_kernel(ProductArgs g, int chunks) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rows = OP == kWgrad ? (int64_t)g.E * g.I : g.I;
  const int64_t i = id / chunks;
  const int j = (int)(id % chunks) * 4;
  if (i >= rows) return;
  if (OP != kWgrad && g.offsets && (i < g.offsets[0] || i >= g.offsets[g.E])) return;
  f32x4 v = {};
  for (int s = 0; s < g.splits; ++s) {
    const float* p = g.part + ((int64_t)s * rows + i) * g.J + j;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (j + r < g.J) v[r] += p[r];
  }
  if (OP == kWgrad)
    finish4(g, result_of(g, (int)(i / g.I)), i % g.I, j, v);
  else
    finish4(g, g.c, i, j, v);
}

bool product_lds_takes(const ProductArgs& a, int op) {
  constexpr int64_t kMaxStride = 1 << 22;  // a tile's byte offsets stay within 32 bits
  const auto ok = [](const uint16_t* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && ld <= kMaxStride;
  };
  if (!ok(a.a, a.lda) || !ok(a.b, a.ldb) || a.w_stride % 8) return false;
  if (op == kFwd) return a.K % 8 == 0;
  if (op == kDgrad) return a.K % 8 == 0 && a.J % 8 == 0;
  return a.I % 8 == 0 && a.J % 8 == 0;
}

template <typename T>
void launch_any(const ProductArgs& a, int op, hipStream_t stream) {
  const int ct = (a.J + kAnyTile - 1) / kAnyTile;
  const int it = (a.I + kAnyTile - 1) / kAnyTile;
  const int64_t rt = op == kWgrad ? (int64_t)it * a.E : row_tiles_most(a, kAnyTile);
  const dim3 grid((unsigned)(rt * ct), (unsigned)a.splits);
  switch (op) {
    case kFwd: hipLaunchKernelGGL((product_any_kernel<T, kFwd>), grid, dim3(256), 0, stream, a, it, ct); break;
    case kDgrad: hipLaunchKernelGGL((product_any_kernel<T, kDgrad>), grid, dim3(256), 0, stream, a, it, ct); break;
    default: hipLaunchKernelGGL((product_any_kernel<T, kWgrad>), grid, dim3(256), 0, stream, a, it, ct); break;
  }
}

}  // namespace

size_t product_workspace(const ProductArgs&, int) { return 0; }

hipError_t launch_product(ProductArgs a, int op, void*, hipStream_t stream) {
  a.splits = 1;
  if (op != kWgrad && a.P == 0) return hipSuccess;
  const auto four = [](const void* p, int64_t ld, int type) {  // rows take 4 elements at once
    return !p || ((reinterpret_cast<uintptr_t>(p) & (type == kF32 ? 15 : 7)) == 0 && ld % 4 == 0);
  };
  a.wide = a.J % 4 == 0 && four(a.c, a.ldc, a.c_type) && a.c_stride % 4 == 0 &&
           four(a.bias, 0, a.bias_type) && four(a.residual, a.ldr, a.c_type) && four(a.z, a.ldz, a.type);
  if (product_lds_takes(a, op)) {
    if (op == kFwd) launch_product_fwd(a, stream);
    else if (op == kDgrad) launch_product_dgrad(a, stream);
    else launch_product_wgrad(a, stream);
  } else if (a.type == kBf16)
    launch_any<Bf16>(a, op, stream);
  else
    launch_any<F16>(a, op, stream);
  return hipGetLastError();
}

}  // namespace moe_fp4
