// 16-bit products grouped by expert, and dense as one expert: which kernel runs,
// and the joining of split sums.
#include "block_device.h"

namespace moe_fp4 {
namespace {

constexpr int kSumStep = 64;
constexpr double kMaxParts = 256e6;  // bytes of a split sum's parts

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
    if (g.J - j >= 4) {
      v += *reinterpret_cast<const f32x4_word*>(p);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (j + r < g.J) v[r] += p[r];
    }
  }
  if (OP == kWgrad)
    finish1<true>(g, result_of(g, (int)(i / g.I)), i % g.I, j, 4, v);
  else
    finish1<true>(g, g.c, i, j, 4, v);
}

// Whether both operands' rows are 16-byte aligned and a multiple of 8 long.
bool wide_rows(const ProductArgs& a, int op) {
  const auto ok = [](const uint16_t* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0;
  };
  if (!ok(a.a, a.lda) || !ok(a.b, a.ldb) || a.w_stride % 8) return false;
  if (op == kFwd) return a.K % 8 == 0;
  if (op == kDgrad) return a.K % 8 == 0 && a.J % 8 == 0;
  return a.I % 8 == 0 && a.J % 8 == 0;
}

// How a product runs, from its sizes alone.
struct Tiles {
  double us;   // estimated time
  int shape;   // where the rows allow it (kAny otherwise)
  int splits;  // of the sum
};
struct Plan {
  int rows;         // forward: 1, 2 or 4 rows a wave, 16 for the few-row kernel, 0 for tiles
  int cut;          // tiles: columns of the first launch; the others take `rest`
  Tiles main, rest;
};

// The tile shape and the number of parts of the sum that come out fastest for J
// columns, by these measurements (us for a step of 64 of the sum, bf16, K = 5120;
// the forms differ by a few percent):
//   Big 256 x 256   up to 180 workgroups 1.22, 256: 1.5, 512: 2.9, 768: 4.35
//   Mid 128 x 128   up to 256: 0.55, 512: 0.94, 768: 1.37, 1024: 1.8
//   Low 64 x 128    up to 256: 0.54, 512: 0.67, 768: 0.98, 1024: 1.32
// So Big goes in rounds of one workgroup a CU, the others flow.  A ragged tile
// with few rows takes less; the weights of all experts take their bytes' time
// whatever the shape (48 experts of 2304 x 5120, 8, 32, 128 and 256 rows each:
// Big 202, 205, 249, 360 us; Mid 200, 212, 309, 410; Low 228, 233, 332, 526).
// Splitting the sum adds a launch and the parts' way to memory and back.
// The estimate does not ask for the rows' alignment: a product whose rows take the
// tiles of any alignment has the splits and the cut of the aligned shapes (2047 x 2303
// x 5119, f16: 122 us forward, 116 rows' gradient, 136 weights' gradient; the library's
// forward 82).
Tiles best_tiles(const ProductArgs& a, int op, int J) {
  static const struct { int bi, bj, occ; double us[3], thin; } kShapes[3] = {
      {256, 256, 1, {1.5, 1.5, 1.5}, 0.45}, {128, 128, 2, {0.55, 0.94, 0.94}, 0.5}, {64, 128, 3, {0.54, 0.67, 0.98}, 0.6}};
  const int64_t live = !a.offsets ? 1 : a.E < a.P ? a.E : a.P > 0 ? a.P : 1;
  const int64_t groups = op == kWgrad ? a.E : live;               // experts with results
  const double rows = op == kWgrad ? a.I : (double)a.P / groups;  // of one, on average
  const double sum = op == kWgrad ? (double)a.P / live : a.K;     // its length
  const bool ragged = op != kWgrad && a.offsets;
  const double results = (double)(op == kWgrad ? (int64_t)a.E * a.I : a.I) * J;
  const double memory = (op == kWgrad ? results * 2 : (double)live * a.K * J * 2) / 5.2e6;
  Tiles best{1e30, kLow, 1};
  for (int s = 0; s < 3; ++s) {
    const auto& h = kShapes[s];
    const double ct = (J + h.bj - 1) / h.bj;
    double tiles;
    if (!ragged) {
      tiles = ct * groups * (((int64_t)rows + h.bi - 1) / h.bi);
    } else {  // half a tile more than the rows fill, on average
      const double nt = rows / h.bi + 0.5 > 1 ? rows / h.bi + 0.5 : 1;
      tiles = ct * groups * (h.thin * nt + (1 - h.thin) * rows / h.bi);
    }
    for (int n = 1; n <= 16; n *= 2) {
      const int64_t steps = (int64_t)(sum / n + kSumStep - 1) / kSumStep;
      if (n > 1 && (steps < 4 || results * 4 * n > kMaxParts)) break;
      const double wgs = tiles * n, at = 256.0 * h.occ, rounds = wgs / at;
      double step;
      if (s == kBig && !ragged) {
        const double whole = (double)(int64_t)rounds, rest = wgs - whole * at;
        step = 1.5 * whole + (rest > 192 ? 1.5 : rest > 0 ? 1.22 : 0);
      } else {
        step = rounds > 1 ? rounds * h.us[h.occ - 1] : h.us[wgs <= 256 ? 0 : wgs <= 512 ? 1 : 2];
      }
      double us = step * (steps + 3);
      if (us < memory) us = memory;
      if (n > 1) us += 6.0 + 2 * n * results * 4 / 4e6;
      if (us < best.us * 0.97) best = {us, s, n};
    }
  }
  return best;
}

Plan plan(const ProductArgs& a, int op) {
  Plan p{};
  if (op == kFwd) {
    // one to four rows: the weights once, straight to registers.  Grouped up to
    // one row an expert on average: 96 rows on 48 of 138 experts 199 us, tiles
    // 235; 192 on 69: 335, 313.
    if (a.offsets ? a.P <= a.E : a.P <= 4) {
      p.rows = a.offsets ? (a.P <= 8 ? 1 : 4) : a.P <= 2 ? a.P : 4;
      return p;
    }
    if (!a.offsets && a.P <= 16) {
      p.rows = 16;
      return p;
    }
  }
  p.main = best_tiles(a, op, a.J);
  p.cut = a.J;
  // A dense product's last round of Big tiles may leave most CUs idle: the
  // columns of the whole rounds go first, the others in a launch of their own
  // (2048 x 9216 x 5120, 288 tiles: 154 us, 175 at once).
  if (!a.offsets) {
    const int64_t rt = (a.I + 255) / 256, ct = (a.J + 255) / 256, rounds = rt * ct / 256;
    const int cut = (int)(rounds * 256 / rt) * 256;
    if (rounds >= 1 && cut > 0 && cut < a.J) {
      const Tiles rest = best_tiles(a, op, a.J - cut);
      const double us = 1.5 * rounds * (double)((a.K + kSumStep - 1) / kSumStep + 3) + rest.us;
      if (us < p.main.us * 0.97) {
        p.main = {us, kBig, 1};
        p.rest = rest;
        p.cut = cut;
      }
    }
  }
  return p;
}

// The product's columns from j0 on, n of them.
ProductArgs columns(const ProductArgs& a, int op, int j0, int n) {
  ProductArgs r = a;
  const auto shift = [&](const void* p, int type) -> const void* {
    return p ? static_cast<const char*>(p) + (int64_t)j0 * (type == kF32 ? 4 : 2) : nullptr;
  };
  r.J = n;
  r.b = a.b + (op == kFwd ? j0 * a.ldb : j0);
  r.c = const_cast<void*>(shift(a.c, a.c_type));
  r.bias = shift(a.bias, a.bias_type);
  r.residual = shift(a.residual, a.c_type);
  r.z = const_cast<void*>(shift(a.z, a.type));
  return r;
}

size_t part_bytes(const ProductArgs& a, int op, int J, int splits) {
  return splits <= 1 ? 0 : (size_t)splits * (op == kWgrad ? (size_t)a.E * a.I : (size_t)a.I) * J * 4;
}

void launch_tiles(ProductArgs a, int op, const Tiles& t, hipStream_t stream) {
  a.splits = t.splits;
  const int shape = wide_rows(a, op) ? t.shape : kAny;
  if (op == kFwd)
    launch_product_fwd(a, shape, stream);
  else if (op == kDgrad)
    launch_product_dgrad(a, shape, stream);
  else
    launch_product_wgrad(a, shape, stream);
  if (a.splits > 1) {
    const int chunks = (a.J + 3) / 4;
    const int64_t threads = (op == kWgrad ? (int64_t)a.E : 1) * a.I * chunks;
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (op == kWgrad)
      hipLaunchKernelGGL(product_join_kernel<kWgrad>, grid, dim3(256), 0, stream, a, chunks);
    else
      hipLaunchKernelGGL(product_join_kernel<kFwd>, grid, dim3(256), 0, stream, a, chunks);
  }
}

}  // namespace

ProductChoice product_choice(const ProductArgs& a, int op) {
  const Plan p = plan(a, op);
  const bool wide = wide_rows(a, op);
  return {p.rows, wide ? p.main.shape : kAny, p.main.splits, p.cut, wide ? p.rest.shape : kAny, p.rest.splits};
}

size_t product_workspace(const ProductArgs& a, int op) {
  if (op != kWgrad && a.P == 0) return 0;
  const Plan p = plan(a, op);
  if (p.rows) return 0;
  const size_t m = part_bytes(a, op, p.cut, p.main.splits), r = part_bytes(a, op, a.J - p.cut, p.rest.splits);
  return m > r ? m : r;
}

hipError_t launch_product(ProductArgs a, int op, void* ws, hipStream_t stream) {
  if (op != kWgrad && a.P == 0) return hipSuccess;
  a.plain = !a.bias && !a.residual && !a.z && !a.accumulate && a.act == kActNone &&
            a.J % (a.c_type == kF32 ? 4 : 8) == 0;
  a.part = static_cast<float*>(ws);
  a.splits = 1;
  const Plan p = plan(a, op);
  if (p.rows == 16) {
    launch_product_few(a, stream);
  } else if (p.rows) {
    launch_product_row(a, p.rows, stream);
  } else if (p.cut == a.J) {
    launch_tiles(a, op, p.main, stream);
  } else {
    launch_tiles(columns(a, op, 0, p.cut), op, p.main, stream);
    launch_tiles(columns(a, op, p.cut, a.J - p.cut), op, p.rest, stream);
  }
  return hipGetLastError();
}

}  // namespace moe_fp4
