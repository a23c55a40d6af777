// The router's losses: per-expert counts, the balance loss and the z loss of every
// sequence, and the gradient of the logits.
//
// With n the sequence's unmasked tokens and p a token's probabilities (softmax of
// its logits, or sigmoids divided by their sum),
//   balance = E / (k n^2) sum_e counts[e] probs[e],  probs[e] = sum_t p[t][e]
//   z = sum_t lse_t^2 / n,  lse = log sum exp
// and with c_e = dbalance E counts[e] / (k n^2),
//   dl_e = p_e (c_e - sum_i p_i c_i) [softmax], times 1 - sigmoid(l_e) [sigmoid]
//        + 2 dz lse softmax_e / n + the gates' part at the chosen experts.
//
// Both passes read the logits once and are bound by those bytes.  A wave takes a
// token, lane l the columns 128 c + 2 l and + 1, so that a lane keeps the same
// columns for every token: the sums over tokens stay in registers, and so do the
// coefficients c of the backward pass.
#include "block_device.h"
#include "router_loss.h"

namespace moe_fp4 {
namespace {

constexpr int kLossWaves = 8;
constexpr int kLossBlocks = 512;  // most workgroups of the forward pass: two a CU

// A row of partial results: the sums of p, the counts, z's sum, the tokens.
__host__ __device__ inline int64_t loss_row(int E) { return 2 * (int64_t)E + 2; }

// Sequence s is tokens [lo, hi).  The offsets are device data that the host has not
// seen: they are held to [0, T], so that no value makes an access leave an array.
__device__ __forceinline__ int seq_at(const RouterLossArgs& g, int s) {
  if (!g.seqs) return s ? g.T : 0;
  const int v = g.seqs[s];
  return v < 0 ? 0 : v > g.T ? g.T : v;
}
// The first sequence that ends past token t (S where none does).
__device__ __forceinline__ int seq_of(const RouterLossArgs& g, int t) {
  int lo = 0, hi = g.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_at(g, mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef f32x2 __attribute__((aligned(4))) f32x2_word;
typedef uint32_t __attribute__((aligned(2))) u32_half;

// Columns j and j + 1 of a row, -inf past the last.
template <typename T>
__device__ __forceinline__ f32x2 load_pair(const void* p, int64_t row, int j, int E) {
  f32x2 v = {-INFINITY, -INFINITY};
  if constexpr (T::kType == kF32) {
    const float* const q = static_cast<const float*>(p) + row + j;
    if (j + 1 < E) v = *reinterpret_cast<const f32x2_word*>(q);
    else if (j < E) v[0] = *q;
  } else {
    const uint16_t* const q = static_cast<const uint16_t*>(p) + row + j;
    if (j + 1 < E) {
      const uint32_t h = *reinterpret_cast<const u32_half*>(q);
      v = f32x2{T::to_f32((uint16_t)h), T::to_f32((uint16_t)(h >> 16))};
    } else if (j < E) {
      v[0] = T::to_f32(*q);
    }
  }
  return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
  v = fmaxf(v, __uint_as_float(dpp_u32<0xB1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_u32<0x4E>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_u32<0x124>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_u32<0x128>(__float_as_uint(v))));
  const float r0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
  const float r1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 16));
  const float r2 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 32));
  const float r3 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 48));
  return fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
}

// A token's scores: soft = exp(l - m), or, with sigmoids, `p` their values times a
// common power; sum and soft_sum their sums.  For logits that are all negative the
// sigmoids are taken as e^(l - m) / (1 + e^l), so that their quotients keep their
// digits where the sigmoids themselves would be 0 in fp32.  A row of -inf alone has
// no probabilities: its sums are 0, and so are their reciprocals and its lse.
template <int NC>
struct Scores {
  f32x2 soft[NC], p[NC], down[NC];  // down: 1 - sigmoid
  float inv, soft_inv, lse;
};
template <int NC>
__device__ __forceinline__ void scores(const f32x2 (&l)[NC], bool sigmoid, Scores<NC>& o) {
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < NC; ++c) m = fmaxf(m, fmaxf(l[c][0], l[c][1]));
  m = wave_max_f32(m);
  if (m == -INFINITY) m = 0.f;
  float soft_sum = 0.f, sum = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.soft[c][i] = exp_f32(l[c][i] - m);
      soft_sum += o.soft[c][i];
    }
  soft_sum = wave_sum_f32(soft_sum);
  o.soft_inv = soft_sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(soft_sum);
  o.lse = soft_sum == 0.f ? 0.f : m + __builtin_amdgcn_logf(soft_sum) * 0.6931471805599453f;
  if (!sigmoid) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      o.p[c] = o.soft[c];
      o.down[c] = f32x2{1.f, 1.f};
    }
    o.inv = o.soft_inv;
    return;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float v = l[c][i], t = exp_f32(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.0f + t), low = t * r;
      o.p[c][i] = m < 0.f ? o.soft[c][i] * r : v < 0.f ? low : r;
      o.down[c][i] = v < 0.f ? r : low;
      sum += o.p[c][i];
    }
  sum = wave_sum_f32(sum);
  o.inv = sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum);
}

// Workgroup b takes the tokens [b B, (b + 1) B), B = tokens_of_block, one piece for
// each sequence among them.  Piece (b, s) writes row b + s of `part`: along the
// pieces b or s grows, so that no two share a row.
template <typename T, int NC>
__global__ void __launch_bounds__(kLossWaves * 64) router_loss_kernel(RouterLossArgs g) {
  __shared__ f32x2 sums[kLossWaves][NC * 64];
  __shared__ int32_t counts[NC * 128];
  __shared__ float zsum[kLossWaves];
  __shared__ int32_t tokens[kLossWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * g.tokens_of_block;
  const int t1 = g.T - t0 < g.tokens_of_block ? g.T : t0 + g.tokens_of_block;
  for (int s = seq_of(g, t0); s < g.S; ++s) {
    int lo = seq_at(g, s), hi = seq_at(g, s + 1);
    if (lo >= t1) break;
    lo = lo < t0 ? t0 : lo;
    hi = hi > t1 ? t1 : hi;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < NC * 128; e += kLossWaves * 64) counts[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < (hi - lo) * g.k; p += kLossWaves * 64) {
      const int t = lo + p / g.k;
      const int e = g.idx[(int64_t)lo * g.k + p];
      if ((!g.mask || g.mask[t]) && e >= 0 && e < g.E) atomicAdd(&counts[e], 1);
    }
    f32x2 acc[NC] = {};
    float zz = 0.f;
    int n = 0;
    for (int t = lo + wave; t < hi; t += kLossWaves) {
      if (g.mask && !g.mask[t]) continue;
      f32x2 l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = load_pair<T>(g.logits, t * g.ld, c * 128 + lane * 2, g.E);
      Scores<NC> o;
      scores<NC>(l, g.score == kScoreSigmoid, o);
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] += o.p[c] * o.inv;
      zz += o.lse * o.lse;
      ++n;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) sums[wave][c * 64 + lane] = acc[c];
    if (lane == 0) {
      zsum[wave] = zz;
      tokens[wave] = n;
    }
    __syncthreads();
    float* const out = g.part + (int64_t)(blockIdx.x + s) * loss_row(g.E);
    for (int e = threadIdx.x; e < g.E; e += kLossWaves * 64) {
      float v = sums[0][e >> 1][e & 1];
#pragma unroll
      for (int w = 1; w < kLossWaves; ++w) v += sums[w][e >> 1][e & 1];
      out[e] = v;
      out[g.E + e] = __int_as_float(counts[e]);
    }
    if (threadIdx.x == 0) {
      float v = zsum[0];
      int m = tokens[0];
      for (int w = 1; w < kLossWaves; ++w) {
        v += zsum[w];
        m += tokens[w];
      }
      out[2 * g.E] = v;
      out[2 * g.E + 1] = __int_as_float(m);
    }
    __syncthreads();
  }
}

// The rows of `part` of sequence s: [first, first + rows).
__device__ __forceinline__ void loss_rows(const RouterLossArgs& g, int s, int64_t& first, int& rows) {
  const int lo = seq_at(g, s), hi = seq_at(g, s + 1), B = g.tokens_of_block;
  first = lo / B + s;
  rows = hi > lo ? (hi - 1) / B - lo / B + 1 : 0;
}

// 32 columns of a sequence: probs and counts.
__global__ void __launch_bounds__(256) router_loss_columns_kernel(RouterLossArgs g) {
  __shared__ float sums[8][32];
  __shared__ int32_t counts[8][32];
  const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
  const int64_t W = loss_row(g.E);
  for (int s = blockIdx.y; s < g.S; s += gridDim.y) {
    int64_t first;
    int rows;
    loss_rows(g, s, first, rows);
    const float* const p = g.part + first * W;
    float v = 0.f;
    int n = 0;
    if (e < g.E) {
      v = column_sum(p + e, W, r0, rows);
      for (int r = r0; r < rows; r += 8) n += __float_as_int(p[r * W + g.E + e]);
    }
    sums[r0][c] = v;
    counts[r0][c] = n;
    __syncthreads();
    if (r0 == 0 && e < g.E) {
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        v += sums[i][c];
        n += counts[i][c];
      }
      g.probs[(int64_t)s * g.E + e] = v;
      g.counts[(int64_t)s * g.E + e] = n;
    }
    __syncthreads();
  }
}

// The losses of a sequence, a wave each: E products and the pieces' sums of lse^2.
__global__ void __launch_bounds__(64) router_loss_finish_kernel(RouterLossArgs g) {
  const int lane = threadIdx.x;
  const int64_t W = loss_row(g.E);
  for (int s = blockIdx.x; s < g.S; s += gridDim.x) {
    int64_t first;
    int rows;
    loss_rows(g, s, first, rows);
    double dot = 0., zz = 0.;
    int n = 0;
    for (int e = lane; e < g.E; e += 64)
      dot += (double)g.counts[(int64_t)s * g.E + e] * g.probs[(int64_t)s * g.E + e];
    for (int r = lane; r < rows; r += 64) {
      const float* const p = g.part + (first + r) * W + 2 * g.E;
      zz += p[0];
      n += __float_as_int(p[1]);
    }
    dot = wave_sum_f64(dot);
    zz = wave_sum_f64(zz);
#pragma unroll
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d, 64);
    if (lane == 0) {
      const double m = n > 0 ? n : 1;
      g.tokens[s] = n;
      g.balance[s] = (float)(dot * g.E / (g.k * m * m));
      g.z[s] = (float)(zz / m);
    }
  }
}

template <typename TO>
__device__ __forceinline__ void store_pair(void* p, int64_t at, int j, int E, f32x2 v, bool accumulate) {
  if (j >= E) return;
  const bool two = j + 1 < E;
  if constexpr (TO::kType == kF32) {
    float* const q = static_cast<float*>(p) + at + j;
    if (two) {
      if (accumulate) v += *reinterpret_cast<const f32x2_word*>(q);
      *reinterpret_cast<f32x2_word*>(q) = v;
    } else {
      *q = accumulate ? v[0] + *q : v[0];
    }
  } else {
    uint16_t* const q = static_cast<uint16_t*>(p) + at + j;
    if (two) {
      if (accumulate) {
        const uint32_t h = *reinterpret_cast<const u32_half*>(q);
        v += f32x2{TO::to_f32((uint16_t)h), TO::to_f32((uint16_t)(h >> 16))};
      }
      *reinterpret_cast<u32_half*>(q) = (uint32_t)TO::from_f32(v[0]) | ((uint32_t)TO::from_f32(v[1]) << 16);
    } else {
      *q = TO::from_f32(accumulate ? v[0] + TO::to_f32(*q) : v[0]);
    }
  }
}

constexpr int kBackWaves = 4;

// A wave takes neighbouring tokens: its sequence's coefficients change rarely.
template <typename T, typename TO, int NC>
__global__ void __launch_bounds__(kBackWaves * 64) router_loss_backward_kernel(RouterLossArgs g, int per_wave) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t w0 = ((int64_t)blockIdx.x * kBackWaves + wave) * per_wave;
  if (w0 >= g.T) return;
  const int t0 = (int)w0, t1 = g.T - t0 < per_wave ? g.T : t0 + per_wave;
  int lo = 0, hi = 0;  // the tokens that the coefficients are of
  f32x2 coef[NC] = {};
  float zc = 0.f;
  for (int t = t0; t < t1; ++t) {
    if (t < lo || t >= hi) {
      const int s = seq_of(g, t);
      if (s >= g.S) return;  // behind the last sequence
      lo = seq_at(g, s);
      hi = seq_at(g, s + 1);
      if (t >= lo) {
        const int n = g.tokens_in ? g.tokens_in[s] : 1;
        const double m = n > 0 ? n : 1;
        const float f = g.dbalance ? (float)(g.dbalance[s] * ((double)g.E / (g.k * m * m))) : 0.f;
        zc = g.dz ? (float)(2. * g.dz[s] / m) : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int e = c * 128 + lane * 2 + i;
            coef[c][i] = g.dbalance && e < g.E ? f * (float)g.counts_in[(int64_t)s * g.E + e] : 0.f;
          }
      }
    }
    if (t < lo) continue;  // before the first sequence
    const bool live = !g.mask || g.mask[t];
    if (!live) {
      if (!g.accumulate)
#pragma unroll
        for (int c = 0; c < NC; ++c) store_pair<TO>(g.dlogits, t * g.ldd, c * 128 + lane * 2, g.E, f32x2{}, false);
      continue;
    }
    f32x2 d[NC] = {};
    if (g.dbalance || g.dz) {
      f32x2 l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = load_pair<T>(g.logits, t * g.ld, c * 128 + lane * 2, g.E);
      Scores<NC> o;
      scores<NC>(l, g.score == kScoreSigmoid, o);
      float along = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          o.p[c][i] *= o.inv;
          along += o.p[c][i] * coef[c][i];
        }
      along = wave_sum_f32(along);
      const float zt = zc * o.lse * o.soft_inv;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          d[c][i] = o.p[c][i] * (coef[c][i] - along) * o.down[c][i] + zt * o.soft[c][i];
    }
    if (g.gates) {
      const bool mine = lane < g.k;
      const int64_t at = (int64_t)t * g.k + (mine ? lane : 0);
      const int id = g.idx[at];
      const float gate = mine ? g.gates[at] : 0.f, dg = mine ? g.dgates[at] : 0.f;
      const float v = gate * (dg - wave_sum_f32(gate * dg));
      for (int j = 0; j < g.k; ++j) {
        const int e = __builtin_amdgcn_readlane(id, j);
        const float add = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (e == c * 128 + lane * 2 + i) d[c][i] += add;
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) store_pair<TO>(g.dlogits, t * g.ldd, c * 128 + lane * 2, g.E, d[c], g.accumulate);
  }
}

int block_tokens(int T) {
  const int b = (T + kLossBlocks - 1) / kLossBlocks;
  return b < kLossWaves ? kLossWaves : b;
}

template <typename F>
void by_columns(int E, const F& run) {
  if (E <= 128) run(IntC<1>{});
  else if (E <= 256) run(IntC<2>{});
  else if (E <= 384) run(IntC<3>{});
  else if (E <= 512) run(IntC<4>{});
  else if (E <= 768) run(IntC<6>{});
  else run(IntC<8>{});
}

}  // namespace

size_t router_loss_workspace(const RouterLossArgs& a) {
  const int B = block_tokens(a.T);
  return ((size_t)(a.T + B - 1) / B + a.S) * loss_row(a.E) * 4;
}

hipError_t launch_router_loss(RouterLossArgs a, hipStream_t stream) {
  a.tokens_of_block = block_tokens(a.T);
  const unsigned blocks = (a.T + a.tokens_of_block - 1) / a.tokens_of_block;
  if (blocks)
    by_columns(a.E, [&](auto nc) {
      constexpr int NC = decltype(nc)::value;
      const auto run = [&](auto k) { hipLaunchKernelGGL(k, dim3(blocks), dim3(kLossWaves * 64), 0, stream, a); };
      if (a.type == kF32) run(router_loss_kernel<F32, NC>);
      else if (a.type == kBf16) run(router_loss_kernel<Bf16, NC>);
      else run(router_loss_kernel<F16, NC>);
    });
  const unsigned most = a.S < 4096 ? a.S : 4096;
  hipLaunchKernelGGL(router_loss_columns_kernel, dim3((a.E + 31) / 32, most), dim3(256), 0, stream, a);
  hipLaunchKernelGGL(router_loss_finish_kernel, dim3(most), dim3(64), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_router_loss_backward(RouterLossArgs a, hipStream_t stream) {
  if (!a.T) return hipSuccess;
  int per_wave = (a.T + 8191) / 8192;  // eight waves a SIMD
  const unsigned blocks = (unsigned)(((int64_t)a.T + kBackWaves * per_wave - 1) / (kBackWaves * per_wave));
  by_columns(a.E, [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    const auto run = [&](auto k) { hipLaunchKernelGGL(k, dim3(blocks), dim3(kBackWaves * 64), 0, stream, a, per_wave); };
    if (a.type == kF32)
      a.out_type == kF32 ? run(router_loss_backward_kernel<F32, F32, NC>)
                         : a.out_type == kBf16 ? run(router_loss_backward_kernel<F32, Bf16, NC>)
                                               : run(router_loss_backward_kernel<F32, F16, NC>);
    else if (a.type == kBf16)
      a.out_type == kF32 ? run(router_loss_backward_kernel<Bf16, F32, NC>) : run(router_loss_backward_kernel<Bf16, Bf16, NC>);
    else
      a.out_type == kF32 ? run(router_loss_backward_kernel<F16, F32, NC>) : run(router_loss_backward_kernel<F16, F16, NC>);
  });
  return hipGetLastError();
}

}  // namespace moe_fp4
