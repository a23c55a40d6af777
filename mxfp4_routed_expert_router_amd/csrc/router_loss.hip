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
// Both passes read the logits once.  L lanes (32 from 129 to 512 experts) take a token, 64 / L
// tokens a wave: a row's maximum and sums are then a few exchanges between neighbouring
// lanes for several tokens at once (with a wave a token the longest backward pass took
// 76 us, 34 now; with 16 lanes 51, for its registers).  A lane keeps the same columns for every token: the sums
// over tokens stay in registers, and so do the coefficients c of the backward pass.
//
// Sums over tokens are held in fp32, the products' sum and that of the pieces' lse^2 in fp64.  An fp32
// sum's additions are a tree (a lane's T L / 2^17 tokens, 64 / L groups, eight waves, 16 rows of
// pieces, 16 of those), so that errors grow slowly: of 16384 tokens and of 2^20 alike, 384
// experts, probs are off by 3.9 * 2^-24 at most and 0.9 on average, balance by 1, z by 2.  N sums of
// 64 bits in a lane would cost waves.
//
// One MI355X: forward, 16384 tokens of 384 experts in fp32, 25 MB, 11.2 us and 8.9 for the
// columns (both chains of loads that wait for one another: offsets, rows, pieces), with sigmoids
// the same, bf16 0.5-1.5 less; 64 sequences in place of 8 53 in all, for a workgroup takes its pieces one
// after the other; 64 tokens 5.5 us.  Backward 14.1 us (50 MB, 3.6 TB/s); 65536 tokens, sigmoid, bf16, 34 us for 101 MB, of which
// the vector units are busy 59 %: about 25 instructions an element.
#include "block_device.h"
#include "router_loss.h"

namespace moe_fp4 {
namespace {

constexpr int kLossWaves = 8, kLossThreads = kLossWaves * 64;
constexpr int kLossBlocks = 256;  // most workgroups of the forward pass
constexpr int kAloneTokens = 128, kAloneSequences = 8;  // what one workgroup finishes alone

// A row of partial results: the sums of p, the counts, z's sum, the tokens.
__host__ __device__ inline int64_t loss_row(int E) { return 2 * (int64_t)E + 2; }

// Sequence s is tokens [lo, hi).  The offsets are device data that the host has not
// seen: they are held to [0, T], so that no value makes an access leave an array.
__device__ __forceinline__ int seq_at(const RouterLossArgs& g, int s) {
  if (!g.seqs) return s ? g.T : 0;
  const int v = g.seqs[s];
  return v < 0 ? 0 : v > g.T ? g.T : v;
}
// The first sequence that ends past token t (S where none does), found by L lanes that
// agree on t: L places at a time.  l: the lane among them.
template <int L>
__device__ __forceinline__ int seq_of(const RouterLossArgs& g, int t, int l) {
  if (!g.seqs) return t < g.T ? 0 : 1;
  int lo = 0, hi = g.S;
  while (lo < hi) {
    const int step = (hi - lo + L - 1) / L, s = lo + l * step;
    const uint64_t before = __ballot(s < hi && seq_at(g, s + 1 <= g.S ? s + 1 : g.S) <= t) >> ((threadIdx.x & 63) - l);
    const int c = __popcll(L == 64 ? before : before & ((1ull << (L & 63)) - 1));
    if (c == 0) return lo;
    const int end = lo + c * step;
    lo += (c - 1) * step + 1;
    hi = end < hi ? end : hi;
  }
  return lo;
}

// ---- a token's logits: lane `l` of its L lanes holds columns 4 (c L + l) + r, r < 4, as
// element 4 c + r of N
template <int L>
__device__ __forceinline__ int column_of(int l, int i) {
  return (i / 4 * L + l) * 4 + i % 4;
}

// A row as loaded: what waits for the load is values().  -inf past the last column.
template <typename T, int L, int N>
struct Row {
  static constexpr int kWords = T::kType == kF32 ? 4 : 2;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  Words raw[N / 4];

  __device__ __forceinline__ void load(const void* p, int64_t row, int l, int E) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int j = (c * L + l) * 4;
      if (E == L * N) {  // every lane's are there
        if constexpr (T::kType == kF32)
          raw[c] = __builtin_bit_cast(Words, *reinterpret_cast<const f32x4_word*>(static_cast<const float*>(p) + row + j));
        else
          raw[c] = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(p) + row + j);
      } else if constexpr (T::kType == kF32) {
        const float* const q = static_cast<const float*>(p) + row + j;
        if (j + 4 <= E) {
          raw[c] = __builtin_bit_cast(Words, *reinterpret_cast<const f32x4_word*>(q));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[c][i] = __float_as_uint(j + i < E ? q[i] : -INFINITY);
        }
      } else {
        constexpr uint32_t none = T::kType == kBf16 ? 0xFF80u : 0xFC00u;  // -inf
        const uint16_t* const q = static_cast<const uint16_t*>(p) + row + j;
        if (j + 4 <= E) {
          raw[c] = *reinterpret_cast<const u32x2_any*>(q);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            raw[c][i] = (j + 2 * i < E ? q[2 * i] : none) | (j + 2 * i + 1 < E ? q[2 * i + 1] : none) << 16;
        }
      }
    }
  }
  // What was made of the row is made anew behind this.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) asm volatile("" : "+v"(raw[c]));
  }
  __device__ __forceinline__ void values(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (T::kType == kF32) v[i] = __uint_as_float(raw[i / 4][i % 4]);
      else v[i] = T::to_f32((uint16_t)(raw[i / 4][i % 4 / 2] >> (16 * (i & 1))));
    }
  }
};

template <typename TO, int L, int N>
__device__ __forceinline__ void store_row(void* p, int64_t row, int l, int E, const float (&d)[N], bool accumulate) {
#pragma unroll
  for (int c = 0; c < N / 4; ++c) {
    const int j = (c * L + l) * 4, n = E == L * N || E - j >= 4 ? 4 : E - j;
    f32x4 v = {d[c * 4], d[c * 4 + 1], d[c * 4 + 2], d[c * 4 + 3]};
    if (E == L * N && !accumulate) {
      store4_from_f32(p, row + j, 4, TO::kType, true, v);
      continue;
    }
    if (n <= 0) continue;
    if (accumulate) v += load4_as_f32(p, row + j, n, TO::kType, n == 4);
    store4_from_f32(p, row + j, n, TO::kType, n == 4, v);
  }
}

// ---- over the L lanes of a token, the result in each of them
__device__ __forceinline__ float swap16(float v, bool high) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(high ? r[1] : r[0]);
}
__device__ __forceinline__ float swap32(float v, bool high) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(high ? r[1] : r[0]);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));   // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp_f32<0x4E>(v));   // quad_perm [2,3,0,1]
  v = fmaxf(v, dpp_f32<0x124>(v));  // row_ror:4
  v = fmaxf(v, dpp_f32<0x128>(v));  // row_ror:8
  if constexpr (L >= 32) v = fmaxf(swap16(v, false), swap16(v, true));
  if constexpr (L >= 64) v = fmaxf(swap32(v, false), swap32(v, true));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x124>(v);
  v += dpp_f32<0x128>(v);
  if constexpr (L >= 32) v = swap16(v, false) + swap16(v, true);
  if constexpr (L >= 64) v = swap32(v, false) + swap32(v, true);
  return v;
}

// A token's scores, p times a common factor.  Exponents are taken to base 2: with M = m log2 e
// rounded once, e = 2^(l log2 e - M) is one multiply-add and one instruction, and M's rounding is in
// all of a row's alike: a factor within 2^(1/16) up to |m| = 1e6, but past fp32's range from 1e10 on.
// Rows further out take e = exp(l - m), whose difference is exact wherever e is not 0.
//
// Softmax: e = exp(l - m), m the row's largest logit; p = e.
// Sigmoids: m = min(largest, 0), down = 1 / (1 + e 2^M) and p = e down: p is sigmoid(l) e^-m, which
// keeps its digits where all logits are far below 0, and down is 1 - sigmoid(l), from one exponential
// and one reciprocal.  Rows with a logit past 24 (`far`, there the sigmoid is 1 in fp32) take e of
// min(l, 24) for it, and 1 - sigmoid and the softmax of the z loss from exponentials of their own:
// the backward pass multiplies by down twice before it does by e, and down^2 = e^-48 times a
// coefficient is still a normal number (from e^-80 on it was 0).
//
// A row of -inf alone has no probabilities: its sums are 0, and so are their reciprocals and
// its lse.
constexpr float kFar = 24.f;
template <int N, bool Sigmoid>
struct Scores {
  float e[N], down[Sigmoid ? N : 1];
  float inv, soft_inv, lse, top;
  bool far;

  template <int L>
  __device__ __forceinline__ void of(const float (&l)[N]) {
    top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = lanes_max<L>(top);
    float m = top == -INFINITY ? 0.f : Sigmoid ? fminf(top, 0.f) : top, soft_sum = 0.f, sum = 0.f;
    const float M = m * kLog2e;
    far = Sigmoid && !(top <= kFar);  // NaN too
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = __builtin_amdgcn_exp2f(l[i] * kLog2e - M);
    if (!(fabsf(m) <= 1e6f)) {  // inf too
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = exp_f32(l[i] - m);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) soft_sum += e[i];
    if constexpr (Sigmoid) {
      if (far) {
        soft_sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          soft_sum += exp_f32(l[i] - top);
          if (l[i] > kFar) e[i] = __builtin_amdgcn_exp2f(kFar * kLog2e);
        }
      }
      const float f = __builtin_amdgcn_exp2f(M);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        down[i] = __builtin_amdgcn_rcpf(1.0f + e[i] * f);
        sum += e[i] * down[i];
      }
      sum = lanes_sum<L>(sum);
      if (far) m = top;
    }
    soft_sum = lanes_sum<L>(soft_sum);
    soft_inv = soft_sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(soft_sum);
    lse = soft_sum == 0.f ? 0.f : m + __builtin_amdgcn_logf(soft_sum) * 0.6931471805599453f;
    inv = !Sigmoid ? soft_inv : sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum);
  }
  __device__ __forceinline__ float p(int i) const {
    if constexpr (Sigmoid) return e[i] * down[i];
    else return e[i];
  }
};

// What a workgroup has of a piece of a sequence goes to a row of `part`, or is finished.
__device__ __forceinline__ void finish_loss(const RouterLossArgs& g, int s, double dot, double zz, int n) {
  const double m = n > 0 ? n : 1;
  g.tokens[s] = n;
  g.balance[s] = (float)(dot * g.E / (g.k * m * m));
  g.z[s] = (float)(zz / m);
}

// Workgroup b takes the tokens [b B, (b + 1) B), B = tokens_of_block, one piece for
// each sequence among them.  Piece (b, s) writes row b + s of `part`: along the
// pieces b or s grows, so that no two share a row.  One workgroup alone takes every
// sequence, also those without tokens, and writes the results.
template <typename T, int L, int N, bool Sigmoid>
__global__ void __launch_bounds__(kLossThreads) router_loss_kernel(RouterLossArgs g, bool alone) {
  constexpr int kTokens = 64 / L;  // of a wave at a time
  __shared__ float sums[kLossWaves][L * N];  // element i of lane l at i L + l
  __shared__ int32_t counts[L * N];
  __shared__ float zsum[kLossWaves];
  __shared__ int32_t tokens[kLossWaves];
  __shared__ double dots[kLossWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane % L, group = lane / L;
  const int t0 = blockIdx.x * g.tokens_of_block;
  const int t1 = g.T - t0 < g.tokens_of_block ? g.T : t0 + g.tokens_of_block;
  if (blockIdx.x == 0 && !alone)
    for (int s = threadIdx.x; s < g.S; s += kLossThreads) g.tickets[s] = 0;
  for (int s = alone ? 0 : seq_of<64>(g, t0, lane), next; s < g.S; s = next) {
    int lo = seq_at(g, s), hi = seq_at(g, s + 1);
    if (!alone && lo >= t1) break;
    lo = lo < t0 ? t0 : lo;
    hi = hi > t1 ? t1 : hi;
    next = s + 1;
    if (hi <= lo) {
      if (!alone) {  // past the empty ones
        const int after = seq_of<64>(g, lo, lane);
        next = after > next ? after : next;
        continue;
      }
      hi = lo;
    }
    // a token a turn for each group of lanes, the next one's logits on their way
    constexpr int kTurn = kLossWaves * kTokens;
    const auto load = [&](int t, Row<T, L, N>& r, bool& live) {
      live = t < hi;
      const int at = live ? t : lo;
      if (hi > lo) r.load(g.logits, at * g.ld, l, g.E);
      if (g.mask && live) live = g.mask[at];
    };
    Row<T, L, N> row[2];
    bool live[2];
    const int pairs = (hi - lo) * g.k;
    const auto choice = [&](int p) {  // the expert of a choice, -1 where it does not count
      if (p >= pairs || (g.mask && !g.mask[lo + p / g.k])) return -1;
      const int e = g.idx[(int64_t)lo * g.k + p];
      return e < g.E ? e : -1;
    };
    load(lo + wave * kTokens + group, row[0], live[0]);
    for (int e = threadIdx.x; e < L * N; e += kLossThreads) counts[e] = 0;
    lds_barrier();
    for (int p = threadIdx.x; p < pairs; p += kLossThreads) {
      const int e = choice(p);
      if (e >= 0) atomicAdd(&counts[e], 1);
    }
    float acc[N] = {}, zz = 0.f;
    int n = 0;
    for (int t = lo + wave * kTokens + group; t - group < hi; t += 2 * kTurn)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        load(t + (a + 1) * kTurn, row[1 - a], live[1 - a]);
        if (!live[a]) continue;
        float v[N];
        row[a].values(v);
        Scores<N, Sigmoid> o;
        o.template of<L>(v);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += o.p(i) * o.inv;
        zz += o.lse * o.lse;
        ++n;
      }
    // the wave's tokens of each turn
    if constexpr (L < 32) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = swap16(acc[i], false) + swap16(acc[i], true);
      zz = swap16(zz, false) + swap16(zz, true);
      n += __shfl_xor(n, 16, 64);
    }
    if constexpr (L < 64) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = swap32(acc[i], false) + swap32(acc[i], true);
      zz = swap32(zz, false) + swap32(zz, true);
      n += __shfl_xor(n, 32, 64);
    }
    if (group == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sums[wave][i * L + l] = acc[i];
    if (lane == 0) {
      zsum[wave] = zz;
      tokens[wave] = n;
    }
    __syncthreads();
    float* const out = alone ? g.probs + (int64_t)s * g.E : g.part + (int64_t)(blockIdx.x + s) * loss_row(g.E);
    int32_t* const out_counts = alone ? g.counts + (int64_t)s * g.E : reinterpret_cast<int32_t*>(out) + g.E;
    double dot = 0.;
    for (int o = threadIdx.x; o < L * N; o += kLossThreads) {
      const int e = column_of<L>(o % L, o / L);
      if (e >= g.E) continue;
      float v = sums[0][o];
#pragma unroll
      for (int w = 1; w < kLossWaves; ++w) v += sums[w][o];
      out[e] = v;
      out_counts[e] = counts[e];
      dot += (double)counts[e] * v;
    }
    if (alone) {
      dot = wave_sum_f64(dot);
      if (lane == 0) dots[wave] = dot;
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      float v = zsum[0];
      int m = tokens[0];
      for (int w = 1; w < kLossWaves; ++w) {
        v += zsum[w];
        m += tokens[w];
      }
      if (alone) {
        for (int w = 1; w < kLossWaves; ++w) dot += dots[w];
        finish_loss(g, s, dot, v, m);
      } else {
        out[2 * g.E] = v;
        reinterpret_cast<int32_t*>(out)[2 * g.E + 1] = m;
      }
    }
    __syncthreads();
  }
}

// 32 columns of a sequence: probs and counts, and their products' sum.  The last
// workgroup of a sequence adds these up, in the columns' order, and the pieces' sums of
// lse^2: the same bits whichever comes last.
constexpr int kColumnRows = 16;
__global__ void __launch_bounds__(32 * kColumnRows) router_loss_columns_kernel(RouterLossArgs g) {
  __shared__ float sums[kColumnRows][32];
  __shared__ int32_t counts[kColumnRows][32];
  __shared__ bool last;
  const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5, e = blockIdx.x * 32 + c, lane = threadIdx.x & 63;
  const int64_t W = loss_row(g.E);
  for (int s = blockIdx.y; s < g.S; s += gridDim.y) {
    const int lo = seq_at(g, s), hi = seq_at(g, s + 1), B = g.tokens_of_block;
    const int rows = hi > lo ? (hi - 1) / B - lo / B + 1 : 0;
    const float* const p = g.part + (lo / B + (int64_t)s) * W;
    float v = 0.f;
    int n = 0;
    if (e < g.E)
      for (int r = r0; r < rows; r += 4 * kColumnRows) {  // four rows in flight
        float a[4];
        int b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = r + u * kColumnRows < rows ? r + u * kColumnRows : r;
          a[u] = p[at * W + e];
          b[u] = __float_as_int(p[at * W + g.E + e]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r + u * kColumnRows < rows) {
            v += a[u];
            n += b[u];
          }
      }
    sums[r0][c] = v;
    counts[r0][c] = n;
    __syncthreads();
    if (threadIdx.x < 64) {
      double dot = 0.;
      if (r0 == 0 && e < g.E) {
#pragma unroll
        for (int i = 1; i < kColumnRows; ++i) {
          v += sums[i][c];
          n += counts[i][c];
        }
        g.probs[(int64_t)s * g.E + e] = v;
        g.counts[(int64_t)s * g.E + e] = n;
        dot = (double)n * v;
      }
      dot = wave_sum_f64(dot);
      if (lane == 0) {
        g.dots[(int64_t)s * gridDim.x + blockIdx.x] = dot;
        __threadfence();
        last = __hip_atomic_fetch_add(&g.tickets[s], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        __threadfence();
      }
    }
    __syncthreads();
    if (last && threadIdx.x < 64) {
      double dot = 0., zz = 0.;
      int m = 0;
      if (lane < (int)gridDim.x)  // E / 32 <= 32 of them
        dot = __hip_atomic_load(&g.dots[(int64_t)s * gridDim.x + lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      for (int r = lane; r < rows; r += 64) {
        zz += p[r * W + 2 * g.E];
        m += __float_as_int(p[r * W + 2 * g.E + 1]);
      }
      dot = wave_sum_f64(dot);
      zz = wave_sum_f64(zz);
#pragma unroll
      for (int d = 32; d; d >>= 1) m += __shfl_xor(m, d, 64);
      if (lane == 0) finish_loss(g, s, dot, zz, m);
    }
    __syncthreads();
  }
}

constexpr int kBackWaves = 4;  // of a workgroup
// Waves of a launch for each SIMD: as many as it holds of them at 384 experts.  (Of 65536
// tokens' bf16 logits with sigmoids, at 128 registers and four waves 34 us; 47 with one
// register more, and 43 where the compiler is told to keep to four, for the order it then takes.)
// Elsewhere the registers may hold one wave fewer, and some workgroups then start late: sigmoids of 513
// to 768 experts in 16 bits with results in them (130 registers), and sigmoids of fp32 logits from
// 385 to 512 and from 769 experts on (169 to 175).
template <typename T, int N, bool Sigmoid>
constexpr int kBackOfSimd = !Sigmoid || (T::kType != kF32 && N <= 12) ? 4 : 3;

// Four counts from column j on, zeros past the last.
__device__ __forceinline__ f32x4 load4_counts(const int32_t* p, int j, int E) {
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
  typedef i32x4 __attribute__((aligned(4))) i32x4_word;
  i32x4 c = {};
  if (j + 4 <= E) {
    c = *reinterpret_cast<const i32x4_word*>(p + j);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (j + r < E) c[r] = p[j + r];
  }
  return f32x4{(float)c[0], (float)c[1], (float)c[2], (float)c[3]};
}

// The L lanes of a token take neighbouring tokens one after the other: their sequence's
// coefficients change rarely.
template <typename T, typename TO, int L, int N, bool Sigmoid>
__global__ void __launch_bounds__(kBackWaves * 64) router_loss_backward_kernel(RouterLossArgs g, int per_group) {
  __shared__ float rows[kBackWaves * 64 / L][L * N];
  const int lane = threadIdx.x & 63, l = lane % L;
  float* const chosen = rows[threadIdx.x / L];  // of this token's lanes alone
  if (g.gates)
#pragma unroll
    for (int i = 0; i < N; ++i) chosen[i * L + l] = 0.f;
  __builtin_amdgcn_wave_barrier();
  const int64_t first = ((int64_t)blockIdx.x * (kBackWaves * 64) + threadIdx.x) / L * per_group;
  if (first >= g.T) return;
  const int t0 = (int)first, t1 = g.T - t0 < per_group ? g.T : t0 + per_group;
  int lo = 0, hi = 0;  // the tokens that the coefficients are of
  float coef[N], zc = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) coef[i] = 0.f;
  struct Token {
    Row<T, L, N> row;
    bool live;
    int id;
    float gate, dg;  // lane j of the token: choice j (k <= 16 <= L)
  };
  const auto load = [&](int t, Token& o) {
    if (g.dbalance || g.dz) o.row.load(g.logits, t * g.ld, l, g.E);
    o.live = !g.mask || g.mask[t];
    o.id = -1;
    o.gate = o.dg = 0.f;
    if (g.gates && l < g.k) {
      const int64_t at = (int64_t)t * g.k + l;
      o.id = g.idx[at];
      o.gate = g.gates[at];
      o.dg = g.dgates[at];
    }
  };
  const auto token = [&](int t, Token& in) {
    if (t < lo || t >= hi) {
      const int s = seq_of<L>(g, t, l);
      lo = s < g.S ? seq_at(g, s) : 0x7FFFFFFF;
      hi = s < g.S ? seq_at(g, s + 1) : 0x7FFFFFFF;
      if (t >= lo) {
        const int n = g.tokens_in ? g.tokens_in[s] : 1;
        const double m = n > 0 ? n : 1;
        const float f = g.dbalance ? (float)(g.dbalance[s] * ((double)g.E / (g.k * m * m))) : 0.f;
        zc = g.dz ? (float)(2. * g.dz[s] / m) : 0.f;
        if (g.dbalance) {
          const int32_t* const q = g.counts_in + (int64_t)s * g.E;
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            const f32x4 c = load4_counts(q, column_of<L>(l, i), g.E);
#pragma unroll
            for (int r = 0; r < 4; ++r) coef[i + r] = f * c[r];
          }
        }
      }
    }
    if (t < lo) {  // in no sequence; the next token may be the first of this one, whose coefficients it loads
      hi = lo;
      return;
    }
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = 0.f;
    if (!in.live) {
      if (!g.accumulate) store_row<TO, L>(g.dlogits, t * g.ldd, l, g.E, d, false);
      return;
    }
    if (g.dbalance || g.dz) {
      float v[N];
      in.row.values(v);
      Scores<N, Sigmoid> o;
      o.template of<L>(v);
      float along = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) along += o.p(i) * coef[i];
      along = lanes_sum<L>(along) * o.inv;
      const float zt = !Sigmoid || g.dz ? zc * o.lse * o.soft_inv : 0.f;  // lse of a logit of inf is NaN
      if (!o.far) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float t = (coef[i] - along) * o.inv;
          if constexpr (Sigmoid) d[i] = o.e[i] * (o.down[i] * (o.down[i] * t) + zt);
          else d[i] = o.e[i] * (t + zt);
        }
      } else if constexpr (Sigmoid) {  // rare: the logits are taken from the row again, not kept for it
        in.row.forget();
        in.row.values(v);
#pragma unroll
        for (int i = 0; i < N; ++i)
          d[i] = o.p(i) * o.inv * (coef[i] - along) * (v[i] > kFar ? exp_f32(-v[i]) : o.down[i]) +
                 zt * exp_f32(fminf(v[i] - o.top, 0.f));  // inf - inf counts for zt alone, which is NaN then
      }
    }
    if (g.gates) {
      // through a row of zeros in LDS; choices of the same expert all write their sum
      const float own = in.gate * (in.dg - lanes_sum<L>(in.gate * in.dg));
      float add = 0.f;
      for (int j = 0; j < g.k; ++j) {
        const int e = __shfl(in.id, j, L);
        const float v = __shfl(own, j, L);
        if (e == in.id) add += v;
      }
      const bool ok = in.id >= 0 && in.id < g.E;
      if (ok) chosen[in.id] = add;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const f32x4 c = *reinterpret_cast<const f32x4*>(chosen + column_of<L>(l, i));
#pragma unroll
        for (int r = 0; r < 4; ++r) d[i + r] += c[r];
      }
      __builtin_amdgcn_wave_barrier();
      if (ok) chosen[in.id] = 0.f;
    }
    store_row<TO, L>(g.dlogits, t * g.ldd, l, g.E, d, g.accumulate);
  };
  Token a, b;
  load(t0, a);
  for (int t = t0; t < t1; t += 2) {
    load(t + 1 < t1 ? t + 1 : t, b);
    token(t, a);
    if (t + 1 >= t1) break;
    load(t + 2 < t1 ? t + 2 : t, a);
    token(t + 1, b);
  }
}

int block_tokens(int T) {
  const int b = (T + kLossBlocks - 1) / kLossBlocks, turn = kLossWaves * 4;
  return b < turn ? turn : (b + turn - 1) / turn * turn;
}
bool loss_alone(const RouterLossArgs& a) { return a.T <= kAloneTokens && a.S <= kAloneSequences; }

// Lanes of a token and elements of a lane.
template <typename F>
void by_experts(int E, const F& run) {
  if (E <= 64) run(IntC<16>{}, IntC<4>{});
  else if (E <= 128) run(IntC<16>{}, IntC<8>{});
  else if (E <= 256) run(IntC<32>{}, IntC<8>{});
  else if (E <= 384) run(IntC<32>{}, IntC<12>{});
  else if (E <= 512) run(IntC<32>{}, IntC<16>{});
  else if (E <= 768) run(IntC<64>{}, IntC<12>{});
  else run(IntC<64>{}, IntC<16>{});
}

// The workspace: the pieces' rows, the columns' sums of products, the tickets.
struct LossWs {
  size_t dots, tickets, total;
};
LossWs loss_ws(const RouterLossArgs& a) {
  LossWs w{};
  if (loss_alone(a)) return w;
  const int B = block_tokens(a.T), blocks = (a.T + B - 1) / B;
  const size_t rows = ((size_t)blocks + a.S) * loss_row(a.E) * 4;
  w.dots = (rows + 255) / 256 * 256;
  w.tickets = w.dots + (size_t)a.S * ((a.E + 31) / 32) * 8;
  w.total = w.tickets + (size_t)a.S * 4;
  return w;
}

}  // namespace

size_t router_loss_workspace(const RouterLossArgs& a) { return loss_ws(a).total; }

hipError_t launch_router_loss(RouterLossArgs a, void* ws, hipStream_t stream) {
  const bool alone = loss_alone(a);
  a.tokens_of_block = alone ? kAloneTokens : block_tokens(a.T);
  const LossWs w = loss_ws(a);
  a.part = static_cast<float*>(ws);
  a.dots = reinterpret_cast<double*>(static_cast<char*>(ws) + w.dots);
  a.tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + w.tickets);
  const unsigned blocks = a.T > a.tokens_of_block ? (a.T + a.tokens_of_block - 1) / a.tokens_of_block : 1;
  by_experts(a.E, [&](auto lanes, auto elements) {
    constexpr int L = decltype(lanes)::value, N = decltype(elements)::value;
    const auto run = [&](auto k) { hipLaunchKernelGGL(k, dim3(blocks), dim3(kLossThreads), 0, stream, a, alone); };
    const auto scored = [&](auto t) {
      using T = decltype(t);
      a.score == kScoreSigmoid ? run(router_loss_kernel<T, L, N, true>) : run(router_loss_kernel<T, L, N, false>);
    };
    a.type == kF32 ? scored(F32{}) : a.type == kBf16 ? scored(Bf16{}) : scored(F16{});
  });
  if (!alone)
    hipLaunchKernelGGL(router_loss_columns_kernel, dim3((a.E + 31) / 32, a.S < 4096 ? a.S : 4096), dim3(32 * kColumnRows), 0,
                       stream, a);
  return hipGetLastError();
}

hipError_t launch_router_loss_backward(RouterLossArgs a, hipStream_t stream) {
  if (!a.T) return hipSuccess;
  by_experts(a.E, [&](auto lanes, auto elements) {
    constexpr int L = decltype(lanes)::value, N = decltype(elements)::value;
    const auto run = [&](auto k, int of_simd) {
      const int groups = of_simd * 4 * 256 * (64 / L), per = (a.T + groups - 1) / groups, tokens = kBackWaves * 64 / L * per;
      hipLaunchKernelGGL(k, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kBackWaves * 64), 0, stream, a, per);
    };
    const auto scored = [&](auto t, auto to) {
      using T = decltype(t);
      using TO = decltype(to);
      a.score == kScoreSigmoid ? run(router_loss_backward_kernel<T, TO, L, N, true>, kBackOfSimd<T, N, true>)
                               : run(router_loss_backward_kernel<T, TO, L, N, false>, kBackOfSimd<T, N, false>);
    };
    if (a.type == kF32) a.out_type == kF32 ? scored(F32{}, F32{}) : a.out_type == kBf16 ? scored(F32{}, Bf16{}) : scored(F32{}, F16{});
    else if (a.type == kBf16) a.out_type == kF32 ? scored(Bf16{}, F32{}) : scored(Bf16{}, Bf16{});
    else a.out_type == kF32 ? scored(F16{}, F32{}) : scored(F16{}, F16{});
  });
  return hipGetLastError();
}

}  // namespace moe_fp4
