// Internal launch interface of the operators around the routed experts: 16-bit
// products (grouped by expert, and dense with an epilogue) and the norms.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe_fp4 {

// Element types, activations and norm kinds: the values of the public header.
enum { kF32 = 0, kBf16 = 1, kF16 = 2 };
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr int kMaxWidth = 65536;         // N and K of a product
constexpr int kMaxProductRows = 1 << 20;  // rows of a product (65535 tokens x 16 experts fit)

// One product C[i][j] = sum_k A(i, k) B(j, k) per expert.  Three forms:
//   forward  i = row (ragged by expert), j = output, k = input:   A = x, B = w
//   dgrad    i = row (ragged by expert), j = input,  k = output:  A = dy, B = w
//   wgrad    i = output, j = input, k = row (ragged by expert):   A = dy, B = x
// so an operand is either contiguous along k (x, dy, w of forward) or along its
// own index (w of dgrad; dy and x of wgrad).  A dense product is one expert
// with no offsets.
enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

struct ProductArgs {
  int E, P;                // experts; rows of the ragged side
  const int32_t* offsets;  // [E+1] first row of each expert, null: one expert with P rows
  const int32_t* rows;     // [P] or null: row s of x is x[rows[s] / row_div] (a zero row outside [0, R))
  int row_div, R;
  int I, J, K;             // forward P, N, K; dgrad P, K, N; wgrad N, K, P
  const uint16_t *a, *b;
  int64_t lda, ldb;
  int64_t w_stride;        // elements between experts' weights (b of forward and dgrad)
  int type;                // kBf16 or kF16: a and b
  // result: c[i][j] (type c_type), wgrad: expert e's at c + e * c_stride
  void* c;
  int64_t ldc, c_stride;
  int c_type, accumulate;
  // epilogue (dense forward): z = sum + bias; c = act(z) + residual
  const void* bias;
  int bias_type, act;
  const void* residual;    // of c_type
  int64_t ldr;
  void* z;                 // of `type`, or null
  int64_t ldz;
  // split of the sum over `splits` workgroups: partial sums in part, [splits] of
  // [I][J] (wgrad [E][I][J]); 1: none
  int splits;
  float* part;
  const float* factor;  // of the sums, on the device, or null (1)
  int plain;  // set by launch_product: the epilogue only multiplies by the factor, rounds and stores, 16 bytes at a time
};

size_t product_workspace(const ProductArgs& a, int op);  // bytes of `part`
hipError_t launch_product(ProductArgs a, int op, void* ws, hipStream_t stream);
// The tile shapes of the products through LDS.  kAny takes rows of any length and
// alignment, the others 16-byte aligned rows whose length is a multiple of 8.
enum { kBig, kMid, kLow, kAny };
// The kernels that launch_product takes.
struct ProductChoice {
  int rows;    // a tile of the streaming kernel (1, 2, 4) or the few-row kernel (16); 0: tiles through LDS
  int shape, splits;            // of the columns up to `cut`
  int cut;
  int rest_shape, rest_splits;  // of the others
};
ProductChoice product_choice(const ProductArgs& a, int op);
void launch_product_fwd(const ProductArgs& a, int shape, hipStream_t stream);
void launch_product_dgrad(const ProductArgs& a, int shape, hipStream_t stream);
void launch_product_wgrad(const ProductArgs& a, int shape, hipStream_t stream);
// Forward for up to m = 1, 2 or 4 rows a tile, and dense for up to 16.
void launch_product_row(const ProductArgs& a, int m, hipStream_t stream);
void launch_product_few(const ProductArgs& a, hipStream_t stream);
// The most row tiles of BM rows that the experts can have.
inline int64_t row_tiles_most(const ProductArgs& a, int BM) {
  if (!a.offsets) return (a.P + BM - 1) / BM;
  const int64_t live = a.E < a.P ? a.E : a.P;  // experts that can have rows
  return (a.P + live * (BM - 1)) / BM;
}

// dz = dy act'(z) in `type`, and the column sums of dz before that rounding.  In
// fp16, dz is multiplied by a power of two 2^s first, which the products of dz take
// back by their factor 2^-s.
constexpr int kSlopeTops = 1024;
struct SlopeArgs {
  int M, N, type, dy_type, act;
  const void* dy;
  int64_t lddy;
  const uint16_t* z;   // null with kActNone
  int64_t ldz;
  uint16_t* dz;        // [M][N] dense, or null (column sums only)
  float* db;           // [N] or null
  int accumulate;      // db +=
  float* part;         // [slope_blocks(M)][N], with db
  float* top;          // [kSlopeTops], with dz in fp16: parts of the largest |dz|
  int tops;            // set by launch_slope: how many parts
  float* factor;       // with dz in fp16: written, 2^-s
};
int slope_blocks(int M);
hipError_t launch_slope(SlopeArgs a, hipStream_t stream);

struct NormArgs {
  int T, H;
  int64_t ldx, ldy, lddx;
  int x_type, y_type, w_type, rms;
  float eps;
  const void *x, *gamma, *beta;
  void* y;
  float *mean, *rstd;      // forward: written where not null
  // backward: dy of y_type with row stride ldy
  const void* dy;
  const float *mean_in, *rstd_in;
  void* dx;
  float *dgamma, *dbeta;
  int accumulate;          // dgamma +=, dbeta +=
  float* part;             // [norm_blocks][2][H]
};
int norm_blocks(const NormArgs& a);  // workgroups of the backward pass
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream);

}  // namespace moe_fp4
