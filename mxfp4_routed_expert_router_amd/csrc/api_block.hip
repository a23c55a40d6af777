// C-ABI of the operators around the routed experts: argument validation,
// workspace layout and launches.  Every check runs on the host before the
// first HIP call, so a rejected call enqueues nothing.
#include "../../include/moe_fp4.h"

#include <math.h>

#include "api_common.h"

using namespace moe_fp4;

namespace {

constexpr int kMaxGroupedExperts = 1024;
constexpr int kMaxNormWidth = 16384;

static_assert(MOE_FP4_F32 == kF32 && MOE_FP4_BF16 == kBf16 && MOE_FP4_F16 == kF16, "types");
static_assert(MOE_FP4_ACT_SILU == kActSilu && MOE_FP4_ACT_RELU == kActRelu &&
                  MOE_FP4_ACT_GELU == kActGelu && MOE_FP4_ACT_GELU_TANH == kActGeluTanh,
              "activations");
static_assert(MOE_FP4_TILES_128X128 - MOE_FP4_TILES_256X256 == kMid && MOE_FP4_TILES_64X128 - MOE_FP4_TILES_256X256 == kLow &&
                  MOE_FP4_TILES_ANY - MOE_FP4_TILES_256X256 == kAny && kBig == 0, "tiles");
static_assert(MOE_FP4_GROUPED_FORWARD == kFwd && MOE_FP4_GROUPED_DGRAD == kDgrad &&
                  MOE_FP4_GROUPED_WGRAD == kWgrad, "forms");

// ---- grouped products
int grouped_args(const moe_fp4_grouped_dims* dims, int op, bool gathered, ProductArgs& a) {
  if (!dims) return MOE_FP4_EINVAL;
  const moe_fp4_grouped_dims& d = *dims;
  if (d.E < 1 || d.P < 0 || d.N < 1 || d.K < 1) return MOE_FP4_EINVAL;
  if (gathered && (d.R < 0 || d.row_div < 1)) return MOE_FP4_EINVAL;
  if (d.E > kMaxGroupedExperts || d.P > kMaxProductRows || d.N > kMaxWidth || d.K > kMaxWidth ||
      (gathered && d.R > kMaxProductRows) || !is16(d.type) ||
      (d.out_type != d.type && d.out_type != kF32) || op < kFwd || op > kWgrad)
    return MOE_FP4_EUNSUPPORTED;
  int64_t ldx, ldw, ldy;
  if (!stride(d.ldx, d.K, ldx) || !stride(d.ldw, d.K, ldw) || !stride(d.ldy, d.N, ldy))
    return MOE_FP4_EINVAL;
  const int64_t es = d.expert_stride ? d.expert_stride : d.N * ldw;
  if (es < (d.N - 1) * ldw + d.K) return MOE_FP4_EINVAL;
  a = ProductArgs{};
  a.E = d.E;
  a.P = d.P;
  a.row_div = gathered ? d.row_div : 1;
  a.R = gathered ? d.R : d.P;
  a.type = d.type;
  a.c_type = d.out_type;
  a.act = kActNone;
  switch (op) {
    case kFwd:
      a.I = d.P; a.J = d.N; a.K = d.K;
      a.lda = ldx; a.ldb = ldw; a.ldc = ldy; a.w_stride = es;
      break;
    case kDgrad:
      a.I = d.P; a.J = d.K; a.K = d.N;
      a.lda = ldy; a.ldb = ldw; a.ldc = ldx; a.w_stride = es;
      break;
    default:
      a.I = d.N; a.J = d.K; a.K = d.P;
      a.lda = ldy; a.ldb = ldx; a.ldc = ldw; a.c_stride = es;
      break;
  }
  return MOE_FP4_OK;
}

const int32_t some_offsets[1] = {0};  // for sizes and plans: their presence only, a grouped product

int grouped(const moe_fp4_grouped_dims* dims, int op, const void* a, const void* b,
            const int32_t* offsets, const int32_t* rows, void* c, int flags, void* ws,
            size_t ws_bytes, hipStream_t stream) {
  if (!dims || !offsets) return MOE_FP4_EINVAL;
  ProductArgs p;
  const int rc = grouped_args(dims, op, rows != nullptr, p);
  if (rc != MOE_FP4_OK) return rc;
  if (flags & ~MOE_FP4_ACCUMULATE) return MOE_FP4_EUNSUPPORTED;
  // arrays without elements may be null: x of no rows, every row array of P = 0
  const int x_rows = rows ? dims->R : dims->P;
  const bool no_a = op == kFwd ? x_rows == 0 : dims->P == 0;
  const bool no_b = op == kWgrad && x_rows == 0;
  if ((!a && !no_a) || (!b && !no_b) || (!c && (op == kWgrad || dims->P > 0)))
    return MOE_FP4_EINVAL;
  if (!aligned(a, 2) || !aligned(b, 2) || !aligned(c, size_of(p.c_type)) || !aligned(offsets, 4) ||
      !aligned(rows, 4))
    return MOE_FP4_EALIGN;
  p.a = static_cast<const uint16_t*>(a);
  p.b = static_cast<const uint16_t*>(b);
  p.c = c;
  p.offsets = offsets;
  p.rows = rows;
  p.accumulate = (flags & MOE_FP4_ACCUMULATE) ? 1 : 0;
  const int wrc = workspace_check(ws, ws_bytes, product_workspace(p, op));
  if (wrc != MOE_FP4_OK) return wrc;
  return done(launch_product(p, op, ws, stream));
}

// ---- dense product
struct LinearStrides {
  int64_t x, w, y, r, z, dx, dw;
};
int linear_check(const moe_fp4_linear_dims* dims, bool backward, LinearStrides& s) {
  if (!dims) return MOE_FP4_EINVAL;
  const moe_fp4_linear_dims& d = *dims;
  if (d.M < 0 || d.N < 1 || d.K < 1) return MOE_FP4_EINVAL;
  if (d.M > kMaxProductRows || d.N > kMaxWidth || d.K > kMaxWidth || !is16(d.type) ||
      (d.out_type != d.type && d.out_type != kF32) || d.act < kActNone || d.act > kActSilu)
    return MOE_FP4_EUNSUPPORTED;
  if (backward ? d.dw_type != d.type && d.dw_type != kF32 : !type_ok(d.bias_type))
    return MOE_FP4_EUNSUPPORTED;
  if (!stride(d.ldx, d.K, s.x) || !stride(d.ldw, d.K, s.w) || !stride(d.ldy, d.N, s.y) ||
      !stride(d.ldr, d.N, s.r) || !stride(d.ldz, d.N, s.z) || !stride(d.lddx, d.K, s.dx) ||
      !stride(d.lddw, d.K, s.dw))
    return MOE_FP4_EINVAL;
  return MOE_FP4_OK;
}
ProductArgs linear_product(const moe_fp4_linear_dims& d) {
  ProductArgs a{};
  a.E = 1;
  a.P = d.M;
  a.R = d.M;
  a.row_div = 1;
  a.type = d.type;
  a.act = kActNone;
  return a;
}
ProductArgs linear_forward_args(const moe_fp4_linear_dims& d, const LinearStrides& s) {
  ProductArgs a = linear_product(d);
  a.I = d.M; a.J = d.N; a.K = d.K;
  a.lda = s.x; a.ldb = s.w; a.ldc = s.y; a.ldr = s.r; a.ldz = s.z;
  a.c_type = d.out_type;
  a.bias_type = d.bias_type;
  a.act = d.act;
  return a;
}
// dz is dy itself where nothing changes between them
bool dz_is_dy(const moe_fp4_linear_dims& d) { return d.act == kActNone && d.out_type == d.type; }
bool dz_has_factor(const moe_fp4_linear_dims& d) { return d.type == kF16 && !dz_is_dy(d); }
ProductArgs linear_dgrad_args(const moe_fp4_linear_dims& d, const LinearStrides& s) {
  ProductArgs a = linear_product(d);
  a.I = d.M; a.J = d.K; a.K = d.N;
  a.lda = dz_is_dy(d) ? s.y : d.N; a.ldb = s.w; a.ldc = s.dx;
  a.c_type = d.type;
  return a;
}
ProductArgs linear_wgrad_args(const moe_fp4_linear_dims& d, const LinearStrides& s) {
  ProductArgs a = linear_product(d);
  a.I = d.N; a.J = d.K; a.K = d.M;
  a.lda = dz_is_dy(d) ? s.y : d.N; a.ldb = s.x; a.ldc = s.dw;
  a.c_type = d.dw_type;
  return a;
}
// Workspace of the backward pass: dz, its power of two in fp16 and the parts that it is
// found from, the column sums' parts, the products' parts (the two run one after the
// other and share theirs).
struct BackwardWs {
  size_t dz, factor, top, part, product, total;
};
BackwardWs backward_layout(const moe_fp4_linear_dims& d, const LinearStrides& s) {
  BackwardWs w{};
  size_t o = 0;
  w.dz = o;
  if (!dz_is_dy(d)) o = align_up(o + (size_t)d.M * d.N * 2);
  w.factor = o;
  if (dz_has_factor(d)) o += kAlign;
  w.top = o;
  if (dz_has_factor(d)) o = align_up(o + kSlopeTops * 4);
  w.part = o;
  o = align_up(o + (size_t)slope_blocks(d.M) * d.N * 4);
  w.product = o;
  const size_t a = product_workspace(linear_dgrad_args(d, s), kDgrad);
  const size_t b = product_workspace(linear_wgrad_args(d, s), kWgrad);
  w.total = align_up(o + (a > b ? a : b));
  return w;
}

// ---- norms
int norm_args(const moe_fp4_norm_dims* dims, NormArgs& a) {
  if (!dims) return MOE_FP4_EINVAL;
  const moe_fp4_norm_dims& d = *dims;
  if (d.T < 0 || d.H < 1 || !(d.eps >= 0.f)) return MOE_FP4_EINVAL;
  if (d.T > kMaxProductRows || d.H > kMaxNormWidth || !type_ok(d.x_type) || !type_ok(d.y_type) ||
      !type_ok(d.w_type) || (d.y_type != d.x_type && d.x_type != kF32) ||
      (d.kind != MOE_FP4_NORM_LAYER && d.kind != MOE_FP4_NORM_RMS))
    return MOE_FP4_EUNSUPPORTED;
  a = NormArgs{};
  if (!stride(d.ldx, d.H, a.ldx) || !stride(d.ldy, d.H, a.ldy) || !stride(d.lddx, d.H, a.lddx))
    return MOE_FP4_EINVAL;
  a.T = d.T;
  a.H = d.H;
  a.x_type = d.x_type;
  a.y_type = d.y_type;
  a.w_type = d.w_type;
  a.rms = d.kind == MOE_FP4_NORM_RMS;
  a.eps = d.eps;
  return MOE_FP4_OK;
}
// The choice for pointers on 16-byte boundaries (the strides count).
int product_plan(const ProductArgs& a, int op, moe_fp4_product_plan* plan) {
  *plan = moe_fp4_product_plan{};
  if (op != kWgrad && a.P == 0) return MOE_FP4_OK;  // nothing runs
  const ProductChoice c = product_choice(a, op);
  plan->rows = c.rows;
  if (c.rows) return MOE_FP4_OK;
  plan->tiles = MOE_FP4_TILES_256X256 + c.shape;
  plan->splits = c.splits;
  plan->columns = c.cut;
  if (c.cut < a.J) {
    plan->rest_tiles = MOE_FP4_TILES_256X256 + c.rest_shape;
    plan->rest_splits = c.rest_splits;
  }
  return MOE_FP4_OK;
}

size_t norm_part_bytes(const NormArgs& a) { return (size_t)norm_blocks(a) * 2 * a.H * 4; }

}  // namespace

extern "C" {

int moe_fp4_grouped_workspace_size(const moe_fp4_grouped_dims* dims, int op, size_t* bytes) {
  if (!bytes) return MOE_FP4_EINVAL;
  ProductArgs a;
  const int rc = grouped_args(dims, op, false, a);
  if (rc != MOE_FP4_OK) return rc;
  a.offsets = some_offsets;
  *bytes = product_workspace(a, op);
  return MOE_FP4_OK;
}

int moe_fp4_grouped_plan(const moe_fp4_grouped_dims* dims, int op, moe_fp4_product_plan* plan) {
  if (!plan) return MOE_FP4_EINVAL;
  ProductArgs a;
  const int rc = grouped_args(dims, op, false, a);
  if (rc != MOE_FP4_OK) return rc;
  a.offsets = some_offsets;
  return product_plan(a, op, plan);
}

int moe_fp4_grouped_forward(const moe_fp4_grouped_dims* dims, const void* x, const void* w,
                            const int32_t* offsets, const int32_t* rows, void* y, int flags,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
  return grouped(dims, kFwd, x, w, offsets, rows, y, flags, ws, ws_bytes, stream);
}

int moe_fp4_grouped_dgrad(const moe_fp4_grouped_dims* dims, const void* dy, const void* w,
                          const int32_t* offsets, void* dx, int flags, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  return grouped(dims, kDgrad, dy, w, offsets, nullptr, dx, flags, ws, ws_bytes, stream);
}

int moe_fp4_grouped_wgrad(const moe_fp4_grouped_dims* dims, const void* dy, const void* x,
                          const int32_t* offsets, const int32_t* rows, void* dw, int flags,
                          void* ws, size_t ws_bytes, hipStream_t stream) {
  return grouped(dims, kWgrad, dy, x, offsets, rows, dw, flags, ws, ws_bytes, stream);
}

int moe_fp4_linear_workspace_size(const moe_fp4_linear_dims* dims, int backward, size_t* bytes) {
  if (!bytes) return MOE_FP4_EINVAL;
  LinearStrides s;
  const int rc = linear_check(dims, backward != 0, s);
  if (rc != MOE_FP4_OK) return rc;
  *bytes = backward ? backward_layout(*dims, s).total
                    : product_workspace(linear_forward_args(*dims, s), kFwd);
  return MOE_FP4_OK;
}

int moe_fp4_linear_plan(const moe_fp4_linear_dims* dims, int op, moe_fp4_product_plan* plan) {
  if (!plan) return MOE_FP4_EINVAL;
  if (op < kFwd || op > kWgrad) return MOE_FP4_EUNSUPPORTED;
  LinearStrides s;
  const int rc = linear_check(dims, op != kFwd, s);
  if (rc != MOE_FP4_OK) return rc;
  return product_plan(op == kFwd ? linear_forward_args(*dims, s) : op == kDgrad ? linear_dgrad_args(*dims, s)
                                                                                 : linear_wgrad_args(*dims, s), op, plan);
}

int moe_fp4_linear(const moe_fp4_linear_dims* dims, const void* x, const void* w, const void* bias,
                   const void* residual, void* y, void* z, int flags, void* ws, size_t ws_bytes,
                   hipStream_t stream) {
  LinearStrides s;
  const int rc = linear_check(dims, false, s);
  if (rc != MOE_FP4_OK) return rc;
  const moe_fp4_linear_dims& d = *dims;
  if (flags & ~MOE_FP4_ACCUMULATE) return MOE_FP4_EUNSUPPORTED;
  if (!w || (d.M > 0 && (!x || !y))) return MOE_FP4_EINVAL;
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(z, 2) || !aligned(y, size_of(d.out_type)) ||
      !aligned(residual, size_of(d.out_type)) || !aligned(bias, size_of(d.bias_type)))
    return MOE_FP4_EALIGN;
  ProductArgs a = linear_forward_args(d, s);
  a.a = static_cast<const uint16_t*>(x);
  a.b = static_cast<const uint16_t*>(w);
  a.c = y;
  a.z = z;
  a.bias = bias;
  a.residual = residual;
  a.accumulate = (flags & MOE_FP4_ACCUMULATE) ? 1 : 0;
  const int wrc = workspace_check(ws, ws_bytes, product_workspace(a, kFwd));
  if (wrc != MOE_FP4_OK) return wrc;
  return done(launch_product(a, kFwd, ws, stream));
}

int moe_fp4_linear_backward(const moe_fp4_linear_dims* dims, const void* dy, const void* x,
                            const void* w, const void* z, void* dx, void* dw, float* db, int flags,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
  LinearStrides s;
  const int rc = linear_check(dims, true, s);
  if (rc != MOE_FP4_OK) return rc;
  const moe_fp4_linear_dims& d = *dims;
  if (flags & ~MOE_FP4_ACCUMULATE) return MOE_FP4_EUNSUPPORTED;
  if (!dx && !dw && !db && d.M > 0) return MOE_FP4_EINVAL;
  if (d.M > 0 && (!dy || (dw && !x) || (dx && !w) || (d.act != kActNone && !z)))
    return MOE_FP4_EINVAL;
  if (!aligned(dy, size_of(d.out_type)) || !aligned(x, 2) || !aligned(w, 2) || !aligned(z, 2) ||
      !aligned(dx, 2) || !aligned(dw, size_of(d.dw_type)) || !aligned(db, 4))
    return MOE_FP4_EALIGN;
  const BackwardWs l = backward_layout(d, s);
  const int wrc = workspace_check(ws, ws_bytes, l.total);
  if (wrc != MOE_FP4_OK) return wrc;
  char* const base = static_cast<char*>(ws);
  const int acc = (flags & MOE_FP4_ACCUMULATE) ? 1 : 0;
  const bool direct = dz_is_dy(d);
  const uint16_t* dz = static_cast<const uint16_t*>(dy);
  float* const factor = dz_has_factor(d) ? reinterpret_cast<float*>(base + l.factor) : nullptr;
  hipError_t err = hipSuccess;
  if (db || (!direct && (dx || dw))) {
    SlopeArgs p{};
    p.M = d.M; p.N = d.N; p.type = d.type; p.dy_type = d.out_type; p.act = d.act;
    p.dy = dy; p.lddy = s.y;
    p.z = static_cast<const uint16_t*>(z); p.ldz = s.z;
    if (!direct && (dx || dw)) {
      p.dz = reinterpret_cast<uint16_t*>(base + l.dz);
      dz = p.dz;
      p.factor = factor;
      p.top = reinterpret_cast<float*>(base + l.top);
    }
    p.db = db; p.accumulate = acc;
    p.part = reinterpret_cast<float*>(base + l.part);
    err = launch_slope(p, stream);
  }
  if (err == hipSuccess && dx) {
    ProductArgs a = linear_dgrad_args(d, s);
    a.a = dz;
    a.b = static_cast<const uint16_t*>(w);
    a.c = dx;
    a.factor = factor;
    err = launch_product(a, kDgrad, base + l.product, stream);
  }
  if (err == hipSuccess && dw) {
    ProductArgs a = linear_wgrad_args(d, s);
    a.a = dz;
    a.b = static_cast<const uint16_t*>(x);
    a.c = dw;
    a.factor = factor;
    a.accumulate = acc;
    err = launch_product(a, kWgrad, base + l.product, stream);
  }
  return done(err);
}

int moe_fp4_norm(const moe_fp4_norm_dims* dims, const void* x, const void* gamma, const void* beta,
                 void* y, float* mean, float* rstd, hipStream_t stream) {
  NormArgs a;
  const int rc = norm_args(dims, a);
  if (rc != MOE_FP4_OK) return rc;
  if (a.T > 0 && (!x || !y)) return MOE_FP4_EINVAL;
  if (!aligned(x, size_of(a.x_type)) || !aligned(y, size_of(a.y_type)) ||
      !aligned(gamma, size_of(a.w_type)) || !aligned(beta, size_of(a.w_type)) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return MOE_FP4_EALIGN;
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return done(launch_norm(a, stream));
}

int moe_fp4_norm_backward_workspace_size(const moe_fp4_norm_dims* dims, size_t* bytes) {
  if (!bytes) return MOE_FP4_EINVAL;
  NormArgs a;
  const int rc = norm_args(dims, a);
  if (rc != MOE_FP4_OK) return rc;
  *bytes = norm_part_bytes(a);
  return MOE_FP4_OK;
}

int moe_fp4_norm_backward(const moe_fp4_norm_dims* dims, const void* dy, const void* x,
                          const void* gamma, const float* mean, const float* rstd, void* dx,
                          float* dgamma, float* dbeta, int flags, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  NormArgs a;
  const int rc = norm_args(dims, a);
  if (rc != MOE_FP4_OK) return rc;
  if (flags & ~MOE_FP4_ACCUMULATE) return MOE_FP4_EUNSUPPORTED;
  if (a.T > 0 && (!dy || !x || !rstd || (!mean && !a.rms) || (!dx && !dgamma && !dbeta)))
    return MOE_FP4_EINVAL;
  if (!aligned(x, size_of(a.x_type)) || !aligned(dx, size_of(a.x_type)) ||
      !aligned(dy, size_of(a.y_type)) || !aligned(gamma, size_of(a.w_type)) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
    return MOE_FP4_EALIGN;
  if (dgamma || dbeta) {
    const int wrc = workspace_check(ws, ws_bytes, norm_part_bytes(a));
    if (wrc != MOE_FP4_OK) return wrc;
  }
  a.x = x;
  a.gamma = gamma;
  a.dy = dy;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dx = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.accumulate = (flags & MOE_FP4_ACCUMULATE) ? 1 : 0;
  a.part = static_cast<float*>(ws);
  return done(launch_norm_backward(a, stream));
}

}  // extern "C"
