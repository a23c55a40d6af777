// C-ABI of the dense product with 4-bit weights: argument validation and launch.
// Every check runs on the host before the first HIP call, so a rejected call
// enqueues nothing.
#include "api_common.h"
#include "w4.h"

using namespace moe_fp4;

static_assert(MOE_FP4_W4_MX == kMx && MOE_FP4_W4_INT4 == kInt4, "codes");

extern "C" int moe_fp4_linear_w4(const moe_fp4_w4_dims* dims, const void* x, const uint8_t* codes,
                                 const void* scales, const uint8_t* zeros, const void* bias,
                                 const void* residual, void* y, int flags, hipStream_t stream) {
  if (!dims) return MOE_FP4_EINVAL;
  const moe_fp4_w4_dims& d = *dims;
  if (d.M < 0 || d.N < 1 || d.K < 1 || d.group < 1) return MOE_FP4_EINVAL;
  const bool int4 = d.code == kInt4;
  if (d.M > kMaxProductRows || d.N > kMaxWidth || d.K > kMaxWidth || d.K % 32 || (!int4 && d.code != kMx) ||
      !is16(d.type) || (d.out_type != d.type && d.out_type != kF32) || !type_ok(d.bias_type) ||
      (int4 && !type_ok(d.scale_type)) || d.act < kActNone || d.act > kActSilu || (flags & ~MOE_FP4_ACCUMULATE))
    return MOE_FP4_EUNSUPPORTED;
  if (d.group != 32 && (!int4 || (d.group != 64 && d.group != 128 && d.group != 256))) return MOE_FP4_EUNSUPPORTED;
  W4Args a{};
  if (!stride(d.ldx, d.K, a.ldx) || !stride(d.ldy, d.N, a.ldy) || !stride(d.ldr, d.N, a.ldr) ||
      !stride(d.ldw, d.K / 2, a.ldw))
    return MOE_FP4_EINVAL;
  if (!codes || !scales || (zeros && !int4) || (d.M > 0 && (!x || !y))) return MOE_FP4_EINVAL;
  if (!aligned(x, 2) || !aligned(codes, 16) || a.ldw % 16 || (int4 && !aligned(scales, size_of(d.scale_type))) ||
      !aligned(bias, size_of(d.bias_type)) || !aligned(residual, size_of(d.out_type)) || !aligned(y, size_of(d.out_type)))
    return MOE_FP4_EALIGN;
  if (d.M == 0) return MOE_FP4_OK;
  a.M = d.M;
  a.N = d.N;
  a.K = d.K;
  a.code = d.code;
  a.group = d.group;
  a.type = d.type;
  a.out_type = d.out_type;
  a.bias_type = d.bias_type;
  a.scale_type = d.scale_type;
  a.act = d.act;
  a.accumulate = (flags & MOE_FP4_ACCUMULATE) ? 1 : 0;
  a.x = static_cast<const uint16_t*>(x);
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.groups = (d.K + d.group - 1) / d.group;
  return done(launch_w4(a, stream));
}
