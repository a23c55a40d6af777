// Internal launch interface of the dense product with 4-bit weights.
#pragma once

#include "block.h"

namespace moe_fp4 {

enum { kMx = 0, kInt4 = 1 };  // the values of the public header

struct W4Args {
  int M, N, K;
  int code, group, type, out_type, bias_type, scale_type, act, accumulate;
  int64_t ldx, ldy, ldr, ldw;
  const uint16_t* x;
  const uint8_t* codes;
  const void* scales;     // [N][groups]
  const uint8_t* zeros;   // [N][groups] or null
  const void *bias, *residual;
  void* y;
  int groups;             // scales of a row
};
void launch_w4_row(const W4Args& a, hipStream_t stream);  // one or two rows
void launch_w4_hold(const W4Args& a, hipStream_t stream); // up to 16 rows; MX, int4 groups of 128 and 256
// Any rows, where the scales and zeros of a column are at most kWideRowBytes: 256 columns' lie in
// LDS from the start, in the 40 KB that codes and rows leave.  That is K up to 5120 for MX and for int4
// groups of 64 with 16-bit scales (3392 with zeros), 2560 for groups of 32, 10240 for 128.  Past it
// the tiles take over: 64 rows of 32768 x 5120 51 us, x 5248 65, x 7168 79.
constexpr int kWideRowBytes = 160;
inline int w4_row_bytes(const W4Args& a) {
  return a.groups * ((a.code == kMx ? 1 : a.scale_type == kF32 ? 4 : 2) + (a.zeros ? 1 : 0));
}
void launch_w4_wide(const W4Args& a, hipStream_t stream);
hipError_t launch_w4(const W4Args& a, hipStream_t stream);

}  // namespace moe_fp4
