// Argument checks shared by the C-ABI sources of the operators around the routed
// experts.  Host only.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_fp4.h"
#include "block.h"

namespace moe_fp4 {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t size_of(int type) { return type == kF32 ? 4 : 2; }
inline bool type_ok(int t) { return t == kF32 || t == kBf16 || t == kF16; }
inline bool is16(int t) { return t == kBf16 || t == kF16; }
// A row stride as given (0: dense); false where rows would overlap, or where a
// tile's byte offsets would not fit the kernels' 32 bits.
constexpr int64_t kMaxRowStride = 1 << 22;
inline bool stride(int64_t given, int width, int64_t& ld) {
  ld = given ? given : width;
  return ld >= width && ld <= kMaxRowStride;
}
inline int workspace_check(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_FP4_OK;
  if (!ws) return MOE_FP4_EINVAL;
  if (!aligned(ws, kAlign)) return MOE_FP4_EALIGN;
  return have < need ? MOE_FP4_EWORKSPACE : MOE_FP4_OK;
}
inline int done(hipError_t e) { return e == hipSuccess ? MOE_FP4_OK : MOE_FP4_EHIP; }

}  // namespace moe_fp4
