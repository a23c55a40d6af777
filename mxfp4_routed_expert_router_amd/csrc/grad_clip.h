// Internal launch interface of the gradients' norm and clipping.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_fp4.h"

namespace moe_fp4 {

constexpr int kMaxGradTensors = 4096;

size_t grad_sumsq_workspace(const moe_fp4_grad_tensor* t, int n);
hipError_t launch_grad_sumsq(const moe_fp4_grad_tensor* t, int n, double* sumsq, int accumulate, void* ws,
                             hipStream_t stream);
hipError_t launch_grad_clip(const moe_fp4_grad_tensor* t, int n, const double* sumsq, float max_norm, float eps,
                            float* norm, hipStream_t stream);

}  // namespace moe_fp4
