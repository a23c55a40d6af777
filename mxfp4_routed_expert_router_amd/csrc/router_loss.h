// Internal launch interface of the router's losses.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe_fp4 {

enum { kScoreSoftmax = 0, kScoreSigmoid = 1 };  // the values of the public header

constexpr int kMaxLossExperts = 1024, kMaxLossSequences = 65536;

struct RouterLossArgs {
  int T, E, k, S;
  int score, type, out_type;
  int64_t ld, ldd;
  const void* logits;
  const int32_t* idx;      // [T][k]
  const int32_t* seqs;     // [S+1], null: one sequence of all tokens
  const uint8_t* mask;     // [T], null: all ones
  // forward
  int32_t *counts, *tokens;            // [S][E], [S]
  float *probs, *balance, *z;          // [S][E], [S], [S]
  // set by launch_router_loss
  int tokens_of_block;
  float* part;                         // rows of a workgroup's piece of a sequence
  double* dots;                        // [S][E / 32, rounded up]
  int32_t* tickets;                    // [S]
  // backward
  const int32_t *counts_in, *tokens_in;
  const float *dbalance, *dz;          // [S], or null
  const float *gates, *dgates;         // [T][k], or null
  void* dlogits;
  int accumulate;
};

size_t router_loss_workspace(const RouterLossArgs& a);
hipError_t launch_router_loss(RouterLossArgs a, void* ws, hipStream_t stream);
hipError_t launch_router_loss_backward(RouterLossArgs a, hipStream_t stream);

}  // namespace moe_fp4
