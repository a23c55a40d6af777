// C-ABI of the router's losses and of the gradients' norm and clipping: argument
// validation and launches.  Every check runs on the host before the first HIP
// call, so a rejected call enqueues nothing.
#include <algorithm>

#include "api_common.h"
#include "grad_clip.h"
#include "router_loss.h"

using namespace moe_fp4;

namespace {

static_assert(MOE_FP4_SCORE_SOFTMAX == kScoreSoftmax && MOE_FP4_SCORE_SIGMOID == kScoreSigmoid, "scores");

int loss_args(const moe_fp4_router_loss_dims* dims, bool backward, RouterLossArgs& a) {
  if (!dims) return MOE_FP4_EINVAL;
  const moe_fp4_router_loss_dims& d = *dims;
  if (d.T < 0 || d.E < 1 || d.k < 1 || d.S < 1 || d.k > d.E) return MOE_FP4_EINVAL;
  if (d.T > kMaxProductRows || d.E > kMaxLossExperts || d.k > 16 || d.S > kMaxLossSequences || !type_ok(d.type) ||
      (d.score != kScoreSoftmax && d.score != kScoreSigmoid))
    return MOE_FP4_EUNSUPPORTED;
  if (backward && (!type_ok(d.out_type) || (d.out_type != d.type && d.type != kF32 && d.out_type != kF32)))
    return MOE_FP4_EUNSUPPORTED;
  a = RouterLossArgs{};
  if (!stride(d.ld, d.E, a.ld) || (backward && !stride(d.ldd, d.E, a.ldd))) return MOE_FP4_EINVAL;
  a.T = d.T;
  a.E = d.E;
  a.k = d.k;
  a.S = d.S;
  a.score = d.score;
  a.type = d.type;
  a.out_type = d.out_type;
  return MOE_FP4_OK;
}

// The tensors' sizes and types (clip: and those of the results).
int grad_check(const moe_fp4_grad_tensor* t, int n, bool clip) {
  if (n < 0 || (n > 0 && !t)) return MOE_FP4_EINVAL;
  if (n > kMaxGradTensors) return MOE_FP4_EUNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    if (t[i].n < 0) return MOE_FP4_EINVAL;
    if (t[i].n > (int64_t)1 << 40 || !type_ok(t[i].type)) return MOE_FP4_EUNSUPPORTED;
    if (clip && t[i].out &&
        (!type_ok(t[i].out_type) || (t[i].out_type != t[i].type && t[i].type != kF32)))
      return MOE_FP4_EUNSUPPORTED;
  }
  return MOE_FP4_OK;
}
int grad_pointers(const moe_fp4_grad_tensor* t, int n, bool clip) {
  for (int i = 0; i < n; ++i) {
    if (t[i].n > 0 && !t[i].data) return MOE_FP4_EINVAL;
    if (!aligned(t[i].data, size_of(t[i].type)) || (clip && t[i].out && !aligned(t[i].out, size_of(t[i].out_type))))
      return MOE_FP4_EALIGN;
  }
  return MOE_FP4_OK;
}

// Whether a written range meets another range, read or written.  A tensor clipped in
// place is one range.
struct Range {
  uintptr_t lo, hi;
  bool written;
};
bool overlaps(const moe_fp4_grad_tensor* t, int n) {
  Range r[2 * kMaxGradTensors];  // 192 KB of the stack
  int m = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(t[i].data), b = reinterpret_cast<uintptr_t>(t[i].out);
    const bool in_place = !b || (b == a && t[i].out_type == t[i].type);
    r[m++] = Range{a, a + (uintptr_t)t[i].n * size_of(t[i].type), in_place};
    if (!in_place) r[m++] = Range{b, b + (uintptr_t)t[i].n * size_of(t[i].out_type), true};
  }
  std::sort(r, r + m, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t any = 0, written = 0;  // the furthest ends so far
  for (int i = 0; i < m; ++i) {
    if (r[i].lo < written || (r[i].written && r[i].lo < any)) return true;
    any = std::max(any, r[i].hi);
    if (r[i].written) written = std::max(written, r[i].hi);
  }
  return false;
}

}  // namespace

extern "C" {

int moe_fp4_router_loss_workspace_size(const moe_fp4_router_loss_dims* dims, size_t* bytes) {
  if (!bytes) return MOE_FP4_EINVAL;
  RouterLossArgs a;
  const int rc = loss_args(dims, false, a);
  if (rc != MOE_FP4_OK) return rc;
  *bytes = router_loss_workspace(a);
  return MOE_FP4_OK;
}

int moe_fp4_router_loss(const moe_fp4_router_loss_dims* dims, const void* logits, const int32_t* idx,
                        const int32_t* seqs, const uint8_t* mask, int32_t* counts, int32_t* tokens,
                        float* probs, float* balance, float* z, void* ws, size_t ws_bytes,
                        hipStream_t stream) {
  RouterLossArgs a;
  const int rc = loss_args(dims, false, a);
  if (rc != MOE_FP4_OK) return rc;
  if (!counts || !tokens || !probs || !balance || !z || (a.T > 0 && (!logits || !idx)) || (!seqs && a.S != 1))
    return MOE_FP4_EINVAL;
  if (!aligned(logits, size_of(a.type)) || !aligned(idx, 4) || !aligned(seqs, 4) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || !aligned(probs, 4) || !aligned(balance, 4) || !aligned(z, 4))
    return MOE_FP4_EALIGN;
  const int wrc = workspace_check(ws, ws_bytes, router_loss_workspace(a));
  if (wrc != MOE_FP4_OK) return wrc;
  a.logits = logits;
  a.idx = idx;
  a.seqs = seqs;
  a.mask = mask;
  a.counts = counts;
  a.tokens = tokens;
  a.probs = probs;
  a.balance = balance;
  a.z = z;
  return done(launch_router_loss(a, ws, stream));
}

int moe_fp4_router_loss_backward(const moe_fp4_router_loss_dims* dims, const void* logits,
                                 const int32_t* idx, const int32_t* seqs, const uint8_t* mask,
                                 const int32_t* counts, const int32_t* tokens, const float* dbalance,
                                 const float* dz, const float* gates, const float* dgates,
                                 void* dlogits, int flags, hipStream_t stream) {
  RouterLossArgs a;
  const int rc = loss_args(dims, true, a);
  if (rc != MOE_FP4_OK) return rc;
  if (flags & ~MOE_FP4_ACCUMULATE) return MOE_FP4_EUNSUPPORTED;
  if (!seqs && a.S != 1) return MOE_FP4_EINVAL;
  if (a.T > 0 && (!dlogits || (!dbalance && !dz && !gates) || (!gates != !dgates) || (gates && !idx) ||
                  ((dbalance || dz) && (!logits || !tokens)) || (dbalance && !counts)))
    return MOE_FP4_EINVAL;
  if (!aligned(logits, size_of(a.type)) || !aligned(idx, 4) || !aligned(seqs, 4) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || !aligned(dbalance, 4) || !aligned(dz, 4) || !aligned(gates, 4) || !aligned(dgates, 4) ||
      !aligned(dlogits, size_of(a.out_type)))
    return MOE_FP4_EALIGN;
  a.logits = logits;
  a.idx = idx;
  a.seqs = seqs;
  a.mask = mask;
  a.counts_in = counts;
  a.tokens_in = tokens;
  a.dbalance = dbalance;
  a.dz = dz;
  a.gates = gates;
  a.dgates = dgates;
  a.dlogits = dlogits;
  a.accumulate = (flags & MOE_FP4_ACCUMULATE) ? 1 : 0;
  return done(launch_router_loss_backward(a, stream));
}

int moe_fp4_grad_sumsq_workspace_size(const moe_fp4_grad_tensor* tensors, int n_tensors, size_t* bytes) {
  if (!bytes) return MOE_FP4_EINVAL;
  const int rc = grad_check(tensors, n_tensors, false);
  if (rc != MOE_FP4_OK) return rc;
  *bytes = grad_sumsq_workspace(tensors, n_tensors);
  return MOE_FP4_OK;
}

int moe_fp4_grad_sumsq(const moe_fp4_grad_tensor* tensors, int n_tensors, double* sumsq, int flags,
                       void* ws, size_t ws_bytes, hipStream_t stream) {
  int rc = grad_check(tensors, n_tensors, false);
  if (rc != MOE_FP4_OK) return rc;
  if (flags & ~MOE_FP4_ACCUMULATE) return MOE_FP4_EUNSUPPORTED;
  if (!sumsq) return MOE_FP4_EINVAL;
  if (!aligned(sumsq, 8)) return MOE_FP4_EALIGN;
  rc = grad_pointers(tensors, n_tensors, false);
  if (rc != MOE_FP4_OK) return rc;
  rc = workspace_check(ws, ws_bytes, grad_sumsq_workspace(tensors, n_tensors));
  if (rc != MOE_FP4_OK) return rc;
  return done(launch_grad_sumsq(tensors, n_tensors, sumsq, flags & MOE_FP4_ACCUMULATE, ws, stream));
}

int moe_fp4_grad_clip(const moe_fp4_grad_tensor* tensors, int n_tensors, const double* sumsq,
                      float max_norm, float eps, float* norm, hipStream_t stream) {
  int rc = grad_check(tensors, n_tensors, true);
  if (rc != MOE_FP4_OK) return rc;
  if (!sumsq || !(max_norm >= 0.f) || !(eps >= 0.f)) return MOE_FP4_EINVAL;
  if (!aligned(sumsq, 8) || !aligned(norm, 4)) return MOE_FP4_EALIGN;
  rc = grad_pointers(tensors, n_tensors, true);
  if (rc != MOE_FP4_OK) return rc;
  if (overlaps(tensors, n_tensors)) return MOE_FP4_EINVAL;
  return done(launch_grad_clip(tensors, n_tensors, sumsq, max_norm, eps, norm, stream));
}

}  // extern "C"
