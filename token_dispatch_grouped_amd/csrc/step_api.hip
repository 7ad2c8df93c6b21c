// C ABI of routing by scores, RMS norm and the AdamW step. Host-side validation, then
// launches; every check runs before anything is enqueued.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "moe_internal.h"

namespace {

moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

bool valid_dtype(moe_dtype dt) { return dt == MOE_F32 || dt == MOE_BF16; }

size_t elem_bytes(moe_dtype dt) { return dt == MOE_BF16 ? 2 : 4; }

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <typename... P>
bool all_aligned(size_t to, P... p) { return (aligned(p, to) && ...); }

template <typename... P>
bool any_null(P... p) { return ((p == nullptr) || ...); }

moe_status check_route(const moe_shape* s, const moe_router* r) {
  if (s == nullptr || r == nullptr) return MOE_EINVAL;
  if (s->T < 0 || s->E < 1 || s->k < 1 || s->k > s->E) return MOE_EINVAL;
  if (s->T > INT32_MAX || s->T * static_cast<int64_t>(s->k) > INT32_MAX) return MOE_EINVAL;
  if (s->E > moe::kMaxExperts) return MOE_EUNSUPPORTED;
  if (r->score != MOE_SOFTMAX && r->score != MOE_SIGMOID) return MOE_EINVAL;
  if (r->renormalize != 0 && r->renormalize != 1) return MOE_EINVAL;
  if (!isfinite(r->scale)) return MOE_EINVAL;
  return MOE_OK;
}

moe_status check_norm(const moe_shape* s, moe_dtype dt, moe_dtype wdt) {
  if (s == nullptr || s->T < 0 || s->d <= 0 || s->d % 8 != 0) return MOE_EINVAL;
  if (!valid_dtype(dt) || !valid_dtype(wdt)) return MOE_EINVAL;
  if (s->d > moe::layer_norm_max_d() || s->T > (int64_t{1} << 30)) return MOE_EUNSUPPORTED;
  if (dt == MOE_F32 && wdt == MOE_BF16) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// ----------------------------------------------------------------------- AdamW

struct Range {
  uintptr_t lo, hi;
  bool written;
};

moe_status check_adamw(const moe_adamw_tensor* t, int32_t n, const moe_adamw_args* a) {
  if (a == nullptr || n < 0 || (n > 0 && t == nullptr)) return MOE_EINVAL;
  if (a->state != MOE_STATE_F32 && a->state != MOE_STATE_E4M3) return MOE_EINVAL;
  if (a->state == MOE_STATE_E4M3 && a->rounding != MOE_NEAREST && a->rounding != MOE_DITHER) return MOE_EINVAL;
  if (!isfinite(a->lr) || !(a->beta1 >= 0 && a->beta1 < 1) || !(a->beta2 >= 0 && a->beta2 < 1)) return MOE_EINVAL;
  if (!(a->eps >= 1e-30) || !isfinite(static_cast<float>(a->eps)) || !isfinite(a->weight_decay)) return MOE_EINVAL;
  if (a->d_step == nullptr && a->step < 1) return MOE_EINVAL;
  if (!all_aligned(4, a->norm, a->d_lr) || !aligned(a->d_step, 8)) return MOE_EINVAL;
  if (a->norm != nullptr && !(a->max_norm >= 0.f && isfinite(a->max_norm))) return MOE_EINVAL;
  const bool e4m3 = a->state == MOE_STATE_E4M3;
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[7 * static_cast<size_t>(n) + 3]);
  if (!r) return MOE_EHIP;
  size_t m = 0;
  auto add = [&](const void* p, size_t bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    r[m++] = Range{at, at + bytes, written};
  };
  if (a->norm != nullptr) add(a->norm, 4, false);
  if (a->d_lr != nullptr) add(a->d_lr, 4, false);
  if (a->d_step != nullptr) add(a->d_step, 8, false);
  for (int32_t i = 0; i < n; ++i) {
    const moe_adamw_tensor& e = t[i];
    if (e.numel < 0 || !valid_dtype(e.param_dt) || !valid_dtype(e.grad_dt)) return MOE_EINVAL;
    if (e.numel > (int64_t{1} << 40)) return MOE_EUNSUPPORTED;
    if (a->weight_decays != nullptr && !isfinite(a->weight_decays[i])) return MOE_EINVAL;
    if (e.master != nullptr && e.param_dt != MOE_BF16) return MOE_EINVAL;
    if (e.numel == 0) continue;
    if (any_null(static_cast<const void*>(e.param), e.grad, static_cast<const void*>(e.exp_avg),
                 static_cast<const void*>(e.exp_avg_sq)))
      return MOE_EINVAL;
    if (!aligned(e.param, elem_bytes(e.param_dt)) || !aligned(e.grad, elem_bytes(e.grad_dt)) || !aligned(e.master, 4))
      return MOE_EINVAL;
    const size_t numel = static_cast<size_t>(e.numel), held = e4m3 ? 1 : 4;
    if (!all_aligned(held, e.exp_avg, e.exp_avg_sq)) return MOE_EINVAL;
    add(e.param, numel * elem_bytes(e.param_dt), true);
    add(e.grad, numel * elem_bytes(e.grad_dt), false);
    if (e.master != nullptr) add(e.master, numel * 4, true);
    add(e.exp_avg, numel * held, true);
    add(e.exp_avg_sq, numel * held, true);
    if (e4m3) {
      if (any_null(e.exp_avg_scale, e.exp_avg_sq_scale) || !all_aligned(4, e.exp_avg_scale, e.exp_avg_sq_scale))
        return MOE_EINVAL;
      const size_t blocks = (numel + MOE_STATE_BLOCK - 1) / MOE_STATE_BLOCK;
      add(e.exp_avg_scale, blocks * 4, true);
      add(e.exp_avg_sq_scale, blocks * 4, true);
    }
  }
  std::sort(r.get(), r.get() + m, [](const Range& x, const Range& y) { return x.lo < y.lo; });
  // the furthest end so far, of any tensor and of the written ones
  uintptr_t any_end = 0, written_end = 0;
  for (size_t j = 0; j < m; ++j) {
    if (r[j].lo < written_end || (r[j].written && r[j].lo < any_end)) return MOE_EINVAL;
    any_end = std::max(any_end, r[j].hi);
    if (r[j].written) written_end = std::max(written_end, r[j].hi);
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_route_experts(const moe_shape* s, const moe_router* r, const float* logits, int32_t* topk_idx,
                             float* topk_w, hipStream_t stream) {
  const moe_status st = check_route(s, r);
  if (st != MOE_OK) return st;
  if (r->groups < 1 || s->E % r->groups != 0 || r->top_groups < 1 || r->top_groups > r->groups) return MOE_EINVAL;
  if (r->group_top != 1 && r->group_top != 2) return MOE_EINVAL;
  if (s->k > r->top_groups * (s->E / r->groups)) return MOE_EINVAL;
  if (!aligned(r->bias, 4)) return MOE_EINVAL;
  if (s->T == 0) return MOE_OK;
  if (any_null(logits, static_cast<const float*>(topk_w)) || topk_idx == nullptr) return MOE_EINVAL;
  if (!all_aligned(4, logits, topk_w, topk_idx)) return MOE_EINVAL;
  return from_hip(moe::launch_route_experts(*r, logits, topk_idx, topk_w, s->T, s->E, s->k, stream));
}

moe_status moe_route_experts_backward(const moe_shape* s, const moe_router* r, const float* logits,
                                      const int32_t* topk_idx, const float* d_topk_w, float* d_logits,
                                      hipStream_t stream) {
  const moe_status st = check_route(s, r);
  if (st != MOE_OK) return st;
  if (s->T == 0) return MOE_OK;
  if (any_null(logits, d_topk_w, static_cast<const float*>(d_logits)) || topk_idx == nullptr) return MOE_EINVAL;
  if (!all_aligned(4, logits, topk_idx, d_topk_w, d_logits)) return MOE_EINVAL;
  return from_hip(moe::launch_route_experts_backward(*r, logits, topk_idx, d_topk_w, d_logits, s->T, s->E, s->k, stream));
}

moe_status moe_rms_norm(const moe_shape* s, moe_dtype dt, const void* x, const void* residual, moe_dtype wdt,
                        const void* weight, float eps, void* y, void* sum, float* rstd, void* q, float* q_scale,
                        hipStream_t stream) {
  const moe_status st = check_norm(s, dt, wdt);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f) || isinf(eps)) return MOE_EINVAL;
  if ((q == nullptr) != (q_scale == nullptr)) return MOE_EINVAL;
  if (q != nullptr && dt != MOE_BF16) return MOE_EUNSUPPORTED;
  if (s->T == 0) return MOE_OK;
  if (any_null(x, weight) || rstd == nullptr || (y == nullptr && q == nullptr)) return MOE_EINVAL;
  if (residual != nullptr && (sum == nullptr || sum == y)) return MOE_EINVAL;
  if (!all_aligned(16, x, residual, weight, y, q) || !all_aligned(4, rstd, q_scale)) return MOE_EINVAL;
  if (residual != nullptr && !aligned(sum, 16)) return MOE_EINVAL;
  return from_hip(moe::launch_rms_norm(x, residual, weight, eps, y, sum, rstd, q, q_scale, s->T, s->d, dt == MOE_BF16,
                                       wdt == MOE_BF16, stream));
}

size_t moe_rms_norm_backward_workspace_bytes(const moe_shape* s) {
  if (check_norm(s, MOE_F32, MOE_F32) != MOE_OK) return 0;
  return moe::rms_norm_backward_workspace_bytes(s->T, s->d);
}

moe_status moe_rms_norm_backward(const moe_shape* s, moe_dtype dt, const void* d_y, const void* sum, moe_dtype wdt,
                                 const void* weight, const float* rstd, const void* d_s, void* d_x, void* d_weight,
                                 void* workspace, hipStream_t stream) {
  const moe_status st = check_norm(s, dt, wdt);
  if (st != MOE_OK) return st;
  if (weight == nullptr || d_weight == nullptr) return MOE_EINVAL;
  // with no rows only the (zero) weight gradient is written
  if (s->T > 0 && (any_null(d_y, sum, static_cast<const void*>(d_x), static_cast<const void*>(workspace)) ||
                   rstd == nullptr))
    return MOE_EINVAL;
  if (!all_aligned(16, d_y, sum, weight, d_s, d_x, d_weight, workspace) || !aligned(rstd, 4)) return MOE_EINVAL;
  return from_hip(moe::launch_rms_norm_backward(d_y, sum, weight, rstd, d_s, d_x, d_weight, workspace, s->T, s->d,
                                                dt == MOE_BF16, wdt == MOE_BF16, stream));
}

moe_status moe_adamw(const moe_adamw_tensor* tensors, int32_t n, const moe_adamw_args* args, hipStream_t stream) {
  const moe_status st = check_adamw(tensors, n, args);
  if (st != MOE_OK) return st;
  return from_hip(moe::launch_adamw(tensors, n, *args, stream));
}

}  // extern "C"
