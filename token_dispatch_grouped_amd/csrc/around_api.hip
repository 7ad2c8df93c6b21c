// C ABI of what stands around the experts: residual add and layer norm, the
// experts in 8-bit integers, the gradient norm and clipping. Host-side validation,
// then launches; every check runs before anything is enqueued.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "moe_internal.h"

namespace {

moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

bool valid_dtype(moe_dtype dt) { return dt == MOE_F32 || dt == MOE_BF16; }

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <typename... P>
bool aligned16(P... p) { return (aligned(p, 16) && ...); }

template <typename... P>
bool any_null(P... p) { return ((p == nullptr) || ...); }

// ------------------------------------------------------------------ layer norm

moe_status check_norm(const moe_shape* s, moe_dtype dt, moe_dtype wdt) {
  if (s == nullptr || s->T < 0 || s->d <= 0 || s->d % 8 != 0) return MOE_EINVAL;
  if (!valid_dtype(dt) || !valid_dtype(wdt)) return MOE_EINVAL;
  if (s->d > moe::layer_norm_max_d() || s->T > (int64_t{1} << 30)) return MOE_EUNSUPPORTED;
  if (dt == MOE_F32 && wdt == MOE_BF16) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// ------------------------------------------------------------------------ int8

int64_t n_max_of(const moe_shape* s) {
  const int64_t e_loc = s->e_end - s->e_begin;
  return s->T * (s->k < e_loc ? s->k : e_loc);
}

// The parts of the int8 workspace, each 256-byte aligned.
struct Int8Workspace {
  size_t xq, xs, h, hq, hs, plan, bytes;
  int tile_rows;
  explicit Int8Workspace(const moe_shape* s) {
    const int64_t n_max = n_max_of(s);
    const int e_loc = s->e_end - s->e_begin, d = s->d, d_ff = s->d_ff;
    const size_t n = static_cast<size_t>(n_max);
    size_t at = 0;
    auto part = [&](size_t b) {
      const size_t here = at;
      at += (b + 255) / 256 * 256;
      return here;
    };
    xq = part(n * moe::int8_kblocks(d) * 64);
    xs = part(n * sizeof(float));
    h = part(n * static_cast<size_t>(d_ff) * 2);
    hq = part(n * moe::int8_kblocks(d_ff) * 64);
    hs = part(n * sizeof(float));
    tile_rows = moe::int8_tile_rows(s->T, s->k, s->E, e_loc, d, d_ff);
    plan = part(n > 0 ? moe::int8_plan_bytes(n_max, e_loc) : 0);
    bytes = at;
  }
};

// d, d_ff and the local range
moe_status check_experts(const moe_shape* s) {
  if (s == nullptr) return MOE_EINVAL;
  if (s->E < 1 || s->d <= 0 || s->d_ff <= 0 || s->d % 8 != 0 || s->d_ff % 8 != 0) return MOE_EINVAL;
  if (s->e_begin < 0 || s->e_end > s->E || s->e_begin >= s->e_end) return MOE_EINVAL;
  if (s->E > moe::kMaxExperts) return MOE_EUNSUPPORTED;
  if (s->d > moe::int8_max_k() || s->d_ff > moe::int8_max_k()) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

moe_status check_int8(const moe_shape* s) {
  const moe_status st = check_experts(s);
  if (st != MOE_OK) return st;
  if (s->T < 0 || s->k < 1 || s->k > s->E) return MOE_EINVAL;
  if (s->T * static_cast<int64_t>(s->k) > INT32_MAX) return MOE_EINVAL;
  return MOE_OK;
}

// The FFN on bf16 rows x, or (scale_x != nullptr) on rows that are codes already
moe_status run_int8(const moe_shape* s, const void* x, const float* scale_x, const int32_t* perm, const int32_t* offsets,
                    const void* q_gate_up, const float* scale_gate_up, const void* q_down, const float* scale_down,
                    void* y, void* workspace, hipStream_t stream) {
  if (s->T == 0) return MOE_OK;
  if (any_null(x, q_gate_up, q_down, static_cast<const void*>(y), static_cast<const void*>(workspace)) ||
      perm == nullptr || offsets == nullptr || scale_gate_up == nullptr || scale_down == nullptr)
    return MOE_EINVAL;
  if (!aligned16(x, q_gate_up, q_down, static_cast<const void*>(y), static_cast<const void*>(workspace)) ||
      !aligned(perm, 4) || !aligned(offsets, 4) || !aligned(scale_gate_up, 4) || !aligned(scale_down, 4))
    return MOE_EINVAL;
  const int64_t n_max = n_max_of(s);
  const int e_loc = s->e_end - s->e_begin, d = s->d, d_ff = s->d_ff;
  const Int8Workspace ws(s);
  char* p = static_cast<char*>(workspace);
  float* xs = reinterpret_cast<float*>(p + ws.xs);
  float* hs = reinterpret_cast<float*>(p + ws.hs);
  if (ws.tile_rows == moe::kInt8FewRows)
    return from_hip(moe::launch_int8_few(x, scale_x, perm, offsets, q_gate_up, scale_gate_up, q_down, scale_down,
                                         p + ws.h, y, d, d_ff, s->E, s->e_begin, e_loc, s->k, s->T, n_max, stream));
  hipError_t e = scale_x != nullptr
                     ? moe::launch_gather_codes(x, scale_x, perm, offsets, p + ws.xq, xs, s->e_begin, s->e_end, s->k,
                                                s->T, d, n_max, p + ws.plan, ws.tile_rows, stream)
                     : moe::launch_quantize_rows(x, perm, offsets, p + ws.xq, xs, s->e_begin, s->e_end, s->k, s->T, d,
                                                 n_max, p + ws.plan, ws.tile_rows, stream);
  if (e == hipSuccess)
    e = moe::launch_grouped_gemm_int8(p + ws.xq, xs, q_gate_up, scale_gate_up, p + ws.h, p + ws.plan, ws.tile_rows, e_loc, d,
                                      d_ff, n_max, true, stream);
  if (e == hipSuccess)
    e = moe::launch_quantize_rows(p + ws.h, nullptr, offsets, p + ws.hq, hs, s->e_begin, s->e_end, s->k, s->T, d_ff,
                                  n_max, nullptr, 0, stream);
  if (e == hipSuccess)
    e = moe::launch_grouped_gemm_int8(p + ws.hq, hs, q_down, scale_down, y, p + ws.plan, ws.tile_rows, e_loc, d_ff, d,
                                      n_max, false, stream);
  return from_hip(e);
}

// ------------------------------------------------------------------- gradients

size_t elem_bytes(moe_dtype dt) { return dt == MOE_BF16 ? 2 : 4; }

moe_status check_list(const moe_tensor* t, int32_t n) {
  if (n < 0 || (n > 0 && t == nullptr)) return MOE_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    if (!valid_dtype(t[i].dt) || t[i].numel < 0) return MOE_EINVAL;
    if (t[i].numel > (int64_t{1} << 48)) return MOE_EUNSUPPORTED;
    if (t[i].numel > 0 && (t[i].data == nullptr || !aligned(t[i].data, elem_bytes(t[i].dt)))) return MOE_EINVAL;
  }
  return MOE_OK;
}

struct Range {
  uintptr_t lo, hi;
  bool written;
};

// Whether the list can be scaled into `out` (null: in place): each tensor's bytes
// are sorted by address, and a written one may meet no other but its own gradient.
// The norm (and the workspace, if any) are among them, written by the call or not.
moe_status check_clip(const moe_tensor* t, const moe_tensor* out, int32_t n, float max_norm, const float* norm,
                      bool norm_written, const void* workspace, size_t ws_bytes) {
  const moe_status st = check_list(t, n);
  if (st != MOE_OK) return st;
  if (!(max_norm >= 0.f) || isinf(max_norm)) return MOE_EINVAL;
  if (out != nullptr) {
    const moe_status so = check_list(out, n);
    if (so != MOE_OK) return so;
    for (int32_t i = 0; i < n; ++i)
      if (out[i].numel != t[i].numel || out[i].dt != t[i].dt) return MOE_EINVAL;
  }
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * static_cast<size_t>(n) + 2]);
  if (!r) return MOE_EHIP;
  size_t m = 0;
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm), ws = reinterpret_cast<uintptr_t>(workspace);
  r[m++] = Range{at, at + sizeof(float), norm_written};
  if (workspace != nullptr) r[m++] = Range{ws, ws + ws_bytes, true};
  for (int32_t i = 0; i < n; ++i) {
    const size_t bytes = static_cast<size_t>(t[i].numel) * elem_bytes(t[i].dt);
    if (bytes == 0) continue;
    const uintptr_t src = reinterpret_cast<uintptr_t>(t[i].data);
    const uintptr_t dst = out != nullptr ? reinterpret_cast<uintptr_t>(out[i].data) : src;
    if (dst != src) r[m++] = Range{src, src + bytes, false};
    r[m++] = Range{dst, dst + bytes, true};
  }
  std::sort(r.get(), r.get() + m, [](const Range& a, const Range& b) { return a.lo < b.lo; });
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

moe_status moe_layer_norm(const moe_shape* s, moe_dtype dt, const void* x, const void* residual, moe_dtype wdt,
                          const void* weight, const void* bias, float eps, void* y, void* sum, float* mean,
                          float* rstd, hipStream_t stream) {
  const moe_status st = check_norm(s, dt, wdt);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f) || isinf(eps)) return MOE_EINVAL;
  if (s->T == 0) return MOE_OK;
  if (any_null(x, weight, static_cast<const void*>(y)) || mean == nullptr || rstd == nullptr) return MOE_EINVAL;
  if (residual != nullptr && (sum == nullptr || sum == y)) return MOE_EINVAL;
  if (!aligned16(x, residual, weight, bias, static_cast<const void*>(y)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return MOE_EINVAL;
  if (residual != nullptr && !aligned(sum, 16)) return MOE_EINVAL;
  return from_hip(moe::launch_layer_norm(x, residual, weight, bias, eps, y, sum, mean, rstd, s->T, s->d,
                                         dt == MOE_BF16, wdt == MOE_BF16, stream));
}

size_t moe_layer_norm_backward_workspace_bytes(const moe_shape* s) {
  if (check_norm(s, MOE_F32, MOE_F32) != MOE_OK) return 0;
  return moe::layer_norm_backward_workspace_bytes(s->T, s->d);
}

moe_status moe_layer_norm_backward(const moe_shape* s, moe_dtype dt, const void* d_y, const void* sum, moe_dtype wdt,
                                   const void* weight, const float* mean, const float* rstd, const void* d_s,
                                   void* d_x, void* d_weight, void* d_bias, void* workspace, hipStream_t stream) {
  const moe_status st = check_norm(s, dt, wdt);
  if (st != MOE_OK) return st;
  if (weight == nullptr || d_weight == nullptr || d_weight == d_bias) return MOE_EINVAL;
  // with no rows only the (zero) parameter gradients are written
  if (s->T > 0 && (any_null(d_y, sum, static_cast<const void*>(d_x), static_cast<const void*>(workspace)) ||
                   mean == nullptr || rstd == nullptr))
    return MOE_EINVAL;
  if (!aligned16(d_y, sum, weight, d_s, static_cast<const void*>(d_x), static_cast<const void*>(d_weight),
                 static_cast<const void*>(d_bias), static_cast<const void*>(workspace)) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return MOE_EINVAL;
  return from_hip(moe::launch_layer_norm_backward(d_y, sum, weight, mean, rstd, d_s, d_x, d_weight, d_bias, workspace,
                                                  s->T, s->d, dt == MOE_BF16, wdt == MOE_BF16, stream));
}

moe_status moe_quantize_experts(const moe_shape* s, moe_dtype dt, const void* w_gate_up, const void* w_down,
                                void* q_gate_up, float* scale_gate_up, void* q_down, float* scale_down,
                                hipStream_t stream) {
  const moe_status st = check_experts(s);
  if (st != MOE_OK) return st;
  if (!valid_dtype(dt)) return MOE_EINVAL;
  if (any_null(w_gate_up, w_down, static_cast<const void*>(q_gate_up), static_cast<const void*>(q_down)) ||
      scale_gate_up == nullptr || scale_down == nullptr)
    return MOE_EINVAL;
  if (!aligned16(w_gate_up, w_down, static_cast<const void*>(q_gate_up), static_cast<const void*>(q_down)) ||
      !aligned(scale_gate_up, 4) || !aligned(scale_down, 4))
    return MOE_EINVAL;
  const int e_loc = s->e_end - s->e_begin;
  hipError_t e = moe::launch_quantize_weights(w_gate_up, q_gate_up, scale_gate_up, e_loc, s->d, 2 * s->d_ff,
                                              dt == MOE_BF16, stream);
  if (e == hipSuccess)
    e = moe::launch_quantize_weights(w_down, q_down, scale_down, e_loc, s->d_ff, s->d, dt == MOE_BF16, stream);
  return from_hip(e);
}

size_t moe_grouped_gemm_int8_workspace_bytes(const moe_shape* s) {
  if (check_int8(s) != MOE_OK) return 0;
  return Int8Workspace(s).bytes;
}

moe_status moe_grouped_gemm_int8(const moe_shape* s, moe_dtype dt, const void* x, const int32_t* perm,
                                 const int32_t* offsets, const void* q_gate_up, const float* scale_gate_up,
                                 const void* q_down, const float* scale_down, void* y, void* workspace,
                                 hipStream_t stream) {
  const moe_status st = check_int8(s);
  if (st != MOE_OK) return st;
  if (!valid_dtype(dt)) return MOE_EINVAL;
  if (dt != MOE_BF16) return MOE_EUNSUPPORTED;
  return run_int8(s, x, nullptr, perm, offsets, q_gate_up, scale_gate_up, q_down, scale_down, y, workspace, stream);
}

moe_status moe_grouped_gemm_int8_rows(const moe_shape* s, const void* q_x, const float* scale_x, const int32_t* perm,
                                      const int32_t* offsets, const void* q_gate_up, const float* scale_gate_up,
                                      const void* q_down, const float* scale_down, void* y, void* workspace,
                                      hipStream_t stream) {
  const moe_status st = check_int8(s);
  if (st != MOE_OK) return st;
  if (s->T > 0 && (scale_x == nullptr || !aligned(scale_x, 4))) return MOE_EINVAL;
  return run_int8(s, q_x, scale_x, perm, offsets, q_gate_up, scale_gate_up, q_down, scale_down, y, workspace, stream);
}

size_t moe_grad_norm_workspace_bytes(int32_t n) { return n < 0 ? 0 : moe::grad_norm_workspace_bytes(n); }

moe_status moe_grad_norm(const moe_tensor* grads, int32_t n, float* norm, void* workspace, hipStream_t stream) {
  const moe_status st = check_list(grads, n);
  if (st != MOE_OK) return st;
  if (norm == nullptr || workspace == nullptr || !aligned(norm, 4) || !aligned(workspace, 8)) return MOE_EINVAL;
  return from_hip(moe::launch_grad_norm(grads, n, norm, workspace, stream));
}

moe_status moe_clip_grads(const moe_tensor* grads, const moe_tensor* out, int32_t n, const float* norm, float max_norm,
                          hipStream_t stream) {
  if (norm == nullptr || !aligned(norm, 4)) return MOE_EINVAL;
  const moe_status st = check_clip(grads, out, n, max_norm, norm, false, nullptr, 0);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  return from_hip(moe::launch_clip_grads(grads, out != nullptr ? out : grads, n, norm, max_norm, stream));
}

moe_status moe_clip_grad_norm(const moe_tensor* grads, const moe_tensor* out, int32_t n, float max_norm, float* norm,
                              void* workspace, hipStream_t stream) {
  if (norm == nullptr || workspace == nullptr || !aligned(norm, 4) || !aligned(workspace, 8)) return MOE_EINVAL;
  const moe_status st =
      check_clip(grads, out, n, max_norm, norm, true, workspace, n < 0 ? 0 : moe::grad_norm_workspace_bytes(n));
  if (st != MOE_OK) return st;
  return from_hip(moe::launch_clip_grad_norm(grads, out != nullptr ? out : grads, n, max_norm, norm, workspace, stream));
}

}  // extern "C"
