// Routing to experts by scores: softmax or sigmoid, a bias for the choice, groups
// of experts, the k best, weights renormalised or not; and the weights' gradient.
//
//   s_e = softmax or sigmoid of the logits;  c_e = round32(s_e + b_e)
//   groups ranked by their largest c or the sum of their two largest, the first
//   top_groups stay;  idx = the k largest c of those;  w = scale * s[idx] (/ sum)
//
// Which experts a token gets hangs on the order of values that may be close, so c is
// computed in fp64 and rounded to fp32 once: two ways to compute it then agree but for
// a value within 2^-52 of the middle between two fp32 numbers. Equal c go to the
// lower id. Without a bias the scores rise with the logits, and these are compared.
#include <math.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / kWave;

// Unsigned integers that order like the values: 0 is left for an expert that is out, a NaN
// comes after every number.
__device__ __forceinline__ uint32_t orderable(float v) {
  if (!(v == v)) return 1u;
  const uint32_t u = __float_as_uint(v + 0.f);  // -0.0 ranks as +0.0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float from_orderable(uint32_t o) {
  if (o == 1u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ double sigmoid64(float x) { return 1.0 / (1.0 + exp(-static_cast<double>(x))); }

template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) {
    const T o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// LDS that only one wave uses: its accesses stay in order, so a wave waits for its own only.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct RouteArgs {
  const float* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int64_t T;
  int E, k, groups, top_groups, group_top;
  float scale;
  bool sigmoid, renormalize;
  bool by_score;  // the choice goes by c, not by the logits
};

RouteArgs make_args(const moe_router& r, const float* logits, int32_t* idx, float* w, int64_t T, int E, int k) {
  RouteArgs a;
  a.logits = logits;
  a.bias = r.bias;
  a.idx = idx;
  a.w = w;
  a.T = T;
  a.E = E;
  a.k = k;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.group_top = r.group_top;
  a.scale = r.scale;
  a.sigmoid = r.score == MOE_SIGMOID;
  a.renormalize = r.renormalize != 0;
  a.by_score = r.bias != nullptr || (r.groups > 1 && r.group_top == 2);
  return a;
}

// Any sizes: one wave per token, the choice values in LDS and, as keys (value, then lower
// id), in registers; k rounds of a maximum over the wave.
__global__ __launch_bounds__(kThreads) void route_any_kernel(const RouteArgs a) {
  constexpr int kPer = kMaxExperts / kWave;
  __shared__ uint32_t values[kWavesPerBlock][kMaxExperts];
  __shared__ uint32_t ranks[kWavesPerBlock][kMaxExperts];  // of the groups
  const int lane = lane_id(), wv = static_cast<int>(threadIdx.x) / kWave;
  uint32_t* c = values[wv];
  uint32_t* gv = ranks[wv];
  const int size = a.E / a.groups;
  // waves take tokens in turns; no barrier of the workgroup is among them
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wv; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWavesPerBlock) {
    const float* x = a.logits + t * a.E;
    // softmax over all experts, where the scores take part
    float top = 0.f;
    double total = 1.0;
    if (!a.sigmoid && (a.by_score || !a.renormalize)) {
      top = -INFINITY;
      for (int e = lane; e < a.E; e += kWave) top = x[e] > top ? x[e] : top;
      top = wave_max(top);
      total = 0.0;
      for (int e = lane; e < a.E; e += kWave) total += exp(static_cast<double>(x[e]) - top);
      total = wave_sum(total);
    }
    auto score = [&](float v) { return a.sigmoid ? sigmoid64(v) : exp(static_cast<double>(v) - top) / total; };
    for (int e = lane; e < a.E; e += kWave) {
      float v = x[e];
      if (a.by_score) v = static_cast<float>(score(v) + (a.bias != nullptr ? static_cast<double>(a.bias[e]) : 0.0));
      c[e] = orderable(v);
    }
    wave_sync();
    if (a.top_groups < a.groups) {
      for (int g = lane; g < a.groups; g += kWave) {
        uint32_t first = 0, second = 0;
        for (int i = g * size; i < (g + 1) * size; ++i) {
          const uint32_t v = c[i];
          second = v > first ? first : (v > second ? v : second);
          first = v > first ? v : first;
        }
        gv[g] = a.group_top == 2 && size > 1 ? orderable(from_orderable(first) + from_orderable(second)) : first;
      }
      wave_sync();
      for (int g = lane; g < a.groups; g += kWave) {
        const uint32_t mine = gv[g];
        int before = 0;
        for (int i = 0; i < a.groups; ++i) before += gv[i] > mine || (gv[i] == mine && i < g);
        if (before >= a.top_groups)
          for (int i = g * size; i < (g + 1) * size; ++i) c[i] = 0;
      }
      wave_sync();
    }
    uint64_t key[kPer];
  #pragma unroll
    for (int v = 0; v < kPer; ++v) {
      const int e = v * kWave + lane;
      const uint32_t o = e < a.E ? c[e] : 0;
      key[v] = o ? static_cast<uint64_t>(o) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(e)) : 0;
    }
    // the chosen ids, over the choice values
    wave_sync();
    for (int r = 0; r < a.k; ++r) {
      uint64_t best = key[0];
  #pragma unroll
      for (int v = 1; v < kPer; ++v) best = key[v] > best ? key[v] : best;
      best = wave_max(best);
  #pragma unroll
      for (int v = 0; v < kPer; ++v) key[v] = key[v] == best ? 0 : key[v];
      if (lane == 0) c[r] = 0xFFFFFFFFu - static_cast<uint32_t>(best);
    }
    wave_sync();
    double by = 1.0;
    if (a.renormalize) {
      if (!a.sigmoid) {  // softmax over the chosen
        top = -INFINITY;
        for (int j = lane; j < a.k; j += kWave) top = x[c[j]] > top ? x[c[j]] : top;
        top = wave_max(top);
        total = 1.0;
      }
      double sum = 0.0;
      for (int j = lane; j < a.k; j += kWave) sum += score(x[c[j]]);
      by = wave_sum(sum) + (a.sigmoid ? 1e-20 : 0.0);
    }
    for (int j = lane; j < a.k; j += kWave) {
      const int e = static_cast<int>(c[j]);
      a.idx[t * a.k + j] = e;
      a.w[t * a.k + j] = static_cast<float>(a.scale * (score(x[e]) / by));
    }
    wave_sync();  // the next token's values are written over these
  }
}

// The gradient. With u = scale * d_w, over the chosen j:
//   softmax, renormalised   q = softmax of the chosen logits:  q_j (u_j - sum u q)
//   softmax                 p_e ([e chosen] u_e - sum u p) for every expert
//   sigmoid, renormalised   S = sum s + 1e-20:  (u_j - sum u s / S) / S * s_j (1 - s_j)
//   sigmoid                 u_j s_j (1 - s_j)
// One wave per token, the row assembled in LDS and copied out.
__global__ __launch_bounds__(kThreads) void route_any_backward_kernel(const RouteArgs a, const float* __restrict__ d_w,
                                                                      float* __restrict__ d_logits) {
  __shared__ float rows[kWavesPerBlock][kMaxExperts];
  const int lane = lane_id(), wv = static_cast<int>(threadIdx.x) / kWave;
  float* row = rows[wv];
  const bool dense = !a.sigmoid && !a.renormalize;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wv; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWavesPerBlock) {
    const float* x = a.logits + t * a.E;
    const int32_t* idx = a.idx + t * a.k;
    const float* up = d_w + t * a.k;
    for (int e = lane; e < a.E; e += kWave) row[e] = 0.f;
    float top = -INFINITY, total = 0.f;
    if (dense) {
      for (int e = lane; e < a.E; e += kWave) top = fmaxf(top, x[e]);
      top = wave_max(top);
      for (int e = lane; e < a.E; e += kWave) total += expf(x[e] - top);
      total = wave_sum(total);
    } else if (!a.sigmoid) {
      for (int j = lane; j < a.k; j += kWave)
        if (static_cast<uint32_t>(idx[j]) < static_cast<uint32_t>(a.E)) top = fmaxf(top, x[idx[j]]);
      top = wave_max(top);
    }
    auto score = [&](float v) { return a.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top); };
    float sum = 0.f, dot = 0.f;
    for (int j = lane; j < a.k; j += kWave) {
      if (static_cast<uint32_t>(idx[j]) >= static_cast<uint32_t>(a.E)) continue;
      const float s = score(x[idx[j]]);
      sum += s;
      dot = fmaf(a.scale * up[j], s, dot);
    }
    sum = wave_sum(sum);
    dot = wave_sum(dot);
    const float by = dense ? total : a.sigmoid ? sum + 1e-20f : sum;
    wave_sync();
    for (int j = lane; j < a.k; j += kWave) {
      const int e = idx[j];
      if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.E)) continue;
      const float v = x[e], u = a.scale * up[j], s = score(v);
      if (dense) row[e] = u;
      else if (!a.sigmoid) row[e] = s / by * (u - dot / by);
      else row[e] = (a.renormalize ? (u - dot / by) / by : u) * s / (1.f + expf(v));
    }
    wave_sync();
    for (int e = lane; e < a.E; e += kWave)
      d_logits[t * a.E + e] = dense ? score(x[e]) / by * (row[e] - dot / by) : row[e];
    wave_sync();
  }
}

// a launch holds fewer than 2^32 threads; tokens past these take turns
unsigned wave_blocks(int64_t T) {
  return static_cast<unsigned>(min((T + kWavesPerBlock - 1) / kWavesPerBlock, int64_t{1} << 20));
}

}  // namespace

hipError_t launch_route_experts(const moe_router& r, const float* logits, int32_t* idx, float* w, int64_t T, int E,
                                int k, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteArgs a = make_args(r, logits, idx, w, T, E, k);
  hipLaunchKernelGGL(route_any_kernel, dim3(wave_blocks(T)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_route_experts_backward(const moe_router& r, const float* logits, const int32_t* idx,
                                         const float* d_w, float* d_logits, int64_t T, int E, int k,
                                         hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouteArgs a = make_args(r, logits, const_cast<int32_t*>(idx), nullptr, T, E, k);
  hipLaunchKernelGGL(route_any_backward_kernel, dim3(wave_blocks(T)), dim3(kThreads), 0, stream, a, d_w, d_logits);
  return hipGetLastError();
}

}  // namespace moe
