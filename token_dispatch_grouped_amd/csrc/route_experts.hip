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
constexpr int64_t kFewLanes = 2 * 1024 * kWave;
constexpr int kTop = 16;  // chosen experts that are kept in registers

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

// e^x in fp64, to about 2^-52: x = n ln 2 + r with |r| <= ln 2 / 2, and e^r by its power series
// (the term r^13 / 13! is below 2^-52). x is held to +-700, so that 1 + e^x and its inverse are
// finite; a NaN stays one. 24 instructions, where a library's, made for any argument, and its division took half
// of the kernel's time (16384 x 256 sigmoids: 22 us against 15).
__device__ __forceinline__ double exp64(double x) {
  const double y = fmin(fmax(x, -700.0), 700.0);
  const double n = rint(y * 1.4426950408889634);
  const double r = fma(n, -0.6931471805599453, y);
  // coefficients from scalar registers: as part of the fused operation, not moved to its result first
  auto scalar = [](double c) {
    asm("" : "+s"(c));
    return c;
  };
  double p = fma(scalar(1.0 / 479001600), r, scalar(1.0 / 39916800));
  p = fma(p, r, scalar(1.0 / 3628800));
  p = fma(p, r, scalar(1.0 / 362880));
  p = fma(p, r, scalar(1.0 / 40320));
  p = fma(p, r, scalar(1.0 / 5040));
  p = fma(p, r, scalar(1.0 / 720));
  p = fma(p, r, scalar(1.0 / 120));
  p = fma(p, r, scalar(1.0 / 24));
  p = fma(p, r, scalar(1.0 / 6));
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  const double e = __builtin_ldexp(p, static_cast<int>(n));
  return x == x ? e : x;
}

// 1 / d for finite d >= 1: two Newton steps from the instruction's 2^-24 or so.
__device__ __forceinline__ double inverse64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(fma(-d, y, 1.0), y, y);
  return fma(fma(-d, y, 1.0), y, y);
}

__device__ __forceinline__ double sigmoid64(float x) { return inverse64(1.0 + exp64(-static_cast<double>(x))); }

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

// Any sizes (more than kTop experts a token, more than 64 groups): one wave per token, the choice values in LDS and, as keys (value, then lower
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
      for (int e = lane; e < a.E; e += kWave) total += exp64(static_cast<double>(x[e]) - top);
      total = wave_sum(total);
    }
    auto score = [&](float v) { return a.sigmoid ? sigmoid64(v) : exp64(static_cast<double>(v) - top) / total; };
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

// Up to kTop experts of at most 64 lanes' values: G lanes (a power of two) share a token, each
// with VPL values in registers; the values are never in LDS and every step but the last
// runs on all lanes.
//   - A value (32 orderable bits) and its id make one key, the mantissa of a double in
//     [1, 2): the larger double is the larger value, then the lower id, and v_max_f64 and
//     v_min_f64 order two keys in two instructions. 1.0 is an expert that is out.
//   - A lane sorts its VPL keys (networks of such pairs) and keeps the largest L; groups are
//     ranked by their lanes' first two keys; then log2 G steps merge the lists of two lanes: the
//     larger of a[i] and b[L - 1 - i] are the L largest of both, in a bitonic order that
//     log2 L more steps sort. Both lanes get the same list.
//   - Lanes 0..k-1 then take one chosen expert each for the weights, in fp64.
// A group lies in P = G / (groups, rounded up to a power of two) consecutive lanes.
__device__ __forceinline__ double key_of(uint32_t ord, int e) {
  const uint32_t hi = 0x3FF00000u | (ord >> 12), lo = (ord << 20) | static_cast<uint32_t>(kMaxExperts - 1 - e);
  return __hiloint2double(static_cast<int>(hi), static_cast<int>(lo));
}
__device__ __forceinline__ uint32_t key_ord(double k) {
  return static_cast<uint32_t>(__double2hiint(k)) << 12 | static_cast<uint32_t>(__double2loint(k)) >> 20;
}
__device__ __forceinline__ int key_id(double k) { return kMaxExperts - 1 - (__double2loint(k) & (kMaxExperts - 1)); }

__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return __builtin_fmin(a, b); }

// The pair (a[i], a[j]) in descending order.
template <int N>
__device__ __forceinline__ void order(double (&a)[N], int i, int j) {
  const double hi = larger(a[i], a[j]), lo = smaller(a[i], a[j]);
  a[i] = hi;
  a[j] = lo;
}

// A bitonic list in descending order.
template <int N>
__device__ __forceinline__ void sort_bitonic(double (&a)[N]) {
#pragma unroll
  for (int stride = N / 2; stride > 0; stride >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & stride) == 0) order(a, i, i + stride);
}

// Any list in descending order: Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_any(double (&a)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k > 0; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(a, i + j, i + j + k);
}

// a := the N largest of two descending lists, descending.
template <int N>
__device__ __forceinline__ void merge(double (&a)[N], const double (&b)[N]) {
  double m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = larger(a[i], b[N - 1 - i]);
  sort_bitonic(m);
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = m[i];
}

// The value of the lane that differs in the bit OFF of its number, where all lanes of a
// smaller block hold the same (the mirrors reach another lane of the same block).
template <int OFF>
__device__ __forceinline__ uint32_t from_partner(uint32_t v) {
  const int i = static_cast<int>(v);
  if constexpr (OFF == 1) return __builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, false);        // quad_perm [1,0,3,2]
  else if constexpr (OFF == 2) return __builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, false);   // quad_perm [2,3,0,1]
  else if constexpr (OFF == 4) return __builtin_amdgcn_update_dpp(0, i, 0x141, 0xF, 0xF, false);  // row_half_mirror
  else if constexpr (OFF == 8) return __builtin_amdgcn_update_dpp(0, i, 0x140, 0xF, 0xF, false);  // row_mirror
  else return __shfl_xor(v, OFF);
}
template <int OFF>
__device__ __forceinline__ double from_partner(double v) {
  return __hiloint2double(static_cast<int>(from_partner<OFF>(static_cast<uint32_t>(__double2hiint(v)))),
                          static_cast<int>(from_partner<OFF>(static_cast<uint32_t>(__double2loint(v)))));
}

template <int G, int OFF = 1, typename T>
__device__ __forceinline__ T group_sum(T v) {
  if constexpr (OFF < G) return group_sum<G, 2 * OFF>(v + __shfl_xor(v, OFF));
  return v;
}
template <int G, int OFF = 1>
__device__ __forceinline__ float group_top(float v) {
  if constexpr (OFF < G) {
    const float o = __shfl_xor(v, OFF);
    return group_top<G, 2 * OFF>(o > v ? o : v);
  }
  return v;
}

template <int G, int L, int OFF = 1>
__device__ __forceinline__ void merge_lanes(double (&a)[L]) {
  if constexpr (OFF < G) {
    double b[L];
#pragma unroll
    for (int i = 0; i < L; ++i) b[i] = from_partner<OFF>(a[i]);
    merge(a, b);
    merge_lanes<G, L, 2 * OFF>(a);
  }
}

// The two largest of the P lanes of a group, to all of them.
template <int G, int OFF = 1>
__device__ __forceinline__ void merge_two(uint32_t& first, uint32_t& second, int P) {
  if constexpr (OFF < G) {
    const uint32_t f = from_partner<OFF>(first), s = from_partner<OFF>(second);
    if (OFF < P) {
      const uint32_t rest = min(first, f);
      first = max(first, f);
      second = max(rest, max(second, s));
    }
    merge_two<G, 2 * OFF>(first, second, P);
  }
}

// What a kernel does with all of a token's logits: sort them; add up their exponentials, which the
// weights of the chosen ones need; or turn each into its score.
enum class Route { kLogits, kLogitsTotal, kSigmoid, kSoftmax };

template <int G, int VPL, int L, Route MODE>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a, int P, int per) {
  constexpr int kTokens = kWave / G;   // of a wave
  constexpr int kSlots = (L + G - 1) / G;
  constexpr int kRun = VPL < L ? VPL : L;
  constexpr float kLog2e = 1.44269504f;
  constexpr bool kScores = MODE == Route::kSigmoid || MODE == Route::kSoftmax;
  const int lane = lane_id(), g = lane % G;
  const int size = a.E / a.groups, group = g / P, first = g % P * per;  // of this lane, in its group
  const int own = group < a.groups ? min(per, size - first) : 0;        // experts of this lane (may be < 0)
  const int e0 = group * size + first;
  const bool fours = (size | per) % 4 == 0;  // no four of a lane lie across the end of the buffer
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + uniform(static_cast<int>(threadIdx.x) / kWave);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWavesPerBlock * kTokens;
  for (int64_t t0 = wave * kTokens; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / G;
    const bool live = t < a.T;
    // The wave's rows as one buffer: a lane reads VPL values from its first expert on, whoever's they are (0 past
    // the last token), and uses its own.
    const __amdgpu_buffer_rsrc_t rows = make_rsrc(
        a.logits + t0 * a.E, static_cast<uint32_t>(min(a.T - t0, static_cast<int64_t>(kTokens)) * a.E * 4));
    const uint32_t row = static_cast<uint32_t>(lane / G * a.E) * 4u;
    float v[VPL], bias[kScores ? VPL : 1];
    auto load = [&](__amdgpu_buffer_rsrc_t from, uint32_t at, float* to) {
      if (fours) {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
          const uint4 q = buffer_load16(from, at + i * 4u);
          to[i] = __uint_as_float(q.x);
          to[i + 1] = __uint_as_float(q.y);
          to[i + 2] = __uint_as_float(q.z);
          to[i + 3] = __uint_as_float(q.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          to[i] = __uint_as_float(static_cast<uint32_t>(
              __builtin_amdgcn_raw_buffer_load_b32(from, static_cast<int>(at + i * 4u), 0, 0)));
      }
    };
    load(rows, row + e0 * 4u, v);
    if constexpr (kScores)  // no bias: a buffer of no bytes, all zeros
      load(make_rsrc(a.bias, a.bias != nullptr ? static_cast<uint32_t>(a.E) * 4u : 0u), e0 * 4u, bias);
    float top = 0.f;
    double total = 1.0;  // its inverse for kSoftmax
    if constexpr (MODE == Route::kLogitsTotal || MODE == Route::kSoftmax) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) top = i < own && v[i] > top ? v[i] : top;
      top = group_top<G>(top);
      if constexpr (MODE == Route::kSoftmax) {
        total = 0.0;
#pragma unroll 4
        for (int i = 0; i < VPL; ++i) total += i < own ? exp64(static_cast<double>(v[i]) - top) : 0.0;
        total = inverse64(group_sum<G>(total));
      } else {  // fp32 is enough for the weights
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += i < own ? __builtin_amdgcn_exp2f((v[i] - top) * kLog2e) : 0.f;
        total = group_sum<G>(sum);
      }
    }
    double best[L];
#pragma unroll
    for (int i = kRun; i < L; ++i) best[i] = 1.0;
    // runs of L values, each sorted alone, then the L largest of it and those before
#pragma unroll
    for (int r = 0; r < VPL; r += kRun) {
      __builtin_amdgcn_sched_barrier(0);  // one run's scores at a time: all at once take 300 registers
      double run[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        float c = v[r + i];
        if constexpr (kScores) {
          const double s = MODE == Route::kSigmoid ? sigmoid64(c) : exp64(static_cast<double>(c) - top) * total;
          c = static_cast<float>(s + static_cast<double>(bias[r + i]));
        }
        run[i] = r + i < own ? key_of(orderable(c), e0 + r + i) : 1.0;
      }
      sort_any(run);
      if constexpr (VPL > L) {
        if (r > 0) merge(best, run);
        else
#pragma unroll
          for (int i = 0; i < L; ++i) best[i] = run[i];
      } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i) best[i] = run[i];
      }
    }
    if (a.top_groups < a.groups) {
      uint32_t one = key_ord(best[0]), two = L > 1 ? key_ord(best[1]) : 0;
      merge_two<G>(one, two, P);
      const uint32_t mine = a.group_top == 2 && size > 1 ? orderable(from_orderable(one) + from_orderable(two)) : one;
      int before = 0;
      for (int i = 0; i < a.groups; ++i) {
        const uint32_t other = __shfl(mine, lane - g + i * P);
        before += other > mine || (other == mine && i < group);
      }
      if (before >= a.top_groups)
#pragma unroll
        for (int i = 0; i < L; ++i) best[i] = 1.0;
    }
    merge_lanes<G>(best);
    // chosen expert s * G + g to lane g
    int id[kSlots];
    float z[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      double mine = best[s * G < L ? s * G : 0];
#pragma unroll
      for (int i = 1; i < G; ++i)
        if (s * G + i < L) mine = g == i ? best[s * G + i] : mine;
      const int j = s * G + g;
      id[s] = key_id(mine);
      const int bits = __builtin_amdgcn_raw_buffer_load_b32(rows, static_cast<int>(row + id[s] * 4u), 0, 0);
      z[s] = live && j < a.k ? __uint_as_float(static_cast<uint32_t>(bits)) : -INFINITY;
    }
    double w[kSlots], sum = 0.0;
    if (!a.sigmoid && a.renormalize) {  // softmax over the chosen
      top = z[0];
#pragma unroll
      for (int s = 1; s < kSlots; ++s) top = z[s] > top ? z[s] : top;
      top = group_top<G>(top);
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      w[s] = a.sigmoid ? sigmoid64(z[s]) : exp64(static_cast<double>(z[s]) - top);
      sum += s * G + g < a.k ? w[s] : 0.0;
    }
    if (a.renormalize) sum = group_sum<G>(sum) + (a.sigmoid ? 1e-20 : 0.0);
    else sum = MODE == Route::kLogitsTotal ? total : MODE == Route::kSoftmax ? 1.0 / total : 1.0;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int j = s * G + g;
      if (live && j < a.k) {
        a.idx[t * a.k + j] = id[s];
        a.w[t * a.k + j] = static_cast<float>(a.scale * (w[s] / sum));
      }
    }
  }
}

template <int G, int VPL, int L, Route MODE>
hipError_t launch_route(const RouteArgs& a, int P, int per, hipStream_t stream) {
  const int64_t tokens = kWavesPerBlock * (kWave / G);
  const int64_t blocks = min((a.T + tokens - 1) / tokens, int64_t{1} << 20);
  hipLaunchKernelGGL((route_kernel<G, VPL, L, MODE>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a,
                     P, per);
  return hipGetLastError();
}

template <int G, int VPL, int L>
hipError_t launch_route_mode(const RouteArgs& a, int P, int per, hipStream_t stream) {
  if (a.by_score && a.sigmoid) return launch_route<G, VPL, L, Route::kSigmoid>(a, P, per, stream);
  if (a.by_score) return launch_route<G, VPL, L, Route::kSoftmax>(a, P, per, stream);
  if (!a.sigmoid && !a.renormalize) return launch_route<G, VPL, L, Route::kLogitsTotal>(a, P, per, stream);
  return launch_route<G, VPL, L, Route::kLogits>(a, P, per, stream);
}

template <int G, int VPL>
hipError_t launch_route_top(const RouteArgs& a, int P, int per, hipStream_t stream) {
  if (a.k <= 4) return launch_route_mode<G, VPL, 4>(a, P, per, stream);
  if (a.k <= 8) return launch_route_mode<G, VPL, 8>(a, P, per, stream);
  return launch_route_mode<G, VPL, 16>(a, P, per, stream);
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
  if (k <= kTop) {
    int blocks = 1;  // groups rounded up to a power of two
    while (blocks < r.groups) blocks *= 2;
    const int size = E / r.groups;
#define MOE_ROUTE(LANES, VALUES)                                                                              \
  if (T * LANES >= least && blocks <= LANES && (size + LANES / blocks - 1) / (LANES / blocks) <= VALUES)      \
    return launch_route_top<LANES, VALUES>(a, LANES / blocks, (size + LANES / blocks - 1) / (LANES / blocks), stream)
    for (const int64_t least : {kFewLanes, int64_t{0}}) {
      MOE_ROUTE(1, 8);
      MOE_ROUTE(2, 8);
      MOE_ROUTE(4, 8);
      if (least > 0) {
        MOE_ROUTE(4, 16);
        MOE_ROUTE(4, 32);
      }
      MOE_ROUTE(8, 8);
      if (least > 0) {
        MOE_ROUTE(8, 16);
        MOE_ROUTE(8, 32);
      }
      MOE_ROUTE(16, 8);
      MOE_ROUTE(16, 16);
      if (least > 0) MOE_ROUTE(16, 32);
      MOE_ROUTE(32, 16);
      if (least > 0) MOE_ROUTE(32, 32);
      MOE_ROUTE(64, 16);
    }
#undef MOE_ROUTE
  }
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
