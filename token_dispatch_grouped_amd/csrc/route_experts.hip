// Routing to experts by scores: softmax or sigmoid, a bias for the choice, groups
// of experts, the k best, weights renormalised or not; and the weights' gradient.
//
//   s_e = softmax or sigmoid of the logits;  c_e = round32(s_e + b_e)
//   groups ranked by their largest c or the sum of their two largest, the first
//   top_groups stay;  idx = the k largest c of those;  w = scale * s[idx] (/ sum)
//
// Which experts a token gets hangs on the order of values that may be close, so c is
// computed in fp64 and rounded to fp32 once: two ways to compute it then agree but for
// a value within 2^-50 (of itself) of the middle between two fp32 numbers. Equal c go to the
// lower id. Without a bias the scores rise with the logits, and these are compared.
// A logit of -infinity masks its expert: c is -infinity then, whatever the bias.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / kWave;
// Lanes of a token. A call of few tokens takes as many as hold 8 values each (16 from 16 lanes on): short chains.
// Fewer lanes with more values are less work in all, and taken where the tokens fill the chip's 1024 SIMDs with two waves
// each all the same. us of 8 experts a token by the first rule and by the second (logits; sigmoids with a bias; softmax
// scores with one):
//   128 experts, 1000 tokens 3.8 4.9 6.6 and 5.8 11.2 13.7; 16384 6.5 9.1 11.9 and 5.1 6.9 11.2; 65536 18.2 28.3 35.8 and 11.7 28.0 33.0
//   512, 1000 tokens 4.9 6.4 9.5 and 6.2 8.1 10.5; 8192 8.7 12.3 20.4 and 7.7 10.4 14.7; 65536 48 75 133 and 37 54 71
constexpr int64_t kFewLanes = 2 * 1024 * kWave;
constexpr int kTop = 16;  // chosen experts that are kept in registers

// Unsigned integers that order like the values: 0 is left for an expert that is out, a NaN
// comes after every number.
__device__ __forceinline__ uint32_t orderable(float v) {
  if (!(v == v)) return 1u;
  const uint32_t u = __float_as_uint(v + 0.f);  // -0.0 ranks as +0.0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr uint32_t kMinusInfinity = 0x007FFFFFu;  // orderable(-INFINITY)

__device__ __forceinline__ float from_orderable(uint32_t o) {
  if (o == 1u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// e^x in fp64, to 2^-51: x = n ln 2 + r with |r| <= ln 2 / 2, and e^r by its power series
// (the term r^13 / 13! is below 2^-52). x is held to +-700, so that 1 + e^x and its inverse are
// finite; a NaN stays one. A few instructions fewer than the library's, made for any argument, and its
// division (131072 x 256 softmax scores, all in fp64: 105 us against 111).
__device__ __forceinline__ double exp64(double x) {
  const double y = fmin(fmax(x, -700.0), 700.0);
  const double n = rint(y * 1.4426950408889634);
  double r = fma(n, -0.6931471805599453, y);
  // coefficients from scalar registers: as part of the fused operation, not moved to its result first
  auto scalar = [](double c) {
    asm("" : "+s"(c));
    return c;
  };
  r = fma(n, scalar(-2.3190468138462996e-17), r);  // one double of ln 2 is off by 12 * 2^-52 for |x| of 80
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

// The bias, or the choice value, of a logit x: a masked expert's is -infinity (a NaN stays one, and comes later still).
__device__ __forceinline__ float masked(float x, float v) { return x == -INFINITY && v == v ? -INFINITY : v; }

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
// id), in registers; k rounds of a maximum over the wave, each waiting for the one before (16384 tokens, 17, 24 and 32 of
// 256: 82, 105 and 133 us).
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
      if (a.by_score)
        v = static_cast<float>(score(v) + static_cast<double>(masked(v, a.bias != nullptr ? a.bias[e] : 0.f)));
      c[e] = orderable(v);
    }
    wave_sync();
    if (a.top_groups < a.groups) {
      bool minus = false;  // a sum of -infinity
      for (int g = lane; g < a.groups; g += kWave) {
        uint32_t first = 0, second = 0;
        for (int i = g * size; i < (g + 1) * size; ++i) {
          const uint32_t v = c[i];
          second = v > first ? first : (v > second ? v : second);
          first = v > first ? v : first;
        }
        gv[g] = a.group_top == 2 && size > 1 ? orderable(from_orderable(first) + from_orderable(second)) : first;
        minus = minus || gv[g] == kMinusInfinity;
      }
      minus = __any(minus);
      wave_sync();
      auto largest = [&](int g) {
        uint32_t top = 0;
        for (int i = g * size; i < (g + 1) * size; ++i) top = c[i] > top ? c[i] : top;
        return top;
      };
      uint32_t leaves = 0;  // of this lane's groups
      for (int g = lane, n = 0; g < a.groups; g += kWave, ++n) {
        const uint32_t mine = gv[g];
        int before = 0;
        if (!minus)
          for (int i = 0; i < a.groups; ++i) before += gv[i] > mine || (gv[i] == mine && i < g);
        else {
          const uint32_t top = mine == kMinusInfinity ? largest(g) : 0;
          for (int i = 0; i < a.groups; ++i) {
            const uint32_t other = gv[i] == mine && mine == kMinusInfinity ? largest(i) : top;
            before += gv[i] > mine || (gv[i] == mine && (other > top || (other == top && i < g)));
          }
        }
        leaves |= static_cast<uint32_t>(before >= a.top_groups) << n;
      }
      wave_sync();
      for (int g = lane, n = 0; g < a.groups; g += kWave, ++n)
        if (leaves >> n & 1)
          for (int i = g * size; i < (g + 1) * size; ++i) c[i] = 0;
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
__device__ __forceinline__ int larger(int a, int b) { return max(a, b); }
__device__ __forceinline__ int smaller(int a, int b) { return min(a, b); }

// The pair (a[i], a[j]) in descending order.
template <typename T, int N>
__device__ __forceinline__ void order(T (&a)[N], int i, int j) {
  const T hi = larger(a[i], a[j]), lo = smaller(a[i], a[j]);
  a[i] = hi;
  a[j] = lo;
}

// A bitonic list in descending order.
template <typename T, int N>
__device__ __forceinline__ void sort_bitonic(T (&a)[N]) {
#pragma unroll
  for (int stride = N / 2; stride > 0; stride >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & stride) == 0) order(a, i, i + stride);
}

// Any list in descending order: Batcher's odd-even merge sort.
template <typename T, int N>
__device__ __forceinline__ void sort_any(T (&a)[N]) {
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
template <typename T, int N>
__device__ __forceinline__ void merge(T (&a)[N], const T (&b)[N]) {
  T m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = larger(a[i], b[N - 1 - i]);
  sort_bitonic(m);
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = m[i];
}

// The value of the lane that differs in the bit OFF of its number, where all lanes of a
// smaller block hold the same (the mirrors reach another lane of the same block).
template <int OFF>
__device__ __forceinline__ int from_partner(int v) {
  if constexpr (OFF == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);        // quad_perm [1,0,3,2]
  else if constexpr (OFF == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // quad_perm [2,3,0,1]
  else if constexpr (OFF == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // row_half_mirror
  else if constexpr (OFF == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // row_mirror
  else return __shfl_xor(v, OFF);
}
template <int OFF>
__device__ __forceinline__ uint32_t from_partner(uint32_t v) {
  return static_cast<uint32_t>(from_partner<OFF>(static_cast<int>(v)));
}
template <int OFF>
__device__ __forceinline__ double from_partner(double v) {
  return __hiloint2double(from_partner<OFF>(__double2hiint(v)), from_partner<OFF>(__double2loint(v)));
}

// The value of the lane whose number differs in the bits of M.
template <int M>
__device__ __forceinline__ int xor_lane(int v) {
  if constexpr (M == 0) return v;
  else if constexpr (M == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  else if constexpr (M == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  else if constexpr (M == 3) return __builtin_amdgcn_mov_dpp(v, 0x1B, 0xF, 0xF, true);  // quad_perm [3,2,1,0]
  else if constexpr (M < 8) return xor_lane<7 ^ M>(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));
  else if constexpr (M < 16) return xor_lane<15 ^ M>(__builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));
  else return __shfl_xor(v, M);
}

// Calls f(value, group) for every other lane of the token's G.
template <int G, int M = 1, typename F>
__device__ __forceinline__ void other_lanes(int v, int g, int log_p, F&& f) {
  if constexpr (M < G) {
    f(xor_lane<M>(v), (g ^ M) >> log_p);
    other_lanes<G, M + 1>(v, g, log_p, f);
  }
}

// Lanes of the groups before this one, by their values `mine`, those of -infinity (SUMS of two) by their largest,
// `top`; then the lower group. OFTEN: where nearly every wave asks, and hardly any has a sum of -infinity.
template <int G, bool SUMS, bool OFTEN>
__device__ __forceinline__ int lanes_before(uint32_t mine, uint32_t top, int g, int log_p) {
  const int group = g >> log_p;
  int before = 0;
  if (SUMS && (!OFTEN || __any(mine == kMinusInfinity))) {
    top = mine == kMinusInfinity ? top : 0;
#pragma unroll 1
    for (int m = 1; m < G; ++m) {
      const uint32_t other = __shfl_xor(mine, m), its_top = __shfl_xor(top, m);
      before += other > mine || (other == mine && (its_top > top || (its_top == top && (g ^ m) >> log_p < group)));
    }
  } else {
    other_lanes<G>(static_cast<int>(mine), g, log_p, [&](int value, int of) {
      const uint32_t other = static_cast<uint32_t>(value);
      before += other > mine || (other == mine && of < group);
    });
  }
  return before;
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

template <int G, int OFF = 1, typename T, int L>
__device__ __forceinline__ void merge_lanes(T (&a)[L]) {
  if constexpr (OFF < G) {
    T b[L];
#pragma unroll
    for (int i = 0; i < L; ++i) b[i] = from_partner<OFF>(a[i]);
    merge(a, b);
    merge_lanes<G, 2 * OFF>(a);
  }
}

// The two largest of the P lanes of a group, to all of them.
template <int G, int OFF = 1, typename T>
__device__ __forceinline__ void merge_two(T& first, T& second, int P) {
  if constexpr (OFF < G) {
    const T f = from_partner<OFF>(first), s = from_partner<OFF>(second);
    if (OFF < P) {
      const T rest = min(first, f);
      first = max(first, f);
      second = max(rest, max(second, s));
    }
    merge_two<G, 2 * OFF>(first, second, P);
  }
}

// What a kernel does with all of a token's logits: sort them; add up their exponentials, which the
// weights of the chosen ones need; or turn each into its score.
enum class Route { kLogits, kLogitsTotal, kSigmoid, kSoftmax };

// The tokens of a wave: their rows as one buffer, from which a lane reads VPL values from its first
// expert on, whoever's they are (0 past the last token), and uses its own.
template <int G, int VPL>
struct Rows {
  static constexpr int kTokens = kWave / G;  // of a wave
  __amdgpu_buffer_rsrc_t buffer;
  uint32_t row;      // of this lane's token, in bytes
  int64_t t;
  bool live, fours;  // fours: no four values of a lane lie across the end of the buffer
  int g, group, own, e0;

  __device__ Rows(const RouteArgs& a, int P, int per, int64_t t0) {
    const int lane = lane_id(), size = a.E / a.groups;
    g = lane % G;
    group = g / P;
    const int first = g % P * per;                                // of this lane, in its group
    own = group < a.groups ? max(min(per, size - first), 0) : 0;  // experts of this lane
    e0 = group * size + first;
    fours = (size | per) % 4 == 0;
    t = t0 + lane / G;
    live = t < a.T;
    row = static_cast<uint32_t>(lane / G * a.E) * 4u;
    buffer = make_rsrc(a.logits + t0 * a.E,
                       static_cast<uint32_t>(min(a.T - t0, static_cast<int64_t>(kTokens)) * a.E * 4));
  }
  __device__ void load(__amdgpu_buffer_rsrc_t from, uint32_t at, float (&to)[VPL]) const {
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
      for (int i = 0; i < VPL; ++i) to[i] = one(from, at + i * 4u);
    }
  }
  __device__ static float one(__amdgpu_buffer_rsrc_t from, uint32_t at) {
    return __uint_as_float(
        static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b32(from, static_cast<int>(at), 0, 0)));
  }
  __device__ void logits(float (&v)[VPL]) const { load(buffer, row + e0 * 4u, v); }
  __device__ float logit(int e) const { return one(buffer, row + e * 4u); }
  // no bias: a buffer of no bytes, all zeros
  __device__ static __amdgpu_buffer_rsrc_t bias_buffer(const RouteArgs& a) {
    return make_rsrc(a.bias, a.bias != nullptr ? static_cast<uint32_t>(a.E) * 4u : 0u);
  }
};

// Whether the wave has a masked expert among its lanes' logits. Most have none and only look for the least, two values an
// instruction (a comparison and a choice for each value: 1000 x 256 softmax scores 8.6 us instead of 8.0).
template <int N>
__device__ __forceinline__ bool any_masked(const float (&logit)[N]) {
  float least = INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) least = fminf(least, logit[i]);
  return __any(least == -INFINITY);
}

// Where a wave keeps its tokens' candidates.
template <int G, int L>
struct Candidates {
  static constexpr int kMost = G < 2 * L ? 2 * L : G;  // of a token
  double key[kWave / G][kMost];
  float logit[kWave / G][kMost], bias[kWave / G][kMost];  // softmax scores only
  uint16_t id[kWave / G][kMost];
};

// The wave's tokens, with every score in fp64. BEHIND the search below: for few waves.
template <int G, int VPL, int L, Route MODE, bool BEHIND>
__device__ __forceinline__ void route_exact(const RouteArgs& a, const Rows<G, VPL>& in, int P) {
  constexpr int kSlots = (L + G - 1) / G;
  constexpr int kRun = VPL < L ? VPL : L;
  constexpr float kLog2e = 1.44269504f;
  constexpr bool kScores = MODE == Route::kSigmoid || MODE == Route::kSoftmax;
  const int lane = lane_id(), g = in.g, own = in.own, e0 = in.e0, group = in.group, size = a.E / a.groups;
  const bool live = in.live;
  const int64_t t = in.t;
  float v[VPL], bias[kScores ? VPL : 1];
  in.logits(v);
  if constexpr (kScores) in.load(in.bias_buffer(a), e0 * 4u, bias);
  const bool masks = kScores && any_masked(v);
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
    float c[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      c[i] = v[r + i];
      if constexpr (kScores) {
        const double s = MODE == Route::kSigmoid ? sigmoid64(c[i]) : exp64(static_cast<double>(c[i]) - top) * total;
        c[i] = static_cast<float>(s + static_cast<double>(bias[r + i]));
      }
    }
    if (masks) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) c[i] = masked(v[r + i], c[i]);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) run[i] = r + i < own ? key_of(orderable(c[i]), e0 + r + i) : 1.0;
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
    if (lanes_before<G, kScores, !BEHIND>(mine, one, g, __ffs(P) - 1) >= a.top_groups * P)
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
    const float x = in.logit(id[s]);
    z[s] = live && j < a.k ? x : -INFINITY;
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

// Signed integers that order like the values (of which none is -0.0); a NaN is above all or below all.
__device__ __forceinline__ int signed_order(float v) {
  const int b = static_cast<int>(__float_as_uint(v));
  return b ^ static_cast<int>(static_cast<uint32_t>(b >> 31) >> 1);
}
__device__ __forceinline__ float from_signed(int o) {
  return __uint_as_float(static_cast<uint32_t>(o ^ static_cast<int>(static_cast<uint32_t>(o >> 31) >> 1)));
}

// Scores on fp32 values alone, 32 bits a comparison: the k-th largest of a token's values is found (not
// whose it is), every expert from it on (less the values' error) becomes a candidate in LDS, and
// the candidates, hardly ever more than k, are ranked by their exact choice values. Softmax scores are
// ranked by the fp32 values where no two are close, as their exact ones take the fp64 sum
// over all experts. Groups that are too close to each other for fp32 are ranked by the exact values of
// their lanes' best two. False where that does not decide: a NaN, a bias above 1e38, or more candidates than
// there is room for (many equal values).
template <int G, int VPL, int L, Route MODE>
__device__ __forceinline__ bool route_quick(const RouteArgs& a, const Rows<G, VPL>& in, int P,
                                            Candidates<G, L>& room) {
  static_assert(G >= 8 && G <= 32, "a lane has room for all of a token's candidates otherwise");
  constexpr int kSlots = Candidates<G, L>::kMost / G;
  constexpr int kRun = VPL < L ? VPL : L;
  constexpr float kLog2e = 1.44269504f;
  constexpr bool kSoftmax = MODE == Route::kSoftmax;
  const int lane = lane_id(), g = in.g, token = lane / G, size = a.E / a.groups;
  int own = in.own;
  float v[VPL], bias[VPL], top = 0.f, inv = 0.f;
  double inv64 = 0.0;  // softmax: of the exact sum, once a wave has needed it
  in.logits(v);
  in.load(in.bias_buffer(a), in.e0 * 4u, bias);
  if (any_masked(v)) {
    // masked() in fewer registers: a NaN or a number near the largest becomes one that is, which leads to route_exact
#pragma unroll
    for (int i = 0; i < VPL; ++i) bias[i] = fminf(bias[i], fmaf(v[i], 0x1p-30f, FLT_MAX));
  }
  if constexpr (kSoftmax) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = i < own && v[i] > top ? v[i] : top;
    top = group_top<G>(top);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // short chains of additions: a tighter margin
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = __builtin_amdgcn_exp2f((v[i] - top) * kLog2e);
      sum[i % 8] += i < own ? v[i] : 0.f;
    }
    inv = __builtin_amdgcn_rcpf(
        group_sum<G>(((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]))));
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if constexpr (kSoftmax) v[i] = v[i] * inv + bias[i];
    else v[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v[i] * -kLog2e)) + bias[i];
  }
  // How far a value can be from the exact one, doubled, with an eighth more. In units of 2^-24:
  //   sigmoid  the exponential's argument |x| s (1 - s) <= 0.23 x 1.3, its value 2 s (1 - s) <= 0.5, the sum with one 1,
  //            the inverse 2: 4
  //   softmax  with z = max - x: the difference and the argument 2.3 z, the exponential 2; the sum has these (its
  //            terms' mean z is below 4.5 for 1024 experts) and 12 additions, the inverse and the product 3: 2.3 z
  //            + 30 of p = inv e^-z, at most 30 of inv
  // and the sum with the bias, and the exact value's rounding to fp32, |c| each.
  const float base = kSoftmax ? inv * 0x1.2p-18f : 0x1.2p-21f;
  auto margin = [&](float c) { return base + fabsf(c) * 0x1.2p-22f; };
  // whether any lane of this lane's token says so
  auto token_any = [&](bool said) {
    return (__ballot(in.live && said) >> (token * G) & ((uint64_t{1} << G) - 1)) != 0;
  };
  // softmax: inv64 of the tokens that ask, one after the other by the whole wave (about 1 us for one of 256)
  auto find_inverse = [&](bool asks) {
    uint64_t todo = __ballot(asks && inv64 == 0.0);
    while (todo != 0) {
      const int from = __ffsll(static_cast<unsigned long long>(todo)) - 1;
      todo &= ~(((uint64_t{1} << G) - 1) << (from / G * G));
      const float* row = a.logits + (in.t - token + from / G) * a.E;
      const float most = __shfl(top, from);
      double sum = 0.0;
#pragma unroll 1
      for (int e = lane; e < a.E; e += kWave) sum += exp64(static_cast<double>(row[e]) - most);
      sum = wave_sum(sum);
      if (token == from / G) inv64 = inverse64(sum);
    }
  };
  // the exact choice value of one expert
  auto exact = [&](int e) {
    const float x = in.logit(e);
    const double s = kSoftmax ? exp64(static_cast<double>(x) - top) * inv64 : sigmoid64(x);
    return static_cast<float>(s + static_cast<double>(masked(x, in.one(in.bias_buffer(a), e * 4u))));
  };
  int o[VPL], best[L];
#pragma unroll
  for (int i = 0; i < VPL; ++i) o[i] = i < own ? signed_order(v[i]) : INT_MIN;
#pragma unroll
  for (int i = kRun; i < L; ++i) best[i] = INT_MIN;
#pragma unroll
  for (int r = 0; r < VPL; r += kRun) {
    int run[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) run[i] = o[r + i];
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
  bool sure = best[0] <= signed_order(1e38f);  // no NaN, and sums and margins of values are finite
  if (a.top_groups < a.groups) {
    int one = best[0], two = best[1];
    merge_two<G>(one, two, P);
    // the group's value lies between low and high: its values' errors, and the roundings of both sums
    const bool pair = a.group_top == 2 && size > 1;
    const float c1 = from_signed(one), c2 = from_signed(two), value = pair ? c1 + c2 : c1;
    const float off = 0.5f * (margin(c1) + (pair ? margin(c2) : 0.f)) + fabsf(value) * 0x1p-22f;
    const bool real = in.group < a.groups;
    const float low = real ? value - off : -INFINITY, high = real ? value + off : -INFINITY;
    int above = 0, beside = 0;  // lanes of groups before this one for sure, and perhaps
    other_lanes<G>(static_cast<int>(__float_as_uint(low)), g, __ffs(P) - 1, [&](int bits, int of) {
      above += of != in.group && __uint_as_float(static_cast<uint32_t>(bits)) > high;
    });
    other_lanes<G>(static_cast<int>(__float_as_uint(high)), g, __ffs(P) - 1, [&](int bits, int of) {
      beside += of != in.group && !(__uint_as_float(static_cast<uint32_t>(bits)) < low);
    });
    const bool close = token_any(in.group < a.groups && above < a.top_groups * P && beside >= a.top_groups * P);
    if (__any(close)) {
      if constexpr (kSoftmax) find_inverse(close);
      const float second = best[1] != INT_MIN ? from_signed(best[1]) : -INFINITY;
      const int from = signed_order(second - margin(second));
      uint32_t near = 0, first_ord = 0, second_ord = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) near |= static_cast<uint32_t>(close && i < own && o[i] >= from) << i;
#pragma unroll 1
      while (near != 0) {
        const int e = in.e0 + __ffs(near) - 1;
        near &= near - 1;
        const uint32_t c = orderable(exact(e));
        second_ord = max(second_ord, min(first_ord, c));
        first_ord = max(first_ord, c);
      }
      merge_two<G>(first_ord, second_ord, P);
      const uint32_t rank_by = in.group >= a.groups ? 0u
                               : a.group_top == 2 && size > 1
                                   ? orderable(from_orderable(first_ord) + from_orderable(second_ord))
                                   : first_ord;
      const int before = lanes_before<G, true, false>(rank_by, first_ord, g, __ffs(P) - 1);
      above = close ? before : above;
    }
    if (above >= a.top_groups * P) {
      own = 0;
#pragma unroll
      for (int i = 0; i < L; ++i) best[i] = INT_MIN;
    }
  }
  merge_lanes<G>(best);
  int least = best[0];
#pragma unroll
  for (int i = 1; i < L; ++i) least = i == a.k - 1 ? best[i] : least;
  least = signed_order(from_signed(least) - margin(from_signed(least)));
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) mine |= static_cast<uint32_t>(o[i] >= least) << i;
  if (own == 0 || !in.live) mine = 0;  // past the last token: no candidates
  // candidates in the order of their ids
  int at = __popc(mine);
#pragma unroll
  for (int off = 1; off < G; off *= 2) {
    const int other = __shfl_up(at, off, G);
    at += g >= off ? other : 0;
  }
  const int count = __shfl(at, lane | (G - 1));
  at -= __popc(mine);
  sure = sure && count >= a.k && count <= Candidates<G, L>::kMost;
  if (__any(in.live && !sure)) return false;
  while (mine != 0) {
    const int i = __ffs(mine) - 1;
    mine &= mine - 1;
    if (at < Candidates<G, L>::kMost) room.id[token][at] = static_cast<uint16_t>(in.e0 + i);
    ++at;
  }
  wave_sync();
  int id[kSlots], rank[kSlots];
  double s[kSlots], key[kSlots];  // s: the score, or its logit's exponential
  auto rank_all = [&]() {
    auto against = [&](int first) {
#pragma unroll
      for (int j = first; j < first + G; ++j) {
        const double other = room.key[token][j];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) rank[q] += other > key[q];
      }
    };
#pragma unroll
    for (int q = 0; q < kSlots; ++q) rank[q] = 0;
    against(0);
#pragma unroll
    for (int q = 1; q < kSlots; ++q)
      if (__any(in.live && count > q * G)) against(q * G);
  };
  auto keep = [&](int q, float c) {
    const int j = q * G + g;
    key[q] = j < count ? key_of(orderable(c), id[q]) : 1.0;
    room.key[token][j] = key[q];
  };
  float c[kSlots], x[kSlots], add[kSlots];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int j = q * G + g;
    id[q] = j < count ? room.id[token][j] : 0;
    x[q] = in.logit(id[q]);
    add[q] = masked(x[q], in.one(in.bias_buffer(a), id[q] * 4u));
    if constexpr (kSoftmax) {
      s[q] = exp64(static_cast<double>(x[q]) - top);
      c[q] = __builtin_amdgcn_exp2f((x[q] - top) * kLog2e) * inv + add[q];
      room.logit[token][j] = x[q];
      room.bias[token][j] = add[q];
    } else {
      s[q] = sigmoid64(x[q]);
      c[q] = static_cast<float>(s[q] + static_cast<double>(add[q]));
    }
    keep(q, c[q]);
  }
  wave_sync();
  if constexpr (kSoftmax) {
    bool close = false;  // to another candidate that is not the very same
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      if (q > 0 && !__any(in.live && count > q * G)) break;
      for (int j = 0; j < count; ++j) {
        const float other = from_orderable(key_ord(room.key[token][j]));
        const bool same = room.logit[token][j] == x[q] && room.bias[token][j] == add[q];
        close = close || (q * G + g < count && !same && !(fabsf(other - c[q]) > margin(c[q])));
      }
    }
    wave_sync();
    close = token_any(close);
    if (__any(close)) {
      find_inverse(close);
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (close) keep(q, static_cast<float>(s[q] * inv64 + static_cast<double>(add[q])));
      wave_sync();
    }
  }
  rank_all();
  wave_sync();  // the next tokens' candidates are written over these
  double sum = 0.0;
  float most = -INFINITY;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    rank[q] = q * G + g < count ? rank[q] : a.k;
    if (kSoftmax) most = rank[q] < a.k && x[q] > most ? x[q] : most;
  }
  if (kSoftmax && a.renormalize) {  // softmax over the chosen
    most = group_top<G>(most);
#pragma unroll
    for (int q = 0; q < kSlots; ++q) s[q] = exp64(static_cast<double>(x[q]) - most);
  }
#pragma unroll
  for (int q = 0; q < kSlots; ++q) sum += rank[q] < a.k ? s[q] : 0.0;
  if (a.renormalize) sum = group_sum<G>(sum) + (kSoftmax ? 0.0 : 1e-20);
  else sum = kSoftmax ? 1.0 / static_cast<double>(inv) : 1.0;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    if (in.live && rank[q] < a.k) {
      a.idx[in.t * a.k + rank[q]] = id[q];
      a.w[in.t * a.k + rank[q]] = static_cast<float>(a.scale * (s[q] / sum));
    }
  }
  return true;
}

// Waves per SIMD (registers: 128 or 170) where tokens are many: 131072 x 256 sigmoids in 8 groups 72 us
// with two, 58 with three, 55 with four; softmax scores, all in fp64, 125, 106, 114; logits with their sum three 43,
// four 50.
template <int G, Route MODE>
constexpr int route_waves() { return MODE == Route::kSoftmax || MODE == Route::kLogitsTotal || G == 32 ? 3 : 4; }

template <int G, int VPL, int L, Route MODE, bool QUICK>
__global__ __launch_bounds__(kThreads, (route_waves<G, MODE>())) void route_kernel(const RouteArgs a, int P, int per) {
  using In = Rows<G, VPL>;
  const int wv = uniform(static_cast<int>(threadIdx.x) / kWave);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWavesPerBlock * In::kTokens;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wv) * In::kTokens; t0 < a.T; t0 += step) {
    const In in(a, P, per, t0);
    if constexpr (QUICK) {
      __shared__ Candidates<G, L> room[kWavesPerBlock];
      if (route_quick<G, VPL, L, MODE>(a, in, P, room[wv])) continue;
    }
    route_exact<G, VPL, L, MODE, QUICK>(a, in, P);
  }
}

template <int G, int VPL, int L, Route MODE, bool QUICK = false>
hipError_t launch_route(const RouteArgs& a, int P, int per, hipStream_t stream) {
  const int64_t tokens = kWavesPerBlock * (kWave / G);
  const int64_t blocks = min((a.T + tokens - 1) / tokens, int64_t{1} << 20);
  hipLaunchKernelGGL((route_kernel<G, VPL, L, MODE, QUICK>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                     stream, a, P, per);
  return hipGetLastError();
}

template <int G, int VPL, int L>
hipError_t launch_route_mode(const RouteArgs& a, int P, int per, hipStream_t stream) {
  // The search for candidates pays where a lane has many values, by what follows it. Sigmoids: 16384 x 256 of 32 values,
  // k = 8 11.2 us (all in fp64 16.3), k = 16 13 (21); 16384 x 128 of 16 values, k = 8 7.1 (8.6); 21169 x 90 of 12 values,
  // k = 9 14.2 (13.2); 64 x 128 of 8 values 4.8 (4.7). Softmax: 131072 x 256 of 32 values, k = 8 76 (107), 16384 16.2
  // (20.4), k = 16 23.1 (21.4); 21169 x 90 of 12 values, k = 8 13.6 (14.3), k = 9 19.0 (16.6).
  constexpr bool kSome = G >= 8 && G <= 32;
  constexpr bool kQuick = kSome && (VPL >= 32 || (VPL >= 16 && L <= 8)), kQuickSoftmax = kSome && VPL >= 32 && L <= 8;
  if (a.by_score && a.sigmoid) return launch_route<G, VPL, L, Route::kSigmoid, kQuick>(a, P, per, stream);
  if (a.by_score) return launch_route<G, VPL, L, Route::kSoftmax, kQuickSoftmax>(a, P, per, stream);
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
// Bound by writing d_logits. Rows are put together in LDS and leave as one run.

// n floats from LDS by one wave.
__device__ __forceinline__ void write_run(const float* __restrict__ from, float* __restrict__ to, int n) {
  typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
  const int lane = lane_id();
  for (int i = lane * 4; i + 4 <= n; i += kWave * 4) {
    const float4 v = *reinterpret_cast<const float4*>(from + i);
    *reinterpret_cast<f32x4*>(to + i) = f32x4{v.x, v.y, v.z, v.w};
  }
  const int i = (n & ~3) + lane;
  if (i < n) to[i] = from[i];
}

// Every gradient but that of the plain softmax is 0 outside the chosen experts. S lanes (a power
// of two, k <= S) share a token, a wave takes as many tokens as their rows fit its LDS.
// 16384 tokens x 8 of 256: 6.3 us (a wave for each token: 10.4); 131072: 30 us, 4.4 TB/s.
constexpr int kRunFloats = 2048;

template <int S>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const RouteArgs a, const float* __restrict__ d_w,
                                                                  float* __restrict__ d_logits) {
  __shared__ __attribute__((aligned(16))) float runs[kWavesPerBlock][kRunFloats];
  const int lane = lane_id(), wv = uniform(static_cast<int>(threadIdx.x) / kWave);
  const int token = lane / S, j = lane % S;
  float* run = runs[wv];
  const int tokens = min(kWave / S, kRunFloats / a.E);  // E <= 1024
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWavesPerBlock * tokens;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wv) * tokens; t0 < a.T; t0 += step) {
    const int here = static_cast<int>(min(a.T - t0, static_cast<int64_t>(tokens)));
    const int64_t t = t0 + token;
    int e = -1;
    float u = 0.f, x = 0.f;
    if (token < here && j < a.k) {
      e = a.idx[t * a.k + j];
      u = a.scale * d_w[t * a.k + j];
      if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.E)) e = -1;
      if (e >= 0) x = a.logits[t * a.E + e];
    }
    for (int i = lane * 4; i < here * a.E; i += kWave * 4) *reinterpret_cast<float4*>(run + i) = make_float4(0, 0, 0, 0);
    float s = 0.f, top = 0.f;
    if (a.sigmoid) {
      s = e >= 0 ? 1.f / (1.f + expf(-x)) : 0.f;
    } else {
      top = group_top<S>(e >= 0 ? x : -INFINITY);
      s = e >= 0 ? expf(x - top) : 0.f;
    }
    float grad = u * s / (1.f + expf(x));  // sigmoid, not renormalised
    if (a.renormalize) {
      const float by = group_sum<S>(s) + (a.sigmoid ? 1e-20f : 0.f), dot = group_sum<S>(u * s);
      grad = a.sigmoid ? (u - dot / by) / by * s / (1.f + expf(x)) : s / by * (u - dot / by);
    }
    wave_sync();
    if (e >= 0) run[token * a.E + e] = grad;
    wave_sync();
    write_run(run, d_logits + t0 * a.E, here * a.E);
    wave_sync();
  }
}

// More than a wave of chosen experts: one wave per token, in turns.
__global__ __launch_bounds__(kThreads) void route_any_backward_kernel(const RouteArgs a, const float* __restrict__ d_w,
                                                                      float* __restrict__ d_logits) {
  __shared__ __attribute__((aligned(16))) float rows[kWavesPerBlock][kMaxExperts];
  const int lane = lane_id(), wv = static_cast<int>(threadIdx.x) / kWave;
  float* row = rows[wv];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wv; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kWavesPerBlock) {
    const float* x = a.logits + t * a.E;
    const int32_t* idx = a.idx + t * a.k;
    const float* up = d_w + t * a.k;
    for (int e = lane; e < a.E; e += kWave) row[e] = 0.f;
    float top = 0.f;
    if (!a.sigmoid) {
      top = -INFINITY;
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
    const float by = wave_sum(sum) + (a.sigmoid ? 1e-20f : 0.f);
    dot = wave_sum(dot);
    wave_sync();
    for (int j = lane; j < a.k; j += kWave) {
      const int e = idx[j];
      if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.E)) continue;
      const float v = x[e], u = a.scale * up[j], s = score(v);
      if (!a.sigmoid) row[e] = s / by * (u - dot / by);
      else row[e] = (a.renormalize ? (u - dot / by) / by : u) * s / (1.f + expf(v));
    }
    wave_sync();
    write_run(row, d_logits + t * a.E, a.E);
    wave_sync();
  }
}

// The plain softmax: G lanes hold a token's row, VPL experts each (16384 x 256: 9.5 us with 32 lanes of 8, 10.3
// with 16 of 16; x 128: 6.4 with 16 of 8, 7.1 with 8 of 16).
template <int G, int VPL>
__global__ __launch_bounds__(kThreads) void route_softmax_backward_kernel(const RouteArgs a,
                                                                          const float* __restrict__ d_w,
                                                                          float* __restrict__ d_logits, int per) {
  using In = Rows<G, VPL>;
  __shared__ __attribute__((aligned(16))) float runs[kWavesPerBlock][kWave * VPL];
  const int wv = uniform(static_cast<int>(threadIdx.x) / kWave);
  float* run = runs[wv];
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWavesPerBlock * In::kTokens;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + wv) * In::kTokens; t0 < a.T; t0 += step) {
    const In in(a, G, per, t0);
    float v[VPL];
    in.logits(v);
    float top = -INFINITY, total = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = i < in.own ? fmaxf(top, v[i]) : top;
    top = group_top<G>(top);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = expf(v[i] - top);
      total += i < in.own ? v[i] : 0.f;
    }
    total = group_sum<G>(total);
    const float inv = 1.f / total;
    float dot = 0.f;
    auto chosen = [&](int j) {  // -1: none of this token's
      const int e = in.live && j < a.k ? a.idx[in.t * a.k + j] : -1;
      return static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E) ? e : -1;
    };
    for (int j = in.g; j < a.k; j += G) {
      const int e = chosen(j);
      if (e >= 0) dot = fmaf(a.scale * d_w[in.t * a.k + j], expf(in.logit(e) - top) * inv, dot);
    }
    dot = group_sum<G>(dot);
    float* row = run + in.row / 4;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < in.own) row[in.e0 + i] = -(v[i] * inv) * dot;
    wave_sync();
    for (int j = in.g; j < a.k; j += G) {
      const int e = chosen(j);
      if (e >= 0) row[e] = expf(in.logit(e) - top) * inv * (a.scale * d_w[in.t * a.k + j] - dot);
    }
    wave_sync();
    write_run(run, d_logits + t0 * a.E, static_cast<int>(min(a.T - t0, static_cast<int64_t>(In::kTokens))) * a.E);
    wave_sync();
  }
}

// a launch holds fewer than 2^32 threads; waves' tokens past these take turns
unsigned wave_blocks(int64_t waves) {
  return static_cast<unsigned>(min((waves + kWavesPerBlock - 1) / kWavesPerBlock, int64_t{1} << 20));
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
    auto per = [&](int lanes) { return (size + lanes / blocks - 1) / (lanes / blocks); };  // values of a lane
    auto fits = [&](int lanes, int values) { return blocks <= lanes && per(lanes) <= values; };
    int few = 1;  // lanes of a call of few tokens
    while (few < kWave && !fits(few, few < 16 ? 8 : 16)) few *= 2;
    // more tokens never take more lanes (2048 x 64 6.5 us with 64, 3.6 with 8; 4096 x 256 sigmoids in groups 9.6 with 32, 6.5 with 16)
#define MOE_ROUTE(LANES, VALUES)                                                                  \
  if (fits(LANES, VALUES) && (least == 0 || (T * LANES >= least && LANES < few)))                 \
    return launch_route_top<LANES, VALUES>(a, LANES / blocks, per(LANES), stream)
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
  moe_router whole = r;  // the choice is made: no groups
  whole.groups = whole.top_groups = whole.group_top = 1;
  const RouteArgs a = make_args(whole, logits, const_cast<int32_t*>(idx), nullptr, T, E, k);
  if (!a.sigmoid && !a.renormalize) {
#define MOE_ROUTE(G, VPL)                                                                                         \
  do {                                                                                                            \
    const int64_t waves = (T * G + kWave - 1) / kWave;                                                            \
    hipLaunchKernelGGL((route_softmax_backward_kernel<G, VPL>), dim3(wave_blocks(waves)), dim3(kThreads), 0,      \
                       stream, a, d_w, d_logits, (E + G - 1) / G);                                                \
    return hipGetLastError();                                                                                     \
  } while (0)
    if (E <= 8) MOE_ROUTE(1, 8);
    if (E <= 16) MOE_ROUTE(2, 8);
    if (E <= 32) MOE_ROUTE(4, 8);
    if (E <= 64) MOE_ROUTE(8, 8);
    if (E <= 128) MOE_ROUTE(16, 8);
    if (E <= 256) MOE_ROUTE(32, 8);
    if (E <= 512) MOE_ROUTE(64, 8);
    MOE_ROUTE(64, 16);
#undef MOE_ROUTE
  }
#define MOE_ROUTE(S)                                                                                                  \
  do {                                                                                                                \
    const int64_t tokens = min(kWave / S, kRunFloats / E), waves = (T + tokens - 1) / tokens;                         \
    hipLaunchKernelGGL(route_backward_kernel<S>, dim3(wave_blocks(waves)), dim3(kThreads), 0, stream, a, d_w, d_logits); \
    return hipGetLastError();                                                                                         \
  } while (0)
  if (k <= 4) MOE_ROUTE(4);
  if (k <= 8) MOE_ROUTE(8);
  if (k <= 16) MOE_ROUTE(16);
  if (k <= 64) MOE_ROUTE(64);
#undef MOE_ROUTE
  hipLaunchKernelGGL(route_any_backward_kernel, dim3(wave_blocks(T)), dim3(kThreads), 0, stream, a, d_w, d_logits);
  return hipGetLastError();
}

}  // namespace moe
