// One AdamW step over a list of tensors, with states in fp32 or in 8 bits.
//
//   g = grad * min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p - (lr wd p + lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// Bound by HBM: every array is read and written once (28 bytes an element for bf16
// weights with masters and fp32 states, 16 with 8-bit states: 398M elements in 1975 us
// and 1160 us, 5.6 and 5.5 TB/s). The tensors of a list are cut into pieces, numbered
// through, a workgroup each (2048 workgroups that take turns: 2180 us for 398M weights
// against 1975). A launch carries its tensors' addresses in the kernel arguments (no table
// to copy, so a captured graph keeps them), up to kList of them.
//
// 8-bit states hold m and sqrt(v), whose range is half of v's in powers of two, as e4m3
// with an fp32 scale per 128 elements: relative errors of 2^-4 down to 2^-15 of the block's
// largest, where codes of equal steps would lose all small elements. sqrt(v) > 0 never
// becomes 0 (m / eps would be the step); its smallest code, 2^-9 / 448 of the largest, is
// too large then, which makes the step smaller. The step itself uses m and v before the rounding.
//
// A step lowers m and sqrt(v) by (1 - b1) and (1 - b2) / 2 of themselves at most, and the nearest code
// is that of the step before where this is less than half a code (3 to 6 %): a state whose gradients
// fade stays where it is (b2 = 0.999, gradients down to a tenth: sqrt(v) 7 to 12 times too large for good).
// Dithered codes go up or down with the probabilities that make their mean the value; the noise that
// stays is about a code (15 % of sqrt(v), whatever b2). Its random bits are a hash of the element's
// index and the step's number: the same inputs give the same codes, however a list is cut. (398M elements
// 1230 us, with the nearest codes 1160: two 32-bit products a hash.)
#include <math.h>

#include "row_group.h"

namespace moe {
namespace {

using rows::kStreamBytes;

constexpr int kThreads = 256;
constexpr int kList = 32;
// Elements of a piece: sixteen a thread, or eight where there are few pieces for the chip.
constexpr int kPiece = 4096;
constexpr int kSmallPiece = 2048;
constexpr int64_t kFewPieces = 1024;
constexpr int64_t kBlocks = int64_t{1} << 23;  // a launch holds fewer than 2^32 threads; pieces past it take turns
constexpr int kStateBlock = MOE_STATE_BLOCK;
constexpr float kClipEps = 1e-6f;
constexpr float kCodeStep = 1.f / 448.f;  // of the largest code
enum class Hold { kF32, kNearest, kDither };  // of the states: fp32, or 8 bits with codes rounded like this
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

struct Entry {
  void* p;
  const void* g;
  float* w;  // the master, or null
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t numel;
  double decay;  // the weight decay
  uint8_t p_bf16, g_bf16;
};
struct List {
  Entry t[kList];
  int64_t piece0[kList + 1];  // first piece of each tensor
  int n;
};

struct Scalars {
  const float* d_lr;
  const int64_t* d_step;
  const float* norm;
  int64_t step;
  double lr, log_b1, log_b2;
  float b1, b2, one_b1, one_b2;  // 1 - b from the fp64 b
  float eps, max_norm;
};

// The finaliser of MurmurHash3 (Appleby): every bit of h changes about half of the result's.
__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ h >> 16) * 0x85EBCA6Bu;
  h = (h ^ h >> 13) * 0xC2B2AE35u;
  return h ^ h >> 16;
}

// Of one call: the rate over the first bias correction, the root's factor, the clip factor, the step's hash.
struct Step {
  double lr;
  float rate, root, coef;
  uint32_t key;
};

__device__ __forceinline__ Step step_of(const Scalars& a) {
  Step s;
  const double lr = a.d_lr != nullptr ? static_cast<double>(*a.d_lr) : a.lr;
  const int64_t step = a.d_step == nullptr ? a.step : *a.d_step < 1 ? 1 : *a.d_step;
  const double t = static_cast<double>(step);
  s.key = mix(static_cast<uint32_t>(step) ^ mix(static_cast<uint32_t>(static_cast<uint64_t>(step) >> 32)));
  s.lr = lr;
  s.rate = static_cast<float>(lr / -expm1(t * a.log_b1));
  s.root = static_cast<float>(1.0 / sqrt(-expm1(t * a.log_b2)));
  s.coef = 1.f;
  if (a.norm != nullptr) {
    const float c = a.max_norm * (1.f / (*a.norm + kClipEps));
    s.coef = c >= 1.f ? 1.f : c;  // a NaN norm gives NaN
  }
  return s;
}

// N consecutive elements, of which `n` (<= N) exist; the others read as 0 (FULL: all exist).
// Vectors are aligned to their elements only, which global memory takes.
template <typename T, int N>
struct Pack {
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

template <bool STREAM, bool FULL, typename T, int N>
__device__ __forceinline__ void load_n(const T* p, int n, T* out) {
  using P = typename Pack<T, N>::type;
  if (FULL || n == N) {
    P v;
    if constexpr (STREAM) v = __builtin_nontemporal_load(reinterpret_cast<const P*>(p));
    else v = *reinterpret_cast<const P*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = i < n ? p[i] : T{};
  }
}

template <bool STREAM, bool FULL, typename T, int N>
__device__ __forceinline__ void store_n(T* p, int n, const T* in) {
  using P = typename Pack<T, N>::type;
  if (FULL || n == N) {
    P v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = in[i];
    if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<P*>(p));
    else *reinterpret_cast<P*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = in[i];
  }
}

template <bool STREAM, bool FULL, int N, bool BF16>
__device__ __forceinline__ void load_f(const void* base, int64_t a, int n, float* f) {
  if constexpr (BF16) {
    uint16_t h[N];
    load_n<STREAM, FULL, uint16_t, N>(static_cast<const uint16_t*>(base) + a, n, h);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = bf16_to_f32(h[i]);
  } else {
    load_n<STREAM, FULL, float, N>(static_cast<const float*>(base) + a, n, f);
  }
}

template <bool STREAM, bool FULL, int N, bool BF16>
__device__ __forceinline__ void store_f(void* base, int64_t a, int n, const float* f) {
  if constexpr (BF16) {
    uint16_t h[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t u = rows::Vec16<true>::round2(f[i], f[i + 1]);
      h[i] = static_cast<uint16_t>(u);
      h[i + 1] = static_cast<uint16_t>(u >> 16);
    }
    store_n<STREAM, FULL, uint16_t, N>(static_cast<uint16_t*>(base) + a, n, h);
  } else {
    store_n<STREAM, FULL, float, N>(static_cast<float*>(base) + a, n, f);
  }
}

// Every product and sum is rounded by itself: which of them a compiler joins would decide, for a
// state near the middle between two codes, which of the two it gets. decay is lr wd itself: 1 - lr wd in fp32 is
// off by 2^-25, all of a decay of 2e-8 and a fifth of one of 1e-7.
__device__ __forceinline__ void update(float& p, float g, float& m, float& v, float& root, const Scalars& a,
                                       const Step& s, float decay) {
#pragma clang fp contract(off)
  g = g * s.coef;
  m = m * a.b1 + g * a.one_b1;
  v = v * a.b2 + g * g * a.one_b2;
  root = sqrtf(v);
  p = p - (p * decay + s.rate * (m / (root * s.root + a.eps)));
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max_u32(v, static_cast<uint32_t>(
                        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false)));
}

// The largest of each aligned 16 lanes, to all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_max<0x141>(v);  // row_half_mirror
  return dpp_max<0x140>(v);  // row_mirror
}

// Four codes and their values.
__device__ __forceinline__ uint32_t codes4(const float* f) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
  return static_cast<uint32_t>(w);
}
__device__ __forceinline__ void values4(const uint8_t (&c)[4], float* f) {
  const int w = static_cast<int>(c[0] | c[1] << 8 | c[2] << 16 | static_cast<uint32_t>(c[3]) << 24);
  f[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0);
  f[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
  f[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2);
  f[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3);
}

// a (at most 448, but for a rounding) as one of the two e4m3 values around it, the larger with the probability of
// a's share of the way there. bits: 16 random ones, the upper of the 20 below a code's own, so that a code's value
// always stays. Below 2^-6 codes are 2^-9 apart, as they are for another 2^-6 on top.
template <bool POSITIVE>
__device__ __forceinline__ float dithered(float a, uint32_t bits) {
  const float mag = POSITIVE ? a : fabsf(a), shift = mag < 0x1p-6f ? 0x1p-6f : 0.f;
  const float up = __uint_as_float((__float_as_uint(mag + shift) + (bits << 4 | 8u)) & 0xFFF00000u) - shift;
  return POSITIVE ? fminf(up, 448.f) : copysignf(fminf(up, 448.f), a);
}

// The block's scale from its 16 lanes' values, and this lane's codes. With DITHER, the upper (ROOT) or lower half of
// an element's 32 random bits.
template <bool ROOT, bool DITHER>
__device__ __forceinline__ float encode(const float (&f)[8], const uint32_t (&random)[DITHER ? 8 : 1],
                                        uint8_t (&codes)[2][4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_u32(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  top = row_max(top);
  const bool finite = top < 0x7F800000u;
  const float scale = fmaxf(__uint_as_float(top) * kCodeStep, kMinScale);
  const float inv = 1.f / scale;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = finite ? f[4 * h + i] * inv : 0.f;
      if constexpr (DITHER) a[i] = dithered<ROOT>(a[i], ROOT ? random[4 * h + i] >> 16 : random[4 * h + i] & 0xFFFFu);
    }
    const uint32_t w = codes4(a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t b = static_cast<uint8_t>(w >> (8 * i));
      codes[h][i] = ROOT && b == 0 && finite && f[4 * h + i] > 0.f ? 1 : b;
    }
  }
  return finite ? scale : __uint_as_float(0x7FC00000u);
}

// A piece with fp32 states: 4 elements of every array at a time, all loads of a thread's
// four such groups before the first is used.
template <int PIECE, bool P_BF16, bool G_BF16, bool MASTER, bool STREAM, bool FULL>
__device__ __forceinline__ void piece_f32(const Entry& e, int64_t first, const Scalars& a, const Step& s, float decay) {
  constexpr int N = 4, kU = PIECE / (kThreads * N);
  float p[kU][N], g[kU][N], m[kU][N], v[kU][N];
  int n[kU];
#pragma unroll
  for (int q = 0; q < kU; ++q) {
    const int64_t i = first + (q * kThreads + static_cast<int>(threadIdx.x)) * N;
    const int64_t left = e.numel - i;
    n[q] = FULL || left >= N ? N : left > 0 ? static_cast<int>(left) : 0;
    load_f<STREAM, FULL, N, G_BF16>(e.g, i, n[q], g[q]);
    if (MASTER) load_f<STREAM, FULL, N, false>(e.w, i, n[q], p[q]);
    else load_f<STREAM, FULL, N, P_BF16>(e.p, i, n[q], p[q]);
    load_f<STREAM, FULL, N, false>(e.m, i, n[q], m[q]);
    load_f<STREAM, FULL, N, false>(e.v, i, n[q], v[q]);
  }
#pragma unroll
  for (int q = 0; q < kU; ++q) {
    const int64_t i = first + (q * kThreads + static_cast<int>(threadIdx.x)) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float root;
      update(p[q][j], g[q][j], m[q][j], v[q][j], root, a, s, decay);
    }
    if (MASTER) store_f<STREAM, FULL, N, false>(e.w, i, n[q], p[q]);
    store_f<STREAM, FULL, N, P_BF16>(e.p, i, n[q], p[q]);
    store_f<STREAM, FULL, N, false>(e.m, i, n[q], m[q]);
    store_f<STREAM, FULL, N, false>(e.v, i, n[q], v[q]);
  }
}

// A piece with 8-bit states: a block of 128 elements is in 16 lanes, four elements of each of
// its halves in a lane, so that a load of fp32 values is one run as well.
template <bool DITHER, int PIECE, bool P_BF16, bool G_BF16, bool MASTER, bool STREAM, bool FULL>
__device__ __forceinline__ void piece_e4m3(const Entry& e, int64_t first, const Scalars& a, const Step& s, float decay) {
  constexpr int N = 4, kHalves = 2, kLanes = kStateBlock / (N * kHalves), kU = PIECE / (kThreads * N * kHalves);
  const int block = static_cast<int>(threadIdx.x) / kLanes, lane = static_cast<int>(threadIdx.x) % kLanes;
  float p[kU][kHalves][N], g[kU][kHalves][N], ms[kU], vs[kU];
  uint8_t mc[kU][kHalves][N], vc[kU][kHalves][N];
  int n[kU][kHalves];
#pragma unroll
  for (int q = 0; q < kU; ++q) {
    const int64_t i0 = first + (q * (kThreads / kLanes) + block) * kStateBlock;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int64_t i = i0 + h * (kStateBlock / kHalves) + lane * N;
      const int64_t left = e.numel - i;
      n[q][h] = FULL || left >= N ? N : left > 0 ? static_cast<int>(left) : 0;
      load_f<STREAM, FULL, N, G_BF16>(e.g, i, n[q][h], g[q][h]);
      if (MASTER) load_f<STREAM, FULL, N, false>(e.w, i, n[q][h], p[q][h]);
      else load_f<STREAM, FULL, N, P_BF16>(e.p, i, n[q][h], p[q][h]);
      load_n<STREAM, FULL, uint8_t, N>(static_cast<const uint8_t*>(e.m) + i, n[q][h], mc[q][h]);
      load_n<STREAM, FULL, uint8_t, N>(static_cast<const uint8_t*>(e.v) + i, n[q][h], vc[q][h]);
    }
    const bool any = FULL || i0 < e.numel;
    ms[q] = any ? e.ms[i0 / kStateBlock] : 0.f;
    vs[q] = any ? e.vs[i0 / kStateBlock] : 0.f;
  }
#pragma unroll
  for (int q = 0; q < kU; ++q) {
    const int64_t i0 = first + (q * (kThreads / kLanes) + block) * kStateBlock;
    float m[kHalves * N], root[kHalves * N];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      values4(mc[q][h], m + h * N);
      values4(vc[q][h], root + h * N);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float& mj = m[h * N + j];
        float& rj = root[h * N + j];
        mj *= ms[q];
        rj *= vs[q];
        float v = rj * rj;
        update(p[q][h][j], g[q][h][j], mj, v, rj, a, s, decay);
        if (!FULL && j >= n[q][h]) mj = rj = 0.f;  // past the last element: not in the block's largest
      }
    }
    uint32_t random[DITHER ? kHalves * N : 1];
    if constexpr (DITHER) {
      const uint32_t high = mix(static_cast<uint32_t>(static_cast<uint64_t>(i0) >> 32) + s.key);  // the block's
#pragma unroll
      for (int j = 0; j < kHalves * N; ++j)
        random[j] = mix((static_cast<uint32_t>(i0) + j / N * (kStateBlock / kHalves) + lane * N + j % N) ^ high);
    }
    const float m_scale = encode<false, DITHER>(m, random, mc[q]), v_scale = encode<true, DITHER>(root, random, vc[q]);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int64_t i = i0 + h * (kStateBlock / kHalves) + lane * N;
      if (MASTER) store_f<STREAM, FULL, N, false>(e.w, i, n[q][h], p[q][h]);
      store_f<STREAM, FULL, N, P_BF16>(e.p, i, n[q][h], p[q][h]);
      store_n<STREAM, FULL, uint8_t, N>(static_cast<uint8_t*>(e.m) + i, n[q][h], mc[q][h]);
      store_n<STREAM, FULL, uint8_t, N>(static_cast<uint8_t*>(e.v) + i, n[q][h], vc[q][h]);
    }
    if (lane == 0 && (FULL || i0 < e.numel)) {
      e.ms[i0 / kStateBlock] = m_scale;
      e.vs[i0 / kStateBlock] = v_scale;
    }
  }
}

template <Hold HOLD, int PIECE, bool STREAM, bool P_BF16, bool G_BF16, bool MASTER>
__device__ __forceinline__ void piece(const Entry& e, int64_t first, const Scalars& a, const Step& s, float decay) {
  constexpr bool kE4m3 = HOLD != Hold::kF32, kDither = HOLD == Hold::kDither;
  // only a tensor's last piece looks where the tensor ends
  if (first + PIECE <= e.numel) {
    if constexpr (kE4m3) piece_e4m3<kDither, PIECE, P_BF16, G_BF16, MASTER, STREAM, true>(e, first, a, s, decay);
    else piece_f32<PIECE, P_BF16, G_BF16, MASTER, STREAM, true>(e, first, a, s, decay);
  } else {
    if constexpr (kE4m3) piece_e4m3<kDither, PIECE, P_BF16, G_BF16, MASTER, STREAM, false>(e, first, a, s, decay);
    else piece_f32<PIECE, P_BF16, G_BF16, MASTER, STREAM, false>(e, first, a, s, decay);
  }
}

template <Hold HOLD, int PIECE, bool STREAM>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const List l, const Scalars a) {
  const Step s = step_of(a);
  const int64_t total = l.piece0[l.n];
  int i = 0;
  for (int64_t at = blockIdx.x; at < total; at += gridDim.x) {
    while (l.piece0[i + 1] <= at) ++i;
    const Entry& e = l.t[i];
    const int64_t first = (at - l.piece0[i]) * PIECE;
    const float decay = static_cast<float>(s.lr * e.decay);
    if (!e.p_bf16) {
      if (e.g_bf16) piece<HOLD, PIECE, STREAM, false, true, false>(e, first, a, s, decay);
      else piece<HOLD, PIECE, STREAM, false, false, false>(e, first, a, s, decay);
    } else if (e.w != nullptr) {
      if (e.g_bf16) piece<HOLD, PIECE, STREAM, true, true, true>(e, first, a, s, decay);
      else piece<HOLD, PIECE, STREAM, true, false, true>(e, first, a, s, decay);
    } else {
      if (e.g_bf16) piece<HOLD, PIECE, STREAM, true, true, false>(e, first, a, s, decay);
      else piece<HOLD, PIECE, STREAM, true, false, false>(e, first, a, s, decay);
    }
  }
}

template <Hold HOLD>
hipError_t launch_list(const List& l, const Scalars& a, bool small, bool big, hipStream_t stream) {
  const int64_t pieces = l.piece0[l.n];
  const dim3 grid(static_cast<unsigned>(pieces < kBlocks ? pieces : kBlocks));
  if (small) hipLaunchKernelGGL((adamw_kernel<HOLD, kSmallPiece, false>), grid, dim3(kThreads), 0, stream, l, a);
  else if (big) hipLaunchKernelGGL((adamw_kernel<HOLD, kPiece, true>), grid, dim3(kThreads), 0, stream, l, a);
  else hipLaunchKernelGGL((adamw_kernel<HOLD, kPiece, false>), grid, dim3(kThreads), 0, stream, l, a);
  return hipGetLastError();
}

// Memory of a tensor that the step touches.
int64_t bytes_of(const moe_adamw_tensor& t, bool e4m3) {
  const int64_t p = t.param_dt == MOE_BF16 ? (t.master != nullptr ? 6 : 2) : 4;
  return t.numel * (p + (t.grad_dt == MOE_BF16 ? 2 : 4) + (e4m3 ? 2 : 8));
}

}  // namespace

hipError_t launch_adamw(const moe_adamw_tensor* t, int n, const moe_adamw_args& args, hipStream_t stream) {
  const bool e4m3 = args.state == MOE_STATE_E4M3;
  Scalars a;
  a.d_lr = args.d_lr;
  a.d_step = args.d_step;
  a.norm = args.norm;
  a.lr = args.lr;
  a.step = args.step;
  a.log_b1 = log(args.beta1);
  a.log_b2 = log(args.beta2);
  a.b1 = static_cast<float>(args.beta1);
  a.b2 = static_cast<float>(args.beta2);
  a.one_b1 = static_cast<float>(1.0 - args.beta1);
  a.one_b2 = static_cast<float>(1.0 - args.beta2);
  a.eps = static_cast<float>(args.eps);
  a.max_norm = args.max_norm;
  int64_t bytes = 0, pieces = 0;
  for (int i = 0; i < n; ++i) {
    bytes += bytes_of(t[i], e4m3);
    pieces += (t[i].numel + kPiece - 1) / kPiece;
  }
  // A list that does not fit the memory-side cache passes it by (398M bf16 weights with masters: 1975 us, and 2080
  // through the cache; with 8-bit states 1160 and 1214). One that fits is found there by the next call (157 MB: 57 us, and 64 past it).
  const bool big = bytes > kStreamBytes;
  // (60 fp32 tensors of 1 to 368641 elements, 1.5M in all: 14.5 us, and 18.7 with the large pieces)
  const bool small = !big && pieces <= kFewPieces;
  const int64_t piece = small ? kSmallPiece : kPiece;
  for (int i0 = 0; i0 < n;) {
    List l;
    l.n = 0;
    l.piece0[0] = 0;
    for (; l.n < kList && i0 < n; ++i0) {
      if (t[i0].numel == 0) continue;
      Entry& e = l.t[l.n];
      e.p = t[i0].param;
      e.g = t[i0].grad;
      e.w = t[i0].master;
      e.m = t[i0].exp_avg;
      e.v = t[i0].exp_avg_sq;
      e.ms = t[i0].exp_avg_scale;
      e.vs = t[i0].exp_avg_sq_scale;
      e.numel = t[i0].numel;
      e.decay = args.weight_decays != nullptr ? args.weight_decays[i0] : args.weight_decay;
      e.p_bf16 = t[i0].param_dt == MOE_BF16;
      e.g_bf16 = t[i0].grad_dt == MOE_BF16;
      l.piece0[l.n + 1] = l.piece0[l.n] + (t[i0].numel + piece - 1) / piece;
      ++l.n;
    }
    if (l.n == 0) break;
    const hipError_t err = !e4m3 ? launch_list<Hold::kF32>(l, a, small, big, stream)
                           : args.rounding == MOE_DITHER ? launch_list<Hold::kDither>(l, a, small, big, stream)
                                                         : launch_list<Hold::kNearest>(l, a, small, big, stream);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
