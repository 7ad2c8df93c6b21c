// Residual add and RMS norm of hidden states, with an output in 8 bits, and its gradient.
//
// Per row of d elements (one rounding per output element):
//   s    = x + r, rounded to the rows' type (the residual stream that the next block
//          reads); s = x without r
//   rstd = 1 / sqrt(sum(s^2) / d + eps);  y = s * rstd * w
//   scale = max(max|y| / 127, 2^-126), q = rint(y * (1 / scale)), of the fp32 y
// and backwards, with h = s * rstd and g = w * dy:
//   dx   = rstd * (g - h * sum(g h) / d) + ds;  dw = sum over rows of dy * h
//
// Squares are summed in fp64: those of bf16 and fp32 values are exact or nearly so there,
// and none over- or underflows (a row of 1e30 has its norm). The rest is fp32. Both
// directions are bound by HBM: a row is read once and held in registers through its
// reductions. 16384 x 7168 bf16 with a residual 153 us (6.1 TB/s); 8192 x 2880 bf16 18.1 us,
// with 8-bit rows 26.5; 32 x 2880 3.4 and 4.3, one launch's latency. The gradient of 4096 x
// 4096 bf16 with ds 23.6 us (5.7 TB/s), and 3.9 for the join of the column sums; of 1024 x 32768 bf16
// 63 us (3.2 TB/s: rows of 1024 threads spill 11 to 14 registers).
#include <limits.h>

#include "int8_code.h"

namespace moe {
namespace {

using namespace rows;

template <int G>
constexpr int block_threads() { return G > 256 ? G : 256; }

// G threads per row, VPT vectors per thread. STREAM: the rows do not fit the caches.
// CODES (bf16 rows): the 8-bit rows [kblocks][T][64] and their scales as well (then y may be null).
template <bool BF16, bool WBF16, int G, int VPT, bool STREAM, bool CODES>
__global__ __launch_bounds__(block_threads<G>()) void rms_norm_kernel(
    const uint4* x, const uint4* r, const void* __restrict__ w, float eps, uint4* y, uint4* s,
    float* __restrict__ rstd, uint8_t* __restrict__ q8, float* __restrict__ q8_scale, int64_t T, int row_vec) {
  using V = Vec16<BF16>;
  static_assert(BF16 || !CODES, "the experts' 8-bit rows are those of bf16 rows");
  constexpr int kRows = block_threads<G>() / G;  // rows per workgroup
  __shared__ double sums[2][G > kWave ? G / kWave : 1];
  __shared__ uint32_t tops[CODES && G > kWave ? G / kWave : 1];
  const int li = static_cast<int>(threadIdx.x) % G;
  int turn = 0;
  // the bound is the same for every group of a workgroup, so barriers inside are uniform
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < T; t0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t t = t0 + threadIdx.x / G;
    const int n = t < T ? row_vec : 0;
    const int64_t base = t * row_vec;
    uint4 v[VPT];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      v[q] = c < n ? load16<STREAM>(x + base + c) : make_uint4(0, 0, 0, 0);
    }
    if (r != nullptr) {
      uint4 u[VPT];
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int c = q * G + li;
        u[q] = c < n ? load16<STREAM>(r + base + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int c = q * G + li;
        float f[V::kN], g[V::kN];
        V::unpack(v[q], f);
        V::unpack(u[q], g);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) f[i] += g[i];
        v[q] = V::pack(f);
        if (c < n) store16<STREAM>(s + base + c, v[q]);
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float f[V::kN];
      V::unpack(v[q], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) sum = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), sum);
    }
    sum = group_reduce<G, Sum>(sum, sums[turn]);
    turn ^= 1;
    const float rs = static_cast<float>(1.0 / sqrt(sum / (row_vec * V::kN) + eps));
    if (n != 0 && li == 0) rstd[t] = rs;
    auto normed = [&](int q, float* f) {
      float wf[V::kN];
      V::unpack(v[q], f);
      load_params<V::kN, WBF16>(w, q * G + li, wf);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) f[i] = f[i] * rs * wf[i];
    };
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      if (c < n) {
        float f[V::kN];
        normed(q, f);
        if (!CODES || y != nullptr) store16<STREAM>(y + base + c, V::pack(f));
        if (CODES)
#pragma unroll
          for (int i = 0; i < V::kN; ++i) top = Max::apply(top, int8::abs_bits(f[i]));
      }
    }
    if constexpr (CODES) {
      // the next row's sum has a barrier between these reads and its writes of tops
      top = group_reduce<G, Max>(top, tops);
      float sc, inv;
      int8::scale_of(top, &sc, &inv);
      if (n != 0 && li == 0) q8_scale[t] = sc;
      const int padded = n != 0 ? (row_vec + 7) / 8 * 8 : 0;  // zeros past the last column
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int c = q * G + li;
        float f[V::kN];
        if (c < n) normed(q, f);
        else
#pragma unroll
          for (int i = 0; i < V::kN; ++i) f[i] = 0.f;
        if (c < padded)
          *reinterpret_cast<uint2*>(q8 + (static_cast<int64_t>(c / 8) * T + t) * 64 + c % 8 * 8) = int8::codes8(f, inv);
      }
    }
  }
}

// The gradient. Workgroups walk rows with a fixed stride and keep their columns' sums of
// dy * h in registers; each leaves one fp32 row of them in `partial` [gridDim.x][d], added
// in a fixed order by the kernel below (no atomics: the same bits every time). Each asks
// for its next row before it reduces the present one.
template <bool BF16, int VPT>
struct GradRow {
  uint4 s[VPT], dy[VPT], ds[VPT];
  float rstd;
};

template <bool BF16, bool WBF16, int G, int VPT, bool STREAM>
__global__ __launch_bounds__(block_threads<G>()) void rms_norm_backward_kernel(
    const uint4* dy, const uint4* __restrict__ s, const void* __restrict__ w, const float* __restrict__ rstd,
    const uint4* ds, uint4* dx, float* __restrict__ partial, int64_t T, int row_vec, float inv_d) {
  using V = Vec16<BF16>;
  constexpr int kRows = block_threads<G>() / G;
  // the next row and the weights stay in registers where there is room for them
  constexpr bool kAhead = G <= 512;
  __shared__ float lds[2][G > kWave ? G / kWave : 1];
  __shared__ float cols[kRows > 1 ? G * VPT * V::kN : 1];  // the groups' column sums, joined
  const int li = static_cast<int>(threadIdx.x) % G;
  using Row = GradRow<BF16, VPT>;
  auto fetch = [&](Row& o, int64_t t) {
    const int n = t < T ? row_vec : 0;
    const int64_t base = t * row_vec;
    o.rstd = n ? rstd[t] : 0.f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      o.s[q] = c < n ? load16<STREAM>(s + base + c) : make_uint4(0, 0, 0, 0);
      o.dy[q] = c < n ? load16<STREAM>(dy + base + c) : make_uint4(0, 0, 0, 0);
      if (kAhead) o.ds[q] = ds != nullptr && c < n ? load16<STREAM>(ds + base + c) : make_uint4(0, 0, 0, 0);
    }
  };
  float wr[kAhead ? VPT : 1][V::kN];
  if constexpr (kAhead) {
#pragma unroll
    for (int q = 0; q < VPT; ++q)
      if (q * G + li < row_vec) load_params<V::kN, WBF16>(w, q * G + li, wr[q]);
  }
  auto weights = [&](int q, float* wf) {
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < V::kN; ++i) wf[i] = wr[q][i];
    } else {
      load_params<V::kN, WBF16>(w, q * G + li, wf);
    }
  };
  float aw[VPT][V::kN];
#pragma unroll
  for (int q = 0; q < VPT; ++q)
#pragma unroll
    for (int i = 0; i < V::kN; ++i) aw[q][i] = 0.f;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  Row row, next;
  if (kAhead && first < T) fetch(next, first + threadIdx.x / G);
  int turn = 0;
  // the bound is the same for every group of a workgroup, so barriers inside are uniform
  for (int64_t t0 = first; t0 < T; t0 += stride) {
    const int64_t t = t0 + threadIdx.x / G;
    const int n = t < T ? row_vec : 0;
    const int64_t base = t * row_vec;
    if constexpr (kAhead) {
      row = next;
      if (t0 + stride < T) fetch(next, t + stride);
    } else {
      fetch(row, t);
    }
    const float rs = row.rstd;
    float dot = 0.f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      if (q * G + li < n) {
        float f[V::kN], g[V::kN], wf[V::kN];
        V::unpack(row.s[q], f);
        V::unpack(row.dy[q], g);
        weights(q, wf);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) {
          const float h = f[i] * rs;
          dot = fmaf(g[i] * wf[i], h, dot);
          aw[q][i] = fmaf(g[i], h, aw[q][i]);
        }
      }
    }
    const float c2 = group_reduce<G, Sum>(dot, lds[turn]) * inv_d;
    turn ^= 1;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      if (c < n) {
        float f[V::kN], g[V::kN], wf[V::kN], e[V::kN];
        V::unpack(row.s[q], f);
        V::unpack(row.dy[q], g);
        if (kAhead) V::unpack(row.ds[q], e);
        else if (ds != nullptr) V::unpack(load16<STREAM>(ds + base + c), e);
        weights(q, wf);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) {
          const float o = rs * (g[i] * wf[i] - f[i] * rs * c2);
          f[i] = ds != nullptr ? o + e[i] : o;
        }
        store16<STREAM>(dx + base + c, V::pack(f));
      }
    }
  }
  const int d = row_vec * V::kN;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * d;
  if constexpr (kRows > 1) {
    // groups add their sums one after the other, in group order
    for (int g = 0; g < kRows; ++g) {
      if (static_cast<int>(threadIdx.x) / G == g) {
#pragma unroll
        for (int q = 0; q < VPT; ++q)
#pragma unroll
          for (int i = 0; i < V::kN; ++i) {
            const int c = (q * G + li) * V::kN + i;
            cols[c] = (g ? cols[c] : 0.f) + aw[q][i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += block_threads<G>()) out[c] = cols[c];
  } else {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      if (c < row_vec) {
#pragma unroll
        for (int i = 0; i < V::kN / 4; ++i)
          reinterpret_cast<float4*>(out + c * V::kN)[i] =
              make_float4(aw[q][4 * i], aw[q][4 * i + 1], aw[q][4 * i + 2], aw[q][4 * i + 3]);
      }
    }
  }
}

// dw[c] = sum over the partial rows: 64 columns per workgroup, 16 waves each taking every
// 16th row, joined in wave order. Rounded once to the weights' type.
template <bool WBF16>
__global__ __launch_bounds__(1024) void rms_norm_columns_kernel(const float* __restrict__ partial, int rows, int d,
                                                                void* __restrict__ dw) {
  __shared__ float part[16][kWave];
  const int wv = static_cast<int>(threadIdx.x) / kWave;
  const int c = static_cast<int>(blockIdx.x) * kWave + lane_id();
  float a = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = wv; i < rows; i += 16) a += partial[static_cast<int64_t>(i) * d + c];
  }
  part[wv][lane_id()] = a;
  __syncthreads();
  if (wv == 0 && c < d) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += part[i][lane_id()];
    if (WBF16) static_cast<__bf16*>(dw)[c] = static_cast<__bf16>(a);
    else static_cast<float*>(dw)[c] = a;
  }
}

template <int G>
unsigned row_blocks(int64_t T, int64_t most) {
  const int64_t per = block_threads<G>() / G;
  const int64_t b = (T + per - 1) / per;
  return static_cast<unsigned>(b < most ? b : most);
}

constexpr int kBackwardBlocks = 512;  // partial rows at most

// Workgroups (and partial rows) of the gradient: as for the layer norm's.
template <int G>
unsigned backward_blocks(int64_t T, int row_vec) {
  const int64_t turns = row_blocks<G>(T, int64_t{1} << 30);  // of one workgroup alone
  if (turns >= 4 * kBackwardBlocks && row_vec <= 768) return kBackwardBlocks;
  const int64_t most = turns / 2 < 128 ? 128 : turns / 2 < 256 ? turns / 2 : 256;
  return static_cast<unsigned>(turns < most ? turns : most);
}

constexpr int64_t kForwardBlocks = int64_t{1} << 21;  // a launch holds fewer than 2^32 threads; rows past it take turns

// F(G, VPT) for a row of that many vectors (with the 8-bit rows: filled up to whole K-blocks), as few
// threads as hold a row without more than four vectors each, and steps between powers of two: a row that
// half fills its threads wastes their loads.
#define MOE_RMS_SHAPES(F)              \
  if (row_vec <= 16) F(16, 1);         \
  else if (row_vec <= 32) F(32, 1);    \
  else if (row_vec <= 64) F(64, 1);    \
  else if (row_vec <= 128) F(64, 2);   \
  else if (row_vec <= 192) F(64, 3);   \
  else if (row_vec <= 256) F(256, 1);  \
  else if (row_vec <= 512) F(256, 2);  \
  else if (row_vec <= 768) F(256, 3);  \
  else if (row_vec <= 1024) F(256, 4); \
  else if (row_vec <= 1536) F(512, 3); \
  else if (row_vec <= 2048) F(512, 4); \
  else F(1024, 4)

// few: a workgroup has a few rows, so that a row's own time counts (512 x 2 and 256 x 3 of 5120 bf16: 777 rows
// 12.5 and 14.0 us, 4096 rows 32.7 and 32.0, 16384 rows 123 and 116)
#define MOE_RMS_BWD_SHAPES(F)           \
  if (row_vec <= 16) F(16, 1);          \
  else if (row_vec <= 32) F(32, 1);     \
  else if (row_vec <= 64) F(64, 1);     \
  else if (row_vec <= 128) F(64, 2);    \
  else if (row_vec <= 192) F(64, 3);    \
  else if (row_vec <= 256) F(256, 1);   \
  else if (row_vec <= 512) F(512, 1);   \
  else if (row_vec <= 768 && few) F(512, 2); \
  else if (row_vec <= 768) F(256, 3);   \
  else if (row_vec <= 1024) F(512, 2);  \
  else if (row_vec <= 1536) F(512, 3);  \
  else if (row_vec <= 2048) F(1024, 2); \
  else F(1024, 4)

struct Forward {
  const void *x, *r, *w;
  float eps;
  void *y, *s;
  float* rstd;
  void* q;
  float* q_scale;
  int64_t T;
  int row_vec;
  bool big;
};

template <bool BF16, bool WBF16, int G, int VPT, bool STREAM, bool CODES>
void launch_one(const Forward& f, hipStream_t stream) {
  hipLaunchKernelGGL((rms_norm_kernel<BF16, WBF16, G, VPT, STREAM, CODES>), dim3(row_blocks<G>(f.T, kForwardBlocks)),
                     dim3(block_threads<G>()), 0, stream, static_cast<const uint4*>(f.x),
                     static_cast<const uint4*>(f.r), f.w, f.eps, static_cast<uint4*>(f.y), static_cast<uint4*>(f.s),
                     f.rstd, static_cast<uint8_t*>(f.q), f.q_scale, f.T, f.row_vec);
}

template <bool BF16, bool WBF16, int G, int VPT>
void launch_shape(const Forward& f, hipStream_t stream) {
  if constexpr (BF16) {
    if (f.q != nullptr) {
      if (f.big) launch_one<BF16, WBF16, G, VPT, true, true>(f, stream);
      else launch_one<BF16, WBF16, G, VPT, false, true>(f, stream);
      return;
    }
  }
  if (f.big) launch_one<BF16, WBF16, G, VPT, true, false>(f, stream);
  else launch_one<BF16, WBF16, G, VPT, false, false>(f, stream);
}

template <bool BF16, bool WBF16>
void launch_forward(const Forward& f, hipStream_t stream) {
  const int row_vec = f.q != nullptr ? (f.row_vec + 7) / 8 * 8 : f.row_vec;
#define MOE_RMS(G, VPT) launch_shape<BF16, WBF16, G, VPT>(f, stream)
  if constexpr (!BF16) {
    if (row_vec > 4096) {
      MOE_RMS(1024, 8);
      return;
    }
  }
  MOE_RMS_SHAPES(MOE_RMS);
#undef MOE_RMS
}

struct Backward {
  const void *dy, *s, *w;
  const float* rstd;
  const void* ds;
  void* dx;
  float* partial;
  int64_t T;
  int row_vec;
  bool big;
};

template <bool BF16, bool WBF16, int G, int VPT>
unsigned launch_backward_shape(const Backward& b, hipStream_t stream) {
  const unsigned blocks = backward_blocks<G>(b.T, b.row_vec);
  const float inv_d = 1.f / static_cast<float>(b.row_vec * Vec16<BF16>::kN);
#define MOE_RMS_BWD(S)                                                                                             \
  hipLaunchKernelGGL((rms_norm_backward_kernel<BF16, WBF16, G, VPT, S>), dim3(blocks), dim3(block_threads<G>()), 0, \
                     stream, static_cast<const uint4*>(b.dy), static_cast<const uint4*>(b.s), b.w, b.rstd,         \
                     static_cast<const uint4*>(b.ds), static_cast<uint4*>(b.dx), b.partial, b.T, b.row_vec, inv_d)
  if (b.big) MOE_RMS_BWD(true);
  else MOE_RMS_BWD(false);
#undef MOE_RMS_BWD
  return blocks;
}

template <bool BF16, bool WBF16>
unsigned launch_backward(const Backward& b, hipStream_t stream) {
  const int row_vec = b.row_vec;
  const bool few = b.T <= 2048;
#define MOE_RMS(G, VPT) return launch_backward_shape<BF16, WBF16, G, VPT>(b, stream)
  if constexpr (!BF16) {
    if (row_vec > 4096) MOE_RMS(1024, 8);
  }
  MOE_RMS_BWD_SHAPES(MOE_RMS);
#undef MOE_RMS
}

}  // namespace

hipError_t launch_rms_norm(const void* x, const void* r, const void* w, float eps, void* y, void* s, float* rstd,
                           void* q, float* q_scale, int64_t T, int d, bool bf16, bool wbf16, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  Forward f;
  f.x = x;
  f.r = r;
  f.w = w;
  f.eps = eps;
  f.y = y;
  f.s = s;
  f.rstd = rstd;
  f.q = q;
  f.q_scale = q_scale;
  f.T = T;
  f.row_vec = bf16 ? d / 8 : d / 4;
  f.big = T * d * ((bf16 ? 2 : 4) * (r != nullptr ? 4 : 2) + (q != nullptr ? 1 : 0)) > kStreamBytes;
  if (bf16 && wbf16) launch_forward<true, true>(f, stream);
  else if (bf16) launch_forward<true, false>(f, stream);
  else launch_forward<false, false>(f, stream);
  return hipGetLastError();
}

size_t rms_norm_backward_workspace_bytes(int64_t T, int d) {
  const int64_t rows = T < kBackwardBlocks ? T : kBackwardBlocks;
  return static_cast<size_t>(rows) * static_cast<size_t>(d) * sizeof(float);
}

hipError_t launch_rms_norm_backward(const void* dy, const void* s, const void* w, const float* rstd, const void* ds,
                                    void* dx, void* dw, void* ws, int64_t T, int d, bool bf16, bool wbf16,
                                    hipStream_t stream) {
  unsigned blocks = 0;
  if (T > 0) {
    Backward b;
    b.dy = dy;
    b.s = s;
    b.w = w;
    b.rstd = rstd;
    b.ds = ds;
    b.dx = dx;
    b.partial = static_cast<float*>(ws);
    b.T = T;
    b.row_vec = bf16 ? d / 8 : d / 4;
    b.big = T * d * (bf16 ? 2 : 4) * (ds != nullptr ? 4 : 3) > kStreamBytes;
    if (bf16 && wbf16) blocks = launch_backward<true, true>(b, stream);
    else if (bf16) blocks = launch_backward<true, false>(b, stream);
    else blocks = launch_backward<false, false>(b, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>((d + kWave - 1) / kWave));
  if (wbf16)
    hipLaunchKernelGGL(rms_norm_columns_kernel<true>, grid, dim3(1024), 0, stream, static_cast<const float*>(ws),
                       static_cast<int>(blocks), d, dw);
  else
    hipLaunchKernelGGL(rms_norm_columns_kernel<false>, grid, dim3(1024), 0, stream, static_cast<const float*>(ws),
                       static_cast<int>(blocks), d, dw);
  return hipGetLastError();
}

}  // namespace moe
