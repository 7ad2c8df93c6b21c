// Residual add and layer norm of hidden states, and its gradient.
//
// The mathematics, per row of d elements (fp32 throughout, one rounding per
// output element):
//   s    = x + r, rounded to the rows' type (it is the residual stream that the
//          next block reads, and the backward starts from it); s = x without r
//   m    = sum(s) / d;  v = sum((s - m)^2) / d;  rstd = 1 / sqrt(v + eps)
//   y    = (s - m) * rstd * w + b
// and backwards, with h = (s - m) * rstd and g = w * dy:
//   dx   = rstd * (g - sum(g)/d - h * sum(g h)/d) + ds
//   dw   = sum over rows of dy * h;  db = sum over rows of dy
//
// Both directions move a few bytes per operation and are bound by HBM: a row is
// read once, held in registers through its reductions (the variance is taken
// around the mean, not from a sum of squares, so a large mean costs no digits),
// and written once.
#include <limits.h>

#include "row_group.h"

namespace moe {
namespace {

using namespace rows;

constexpr int kMaxD = 32768;

template <int G>
constexpr int block_threads() { return G > 256 ? G : 256; }

// G threads per row, VPT vectors per thread. STREAM: the rows do not fit the caches.
template <bool BF16, bool WBF16, int G, int VPT, bool STREAM>
__global__ __launch_bounds__(block_threads<G>()) void layer_norm_kernel(
    const uint4* x, const uint4* r, const void* __restrict__ w, const void* __restrict__ b, float eps, uint4* y,
    uint4* s, float* __restrict__ mean, float* __restrict__ rstd, int64_t T, int row_vec) {
  using V = Vec16<BF16>;
  static_assert(G * VPT * V::kN <= kMaxD, "no row is that long");
  constexpr int kRows = block_threads<G>() / G;  // rows per workgroup
  __shared__ float lds[2][G > kWave ? G / kWave : 1];
  const float d = static_cast<float>(row_vec * V::kN);
  const int li = static_cast<int>(threadIdx.x) % G;
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
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float f[V::kN];
      V::unpack(v[q], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) sum += f[i];
    }
    // A quotient, so that a constant row of bf16 has that constant as its mean: d values of 8 significant bits
    // add up exactly in 24. A sum of fp32 values rounds, and so does its quotient: a few units of the last
    // place (7168 times 1000.1: 1000.10004).
    const float m = group_reduce<G, Sum>(sum, lds[0]) / d;
    float var = 0.f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float f[V::kN], p = 0.f;
      V::unpack(v[q], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) p = fmaf(f[i] - m, f[i] - m, p);
      var += q * G + li < n ? p : 0.f;
    }
    const float rs = 1.f / sqrtf(group_reduce<G, Sum>(var, lds[1]) / d + eps);
    if (n != 0 && li == 0) {
      mean[t] = m;
      rstd[t] = rs;
    }
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      if (c < n) {
        float f[V::kN], wf[V::kN], bf[V::kN];
        V::unpack(v[q], f);
        load_params<V::kN, WBF16>(w, c, wf);
        if (b != nullptr) load_params<V::kN, WBF16>(b, c, bf);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) {
          const float h = (f[i] - m) * rs;
          f[i] = b != nullptr ? fmaf(h, wf[i], bf[i]) : h * wf[i];
        }
        store16<STREAM>(y + base + c, V::pack(f));
      }
    }
  }
}

// The gradient. Workgroups walk rows with a fixed stride and keep their columns'
// sums of dy * h and dy in registers; each leaves one fp32 row of both in
// `partial` [gridDim.x][2][d], added in a fixed order by the kernel below (no
// atomics: the same bits every time). There are one or two workgroups per CU (more
// would leave more partial rows), so each asks for its next row before it reduces
// the present one.
template <bool BF16, int VPT>
struct GradRow {
  uint4 s[VPT], dy[VPT], ds[VPT];
  float mean, rstd;
};

template <bool BF16, bool WBF16, int G, int VPT, bool STREAM>
__global__ __launch_bounds__(block_threads<G>()) void layer_norm_backward_kernel(
    const uint4* dy, const uint4* __restrict__ s, const void* __restrict__ w, const float* __restrict__ mean,
    const float* __restrict__ rstd, const uint4* ds, uint4* dx, float* __restrict__ partial, int64_t T, int row_vec,
    float inv_d) {
  using V = Vec16<BF16>;
  static_assert(G * VPT * V::kN <= kMaxD, "no row is that long");
  constexpr int kRows = block_threads<G>() / G;
  // the next row and the weights stay in registers where there is room for them
  constexpr bool kAhead = G <= 512;
  __shared__ float lds[2][G > kWave ? 2 * G / kWave : 1];
  __shared__ float cols[kRows > 1 ? 2 * G * VPT * V::kN : 1];  // the groups' column sums, joined
  const int li = static_cast<int>(threadIdx.x) % G;
  using Row = GradRow<BF16, VPT>;
  auto fetch = [&](Row& o, int64_t t) {
    const int n = t < T ? row_vec : 0;
    const int64_t base = t * row_vec;
    o.mean = n ? mean[t] : 0.f;
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
  float aw[VPT][V::kN], ab[VPT][V::kN];
#pragma unroll
  for (int q = 0; q < VPT; ++q)
#pragma unroll
    for (int i = 0; i < V::kN; ++i) aw[q][i] = ab[q][i] = 0.f;
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
    const float m = row.mean, rs = row.rstd;
    float c12[2] = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      if (q * G + li < n) {
        float f[V::kN], g[V::kN], wf[V::kN];
        V::unpack(row.s[q], f);
        V::unpack(row.dy[q], g);
        weights(q, wf);
#pragma unroll
        for (int i = 0; i < V::kN; ++i) {
          const float h = (f[i] - m) * rs, gw = g[i] * wf[i];
          c12[0] += gw;
          c12[1] = fmaf(gw, h, c12[1]);
          aw[q][i] = fmaf(g[i], h, aw[q][i]);
          ab[q][i] += g[i];
        }
      }
    }
    group_reduce<G, Sum>(c12, lds[turn]);
    turn ^= 1;
    const float c1 = c12[0] * inv_d, c2 = c12[1] * inv_d;
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
          const float h = (f[i] - m) * rs;
          const float o = rs * (fmaf(g[i], wf[i], -c1) - h * c2);
          f[i] = ds != nullptr ? o + e[i] : o;
        }
        store16<STREAM>(dx + base + c, V::pack(f));
      }
    }
  }
  const int d = row_vec * V::kN;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * d;
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
            cols[G * VPT * V::kN + c] = (g ? cols[G * VPT * V::kN + c] : 0.f) + ab[q][i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += block_threads<G>()) {
      out[c] = cols[c];
      out[d + c] = cols[G * VPT * V::kN + c];
    }
  } else {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = q * G + li;
      if (c < row_vec) {
#pragma unroll
        for (int i = 0; i < V::kN / 4; ++i) {
          reinterpret_cast<float4*>(out + c * V::kN)[i] =
              make_float4(aw[q][4 * i], aw[q][4 * i + 1], aw[q][4 * i + 2], aw[q][4 * i + 3]);
          reinterpret_cast<float4*>(out + d + c * V::kN)[i] =
              make_float4(ab[q][4 * i], ab[q][4 * i + 1], ab[q][4 * i + 2], ab[q][4 * i + 3]);
        }
      }
    }
  }
}

// dw[c] and db[c] (the second half of a partial row) = sum over the partial rows:
// 64 columns per workgroup, 16 waves each taking every 16th row, joined in wave
// order. Rounded once to the parameters' type.
template <bool WBF16>
__global__ __launch_bounds__(1024) void layer_norm_columns_kernel(const float* __restrict__ partial, int rows, int d,
                                                                  void* __restrict__ dw, void* __restrict__ db) {
  __shared__ float part[16][kWave];
  const int wv = static_cast<int>(threadIdx.x) / kWave;
  const int c = static_cast<int>(blockIdx.x) * kWave + lane_id();
  float a = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int i = wv; i < rows; i += 16) a += partial[static_cast<int64_t>(i) * 2 * d + c];
  }
  part[wv][lane_id()] = a;
  __syncthreads();
  if (wv == 0 && c < 2 * d) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += part[i][lane_id()];
    void* out = c < d ? dw : db;
    const int k = c < d ? c : c - d;
    if (out != nullptr) {
      if (WBF16) static_cast<__bf16*>(out)[k] = static_cast<__bf16>(a);
      else static_cast<float*>(out)[k] = a;
    }
  }
}

template <int G>
unsigned row_blocks(int64_t T, int64_t most) {
  const int64_t per = block_threads<G>() / G;
  const int64_t b = (T + per - 1) / per;
  return static_cast<unsigned>(b < most ? b : most);
}

constexpr int kBackwardBlocks = 512;  // partial rows at most

// Workgroups (and partial rows) of the gradient. Two per CU where every one then has four turns or more:
// a partial row is 2 d fp32 values written and read again, and a workgroup of one or two turns has
// nothing to prefetch. Of bf16, two, one and half a workgroup per CU: 256 x 2880 9.7, 9.7, 8.5 us; 777 x 2880 15.1,
// 12.1, 12.9; 2048 x 2880 17.5, 17.9, 24.6; 16384 x 2880 69, 100, 183. One per CU is as many as fit (and
// prefetch) where a row has more than 768 vectors: 2048 x 7168 33, 28, 37; 12000 x 8192 137, 133, 210.
template <int G>
unsigned backward_blocks(int64_t T, int row_vec) {
  const int64_t turns = row_blocks<G>(T, int64_t{1} << 30);  // of one workgroup alone
  if (turns >= 4 * kBackwardBlocks && row_vec <= 768) return kBackwardBlocks;
  const int64_t most = turns / 2 < 128 ? 128 : turns / 2 < 256 ? turns / 2 : 256;
  return static_cast<unsigned>(turns < most ? turns : most);
}

constexpr int64_t kForwardBlocks = int64_t{1} << 21;  // a launch holds fewer than 2^32 threads; rows past it take turns

// F(G, VPT) for a row of up to 4096 vectors, as many as bf16 rows have; longer fp32 rows take 1024 x 8. A row that no more than half fills its threads wastes
// their loads, hence the steps between powers of two (16384 x 1032 bf16, three vectors of a wave against
// one of a workgroup: forward 26 us against 30, gradient 32 against 45; 16384 x 4104, gradient 112
// against 142). Rows past 16384 bf16 elements run the gradient at 2.1-2.3 TB/s (16384 x 32768): beside the row,
// their column sums do not fit the registers of 1024 threads, and 70 to 100 of them are spilled. Column sums in
// a second pass over dy and s would move 5/3 of the bytes (with ds 3/2); not tried.
#define MOE_NORM_SHAPES(F)             \
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

#define MOE_NORM_BWD_SHAPES(F)         \
  if (row_vec <= 16) F(16, 1);         \
  else if (row_vec <= 32) F(32, 1);    \
  else if (row_vec <= 64) F(64, 1);    \
  else if (row_vec <= 128) F(64, 2);   \
  else if (row_vec <= 192) F(64, 3);   \
  else if (row_vec <= 256) F(256, 1);  \
  else if (row_vec <= 512) F(512, 1);  \
  else if (row_vec <= 768) F(256, 3);  \
  else if (row_vec <= 1024) F(512, 2); \
  else if (row_vec <= 1536) F(512, 3); \
  else if (row_vec <= 2048) F(1024, 2); \
  else F(1024, 4)

}  // namespace

int64_t layer_norm_max_d() { return kMaxD; }

hipError_t launch_layer_norm(const void* x, const void* r, const void* w, const void* b, float eps, void* y, void* s,
                             float* mean, float* rstd, int64_t T, int d, bool bf16, bool wbf16, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int row_vec = bf16 ? d / 8 : d / 4;
  const bool big = T * d * (bf16 ? 2 : 4) * (r != nullptr ? 4 : 2) > kStreamBytes;
#define MOE_NORM_S(B, W, G, VPT, S)                                                                              \
  hipLaunchKernelGGL((layer_norm_kernel<B, W, G, VPT, S>), dim3(row_blocks<G>(T, kForwardBlocks)),               \
                     dim3(block_threads<G>()), 0, stream, static_cast<const uint4*>(x),                          \
                     static_cast<const uint4*>(r), w, b, eps, static_cast<uint4*>(y), static_cast<uint4*>(s),    \
                     mean, rstd, T, row_vec)
#define MOE_NORM(B, W, G, VPT)                 \
  do {                                         \
    if (big) MOE_NORM_S(B, W, G, VPT, true);   \
    else MOE_NORM_S(B, W, G, VPT, false);      \
  } while (0)
#define MOE_NORM_BB(G, VPT) MOE_NORM(true, true, G, VPT)
#define MOE_NORM_BF(G, VPT) MOE_NORM(true, false, G, VPT)
#define MOE_NORM_FF(G, VPT) MOE_NORM(false, false, G, VPT)
  if (bf16 && wbf16) { MOE_NORM_SHAPES(MOE_NORM_BB); }
  else if (bf16) { MOE_NORM_SHAPES(MOE_NORM_BF); }
  else if (row_vec > 4096) MOE_NORM_FF(1024, 8);
  else { MOE_NORM_SHAPES(MOE_NORM_FF); }
#undef MOE_NORM_BB
#undef MOE_NORM_BF
#undef MOE_NORM_FF
#undef MOE_NORM
#undef MOE_NORM_S
  return hipGetLastError();
}

size_t layer_norm_backward_workspace_bytes(int64_t T, int d) {
  const int64_t rows = T < kBackwardBlocks ? T : kBackwardBlocks;
  return static_cast<size_t>(rows) * 2 * static_cast<size_t>(d) * sizeof(float);
}

hipError_t launch_layer_norm_backward(const void* dy, const void* s, const void* w, const float* mean,
                                      const float* rstd, const void* ds, void* dx, void* dw, void* db, void* ws,
                                      int64_t T, int d, bool bf16, bool wbf16, hipStream_t stream) {
  const int row_vec = bf16 ? d / 8 : d / 4;
  const float inv_d = 1.f / static_cast<float>(d);
  float* partial = static_cast<float*>(ws);
  unsigned blocks = 0;
  if (T > 0) {
    const bool big = T * d * (bf16 ? 2 : 4) * (ds != nullptr ? 4 : 3) > kStreamBytes;
#define MOE_NORM_BWD_S(B, W, G, VPT, S)                                                                           \
  hipLaunchKernelGGL((layer_norm_backward_kernel<B, W, G, VPT, S>), dim3(blocks), dim3(block_threads<G>()), 0,    \
                     stream, static_cast<const uint4*>(dy), static_cast<const uint4*>(s), w, mean, rstd,          \
                     static_cast<const uint4*>(ds), static_cast<uint4*>(dx), partial, T, row_vec, inv_d)
#define MOE_NORM_BWD(B, W, G, VPT)                   \
  do {                                               \
    blocks = backward_blocks<G>(T, row_vec);         \
    if (big) MOE_NORM_BWD_S(B, W, G, VPT, true);     \
    else MOE_NORM_BWD_S(B, W, G, VPT, false);        \
  } while (0)
#define MOE_NORM_BWD_BB(G, VPT) MOE_NORM_BWD(true, true, G, VPT)
#define MOE_NORM_BWD_BF(G, VPT) MOE_NORM_BWD(true, false, G, VPT)
#define MOE_NORM_BWD_FF(G, VPT) MOE_NORM_BWD(false, false, G, VPT)
    if (bf16 && wbf16) { MOE_NORM_BWD_SHAPES(MOE_NORM_BWD_BB); }
    else if (bf16) { MOE_NORM_BWD_SHAPES(MOE_NORM_BWD_BF); }
    else if (row_vec > 4096) MOE_NORM_BWD_FF(1024, 8);
    else { MOE_NORM_BWD_SHAPES(MOE_NORM_BWD_FF); }
#undef MOE_NORM_BWD_BB
#undef MOE_NORM_BWD_BF
#undef MOE_NORM_BWD_FF
#undef MOE_NORM_BWD
#undef MOE_NORM_BWD_S
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>((2 * d + kWave - 1) / kWave));
  if (wbf16)
    hipLaunchKernelGGL(layer_norm_columns_kernel<true>, grid, dim3(1024), 0, stream, partial, static_cast<int>(blocks),
                       d, dw, db);
  else
    hipLaunchKernelGGL(layer_norm_columns_kernel<false>, grid, dim3(1024), 0, stream, partial,
                       static_cast<int>(blocks), d, dw, db);
  return hipGetLastError();
}

}  // namespace moe
