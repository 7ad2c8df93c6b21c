// The global gradient norm over a list of tensors, and clipping to it.
//
//   norm  = sqrt(sum over all tensors of g^2)
//   out   = g * min(1, max_norm / (norm + 1e-6))
//
// Bound by HBM: the norm reads every element once, the clip reads once more and
// writes once. The tensors of a list are cut into pieces of kPieceBytes at
// 16-byte boundaries of their addresses, numbered through; workgroup i takes
// pieces i, i + grid, ... . A launch carries its tensors' addresses in the kernel
// arguments (no table to copy, so a captured graph keeps them), up to kList of
// them.
//
// The squares are summed in fp64: a product of two fp32 values is exact there, no
// gradient's square over- or underflows, and the sum over billions of elements
// keeps more digits than the fp32 result has. Sums are joined in a fixed order.
#include <limits.h>

#include "row_group.h"

namespace moe {
namespace {

using rows::kStreamBytes;
using rows::load16;
using rows::store16;
using rows::Vec16;

constexpr int kThreads = 256;
constexpr int kList = 64;
constexpr int kPieceVecs = 2048;                 // 16-byte vectors per piece
constexpr int kPieceBytes = kPieceVecs * 16;     // 32 KB
constexpr int kUnroll = kPieceVecs / kThreads;   // vectors per thread and piece
constexpr int kNormBlocks = 2048;
constexpr float kClipEps = 1e-6f;

struct Entry {
  const void* src;
  void* dst;       // clip only
  int64_t numel;
};
struct List {
  Entry t[kList];
  int64_t piece0[kList + 1];  // first piece of each tensor
  uint8_t bf16[kList];
  int n;
};

// Calls piece(addr-aligned vector pointer ...) for this workgroup's pieces.
template <typename F>
__device__ __forceinline__ void for_pieces(const List& l, F&& f) {
  const int64_t total = l.piece0[l.n];
  int i = 0;
  for (int64_t p = blockIdx.x; p < total; p += gridDim.x) {
    while (l.piece0[i + 1] <= p) ++i;
    f(i, p - l.piece0[i]);
  }
}

// Elements [lo, hi) of tensor e that lie in its piece number p, as vectors of the
// piece: vector c holds elements [first + c * N, first + (c + 1) * N).
template <int N>
struct PieceSpan {
  int64_t first, numel;
  __device__ PieceSpan(const Entry& e, int64_t p) : numel(e.numel) {
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(e.src) & 15) / (16 / N));
    first = p * (kPieceVecs * N) - off;
  }
  __device__ bool whole(int c) const {
    const int64_t a = first + static_cast<int64_t>(c) * N;
    return a >= 0 && a + N <= numel;
  }
};

template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

template <bool BF16, bool STREAM>
__device__ __forceinline__ double piece_sumsq(const Entry& e, int64_t p) {
  using V = Vec16<BF16>;
  const PieceSpan<V::kN> span(e, p);
  const char* src = static_cast<const char*>(e.src);
  uint4 v[kUnroll];
  double acc = 0.0;
#pragma unroll
  for (int q = 0; q < kUnroll; ++q) {
    const int c = q * kThreads + static_cast<int>(threadIdx.x);
    const int64_t a = span.first + static_cast<int64_t>(c) * V::kN;
    v[q] = span.whole(c) ? load16<STREAM>(reinterpret_cast<const uint4*>(src + a * (16 / V::kN))) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < kUnroll; ++q) {
    float f[V::kN];
    V::unpack(v[q], f);
#pragma unroll
    for (int i = 0; i < V::kN; ++i) acc = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), acc);
  }
  // the piece's first and last vector may hold elements that are not the tensor's
#pragma unroll
  for (int q = 0; q < kUnroll; ++q) {
    const int c = q * kThreads + static_cast<int>(threadIdx.x);
    const int64_t a = span.first + static_cast<int64_t>(c) * V::kN;
    if (!span.whole(c) && a + V::kN > 0 && a < span.numel) {
      for (int i = 0; i < V::kN; ++i)
        if (a + i >= 0 && a + i < span.numel) {
          const double g = load_one<BF16>(e.src, a + i);
          acc = fma(g, g, acc);
        }
    }
  }
  return acc;
}

__device__ __forceinline__ double block_sum(double v, double* lds) { return rows::group_reduce<kThreads, rows::Sum>(v, lds); }

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void sumsq_kernel(const List l, double* __restrict__ partial) {
  __shared__ double lds[kThreads / kWave];
  double acc = 0.0;
  for_pieces(l, [&](int i, int64_t p) {
    acc += l.bf16[i] ? piece_sumsq<true, STREAM>(l.t[i], p) : piece_sumsq<false, STREAM>(l.t[i], p);
  });
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// The norm from the partial sums: every workgroup that asks gets the same bits.
__device__ __forceinline__ float norm_of(const double* __restrict__ partial, int n, double* lds) {
  double acc = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += kThreads) acc += partial[i];
  return static_cast<float>(sqrt(block_sum(acc, lds)));
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double* __restrict__ partial, int n,
                                                        float* __restrict__ norm) {
  __shared__ double lds[kThreads / kWave];
  const float v = norm_of(partial, n, lds);
  if (threadIdx.x == 0) *norm = v;
}

template <bool BF16, bool STREAM>
__device__ __forceinline__ void piece_scale(const Entry& e, int64_t p, float coef) {
  using V = Vec16<BF16>;
  const PieceSpan<V::kN> span(e, p);
  const char* src = static_cast<const char*>(e.src);
  char* dst = static_cast<char*>(e.dst);
  // vectors of the source; the destination is written in vectors where it has the source's alignment
  const bool same = ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  uint4 v[kUnroll];
#pragma unroll
  for (int q = 0; q < kUnroll; ++q) {
    const int c = q * kThreads + static_cast<int>(threadIdx.x);
    const int64_t a = span.first + static_cast<int64_t>(c) * V::kN;
    v[q] = span.whole(c) ? load16<STREAM>(reinterpret_cast<const uint4*>(src + a * (16 / V::kN))) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < kUnroll; ++q) {
    const int c = q * kThreads + static_cast<int>(threadIdx.x);
    const int64_t a = span.first + static_cast<int64_t>(c) * V::kN;
    if (span.whole(c)) {
      float f[V::kN];
      V::unpack(v[q], f);
#pragma unroll
      for (int i = 0; i < V::kN; ++i) f[i] *= coef;
      const uint4 o = V::pack(f);
      if (same) {
        store16<STREAM>(reinterpret_cast<uint4*>(dst + a * (16 / V::kN)), o);
      } else {
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
        for (int i = 0; i < V::kN; ++i) {
          if (BF16) reinterpret_cast<uint16_t*>(dst)[a + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
          else reinterpret_cast<uint32_t*>(dst)[a + i] = w[i & 3];
        }
      }
    } else if (a + V::kN > 0 && a < span.numel) {
      for (int i = 0; i < V::kN; ++i)
        if (a + i >= 0 && a + i < span.numel) {
          const float g = load_one<BF16>(src, a + i) * coef;
          if (BF16) reinterpret_cast<__bf16*>(dst)[a + i] = static_cast<__bf16>(g);
          else reinterpret_cast<float*>(dst)[a + i] = g;
        }
    }
  }
}

// partial != nullptr: the norm is taken from n partial sums (and written by the
// first workgroup of the first launch); else it is read from *norm.
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void clip_kernel(const List l, const double* __restrict__ partial, int n,
                                                        float* norm, int write_norm, float max_norm) {
  __shared__ double lds[kThreads / kWave];
  const float v = partial != nullptr ? norm_of(partial, n, lds) : *norm;
  if (partial != nullptr && write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  // a NaN norm gives NaN, as the product with it would
  const float c = max_norm / (v + kClipEps);
  const float coef = c >= 1.f ? 1.f : c;
  for_pieces(l, [&](int i, int64_t p) {
    if (coef == 1.f && l.t[i].src == l.t[i].dst) return;  // times one, in place
    if (l.bf16[i]) piece_scale<true, STREAM>(l.t[i], p, coef);
    else piece_scale<false, STREAM>(l.t[i], p, coef);
  });
}

int64_t pieces_of(const moe_tensor& t) {
  const int64_t b = t.dt == MOE_BF16 ? 2 : 4;
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.data) & 15);
  return t.numel > 0 ? (off + t.numel * b + kPieceBytes - 1) / kPieceBytes : 0;
}

// tensors [i0, i0 + kList) of the list (out may be null); returns how many
int fill(List* l, const moe_tensor* in, const moe_tensor* out, int i0, int n) {
  int m = 0;
  l->piece0[0] = 0;
  for (; m < kList && i0 + m < n; ++m) {
    const moe_tensor& t = in[i0 + m];
    l->t[m] = Entry{t.data, out != nullptr ? out[i0 + m].data : nullptr, t.numel};
    l->bf16[m] = t.dt == MOE_BF16;
    l->piece0[m + 1] = l->piece0[m] + pieces_of(t);
  }
  l->n = m;
  return m;
}

unsigned list_blocks(const List& l) {
  const int64_t p = l.piece0[l.n];
  return static_cast<unsigned>(p < 1 ? 1 : p < kNormBlocks ? p : kNormBlocks);
}

// Whether a list is streamed past the caches. The reading pass then runs at 6.9 TB/s instead of
// 6.1 (2.8 GB of bf16: 412 us against 463) and the clip takes 1445 us instead of 1555; a list
// that fits finds its gradients in the caches in the second pass (32 MB: 18 us against 22).
bool stream_list(const moe_tensor* t, int n, int sides) {
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) bytes += t[i].numel * (t[i].dt == MOE_BF16 ? 2 : 4);
  return bytes * sides > kStreamBytes;
}

hipError_t sum_squares(const moe_tensor* t, int n, bool big, double* partial, int* count, hipStream_t stream) {
  *count = 0;
  for (int i0 = 0; i0 < n;) {
    List l;
    i0 += fill(&l, t, nullptr, i0, n);
    const unsigned blocks = list_blocks(l);
    if (big) hipLaunchKernelGGL(sumsq_kernel<true>, dim3(blocks), dim3(kThreads), 0, stream, l, partial + *count);
    else hipLaunchKernelGGL(sumsq_kernel<false>, dim3(blocks), dim3(kThreads), 0, stream, l, partial + *count);
    *count += static_cast<int>(blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t join_partials(const double* partial, int count, float* norm, hipStream_t stream) {
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kThreads), 0, stream, partial, count, norm);
  return hipGetLastError();
}

hipError_t scale_all(const moe_tensor* t, const moe_tensor* out, int n, bool big, const double* partial, int count, float* norm,
                     float max_norm, hipStream_t stream) {
  int i0 = 0;
  do {
    List l;
    const int first = i0 == 0;
    i0 += fill(&l, t, out, i0, n);
    if (big)
      hipLaunchKernelGGL(clip_kernel<true>, dim3(list_blocks(l)), dim3(kThreads), 0, stream, l, partial, count, norm,
                         first, max_norm);
    else
      hipLaunchKernelGGL(clip_kernel<false>, dim3(list_blocks(l)), dim3(kThreads), 0, stream, l, partial, count, norm,
                         first, max_norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } while (i0 < n);
  return hipSuccess;
}

}  // namespace

size_t grad_norm_workspace_bytes(int n) {
  const size_t launches = n > 0 ? (static_cast<size_t>(n) + kList - 1) / kList : 1;
  return launches * kNormBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const moe_tensor* t, int n, float* norm, void* ws, hipStream_t stream) {
  int count = 0;
  hipError_t e = sum_squares(t, n, stream_list(t, n, 1), static_cast<double*>(ws), &count, stream);
  if (e != hipSuccess) return e;
  return join_partials(static_cast<const double*>(ws), count, norm, stream);
}

hipError_t launch_clip_grads(const moe_tensor* t, const moe_tensor* out, int n, const float* norm, float max_norm,
                             hipStream_t stream) {
  return scale_all(t, out, n, stream_list(t, n, out == t ? 1 : 2), nullptr, 0, const_cast<float*>(norm), max_norm, stream);
}

// The clip's workgroups join the partial sums themselves, which saves a launch, as long as there are no
// more than one launch's worth. There are as many workgroups as partial sums, so their reads would grow
// with the square of a list that takes many launches, and those are joined once, by a launch of its own
// (tensors of 1 MB, joined by every workgroup and once: 65 of them 95 us both, 1000 1652 and 1332, 4096
// 12.0 ms and 5.3).
hipError_t launch_clip_grad_norm(const moe_tensor* t, const moe_tensor* out, int n, float max_norm, float* norm,
                                 void* ws, hipStream_t stream) {
  int count = 0;
  const bool big = stream_list(t, n, out == t ? 1 : 2);
  hipError_t e = sum_squares(t, n, big, static_cast<double*>(ws), &count, stream);
  if (e != hipSuccess) return e;
  if (count <= kNormBlocks)
    return scale_all(t, out, n, big, static_cast<const double*>(ws), count, norm, max_norm, stream);
  e = join_partials(static_cast<const double*>(ws), count, norm, stream);
  if (e != hipSuccess) return e;
  return scale_all(t, out, n, big, nullptr, 0, norm, max_norm, stream);
}

}  // namespace moe
