// Row-wise kernels: a group of kG threads owns one row of 16-byte vectors and
// keeps its kVpt vectors per thread in registers, so a row is read once however
// many reductions it takes. Groups of up to a wave reduce by lane exchanges;
// wider groups (a whole workgroup) add one pass through LDS.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace rows {

// The 8 bf16 or 4 fp32 elements of a 16-byte vector.
template <bool BF16>
struct Vec16;

template <>
struct Vec16<true> {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  // round to nearest even; NaN stays NaN (the carry of the rounding must not run over its payload)
  __device__ static uint32_t round2(float lo, float hi) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t p = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, p);
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(round2(f[0], f[1]), round2(f[2], f[3]), round2(f[4], f[5]), round2(f[6], f[7]));
  }
};

template <>
struct Vec16<false> {
  static constexpr int kN = 4;
  __device__ static void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// A 16-byte vector, with STREAM past the caches (data that is too large to be found there again).
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint4* p) {
  if constexpr (STREAM) {
    const i32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(p));
    return make_uint4(static_cast<uint32_t>(v.x), static_cast<uint32_t>(v.y), static_cast<uint32_t>(v.z),
                      static_cast<uint32_t>(v.w));
  } else {
    return *p;
  }
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint4* p, const uint4& v) {
  if constexpr (STREAM) {
    const i32x4_t d = {static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w)};
    __builtin_nontemporal_store(d, reinterpret_cast<i32x4_t*>(p));
  } else {
    *p = v;
  }
}

// Bytes of one call from which its tensors are streamed: the memory-side cache holds 256 MB, so
// a call that moves more finds little of its data there again, and neither does the next one.
constexpr int64_t kStreamBytes = int64_t{256} << 20;

// kN consecutive parameters (N = 8 or 4) from vector c of a bf16 or fp32 array
template <int N, bool BF16>
__device__ __forceinline__ void load_params(const void* p, int c, float* f) {
  if constexpr (BF16) {
    static_assert(N == 8, "bf16 parameters go with bf16 rows");
    Vec16<true>::unpack(static_cast<const uint4*>(p)[c], f);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) Vec16<false>::unpack(static_cast<const uint4*>(p)[c * (N / 4) + i], f + 4 * i);
  }
}

struct Sum {
  template <typename T>
  __device__ static T apply(T a, T b) { return a + b; }
};
struct Max {
  template <typename T>
  __device__ static T apply(T a, T b) { return a > b ? a : b; }
};

// Reduction of N values per thread over a group of G threads (a power of two); every
// thread gets the results, which are the same bits in each and do not depend on
// timing. For G > 64 the group is the workgroup and `lds` holds N * G / 64 values:
// it must not be the buffer of the call before (which a slower wave may still read),
// so callers alternate between two.
template <int G, typename Op, int N, typename T>
__device__ __forceinline__ void group_reduce(T (&v)[N], T* lds) {
#pragma unroll
  for (int off = (G < kWave ? G : kWave) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Op::apply(v[i], __shfl_xor(v[i], off));
  if constexpr (G > kWave) {
    constexpr int kW = G / kWave;
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) lds[i * kW + threadIdx.x / kWave] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = lds[i * kW];
#pragma unroll
      for (int w = 1; w < kW; ++w) v[i] = Op::apply(v[i], lds[i * kW + w]);
    }
  }
}

template <int G, typename Op, typename T>
__device__ __forceinline__ T group_reduce(T v, T* lds) {
  T a[1] = {v};
  group_reduce<G, Op, 1, T>(a, lds);
  return a[0];
}

}  // namespace rows
}  // namespace moe
