// The 8-bit code of a row's element and the row's scale, as the header defines them.
#pragma once

#include "row_group.h"

namespace moe {
namespace int8 {

constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// scale and 1 / scale from the largest absolute value's bits (as unsigned
// integers these order like the values, infinities and NaN above all others)
__device__ __forceinline__ void scale_of(uint32_t amax_bits, float* scale, float* inv) {
  if (amax_bits >= 0x7F800000u) {
    *scale = __uint_as_float(0x7FC00000u);
    *inv = 0.f;
  } else {
    *scale = fmaxf(__uint_as_float(amax_bits) / 127.f, kMinScale);
    *inv = 1.f / *scale;
  }
}

__device__ __forceinline__ uint32_t code(float f, float inv) {
  // inv = 0 marks a row without finite scale
  return inv == 0.f ? 0u : static_cast<uint32_t>(static_cast<int>(rintf(f * inv))) & 0xFFu;
}

__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
  uint2 o;
  o.x = code(f[0], inv) | code(f[1], inv) << 8 | code(f[2], inv) << 16 | code(f[3], inv) << 24;
  o.y = code(f[4], inv) | code(f[5], inv) << 8 | code(f[6], inv) << 16 | code(f[7], inv) << 24;
  return o;
}

__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  float f[8];
  rows::Vec16<true>::unpack(v, f);
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = rows::Max::apply(top, abs_bits(f[j]));
  return top;
}

}  // namespace int8
}  // namespace moe
