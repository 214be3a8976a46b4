// i8_codes.cuh — int8 codes as f16 operands, and the query and value scaling that the
// attention kernels over token-scaled caches share.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"

namespace pkv {
namespace i8 {

__device__ __forceinline__ uint32_t minus_1152(uint32_t w) {
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&w), off);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Four int8 codes, each with its top bit flipped -> four f16 values, exact: code + 128 in the
// low byte of 0x64.. is 1152 + code in f16.
__device__ __forceinline__ uint2 widen4_flipped(uint32_t u) {
  return make_uint2(minus_1152(__byte_perm(u, 0x64646464u, 0x4140)), minus_1152(__byte_perm(u, 0x64646464u, 0x4342)));
}
__device__ __forceinline__ uint32_t flip4(uint32_t w) { return w ^ 0x80808080u; }
__device__ __forceinline__ uint2 widen4(uint32_t w) { return widen4_flipped(flip4(w)); }

// A weight times its token's value scale is an f16 operand.  A row's weights are 2^(z - m +
// kTopWeight) with m the largest z + scale_exponent of the tokens that it sees: the products
// then reach 2^kTopWeight and, with a reference that lags by 2^8 and a scale's fraction below 2,
// stay under 2^15.  The weights themselves and their sum are binary32; a product smaller than
// 2^-20 of the row's largest is a subnormal f16 number, off by at most 2^-31 of that.
constexpr float kTopWeight = 6.f;

// floor(log2 |s|) of a value scale; that of 2^-80 for smaller ones, 0 among them, so that a weight
// is below 2^(14 + 80) and a sum of 2^30 of them a binary32 number.  (Scales below 2^-100 lose
// bits, as do sums beside scales above 2^90: 2^-126 is the smallest weight.)  What is no number
// moves no reference.
__device__ __forceinline__ float scale_exponent(float s) {
  const float a = fabsf(s), b = a < INFINITY ? fmaxf(a, 0x1p-80f) : 0x1p-80f;
  return float(int(__float_as_uint(b) >> 23) - 127);
}

// The power of two that a query row with largest magnitude `top` is multiplied by before it
// becomes f16: 2^(14 - exponent of the largest), which is at least 2^-113, and at most 2^126, whose
// inverse is a normal number (the smallest bf16 number, 2^-133, then becomes 2^-7).
__device__ __forceinline__ int query_shift(float top) {
  const int ex = int(__float_as_uint(top) >> 23) - 127;
  return top > 0.f && top < INFINITY ? min(126, 14 - ex) : 0;
}
__device__ __forceinline__ float power(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

}  // namespace i8
}  // namespace pkv
