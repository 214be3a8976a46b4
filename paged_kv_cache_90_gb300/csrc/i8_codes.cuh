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

// Largest of a warp's values, NaN aside (an order-preserving map to integers).
__device__ __forceinline__ float warp_max(float x) {
  const int i = __float_as_int(x == x ? x : -INFINITY);
  const int o = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
  return __int_as_float(o ^ ((o >> 31) & 0x7fffffff));
}

// The power of two at or above x > 0 (subnormal ones: the smallest normal; at most 2^127).
__device__ __forceinline__ float power_above(float x) {
  const uint32_t b = __float_as_uint(fmaxf(x, 0x1p-126f));
  return fminf(__uint_as_float((b & 0x7f800000u) + ((b & 0x7fffffu) ? 0x800000u : 0u)), 0x1p127f);
}

// The power of two that a query row with largest magnitude `top` is multiplied by before it
// becomes f16: 2^(14 - exponent of the largest), kept within 2^-100 .. 2^100.
__device__ __forceinline__ int query_shift(float top) {
  const int ex = int(__float_as_uint(top) >> 23) - 127;
  return top > 0.f && top < INFINITY ? max(-100, min(100, 14 - ex)) : 0;
}
__device__ __forceinline__ float power(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

}  // namespace i8
}  // namespace pkv
