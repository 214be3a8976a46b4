// e2m1_codes.cuh — 4-bit codes and their group scales: encoding (the cache writes) and
// decoding (reads and attention).
//
// A code is a sign, two exponent bits of bias 1 and one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4,
// 6.  A scale for 16 columns is an e4m3 number, of four significant bits and at least 2^-9, so
// code * scale has at most six and is an f16 number, exactly.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"

namespace pkv {
namespace e2m1 {

// Eight codes (a word, code 0 in the low bits) -> four f16 pairs, exact, the lower code in the
// lower half.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Four codes in the low half of a word -> floats, exact.
__device__ __forceinline__ void widen4(uint32_t w, float* f) {
  uint32_t a, b;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(a), "=r"(b) : "r"(w));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}

// A group scale's byte (e4m3), and two of them side by side, as numbers.
__device__ __forceinline__ uint32_t scales2(uint32_t two) {  // an f16 pair
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ float scale1(uint32_t byte) {
  const uint32_t h = scales2(byte);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// A cache's factor f, and division by 6 f.  (Made once where it serves all rows: the reciprocal in it
// costs more than the rest of a group's scale; the rotary write makes it for each row.)
struct Factor {
  float f;
  DivRn six;
  __device__ __forceinline__ explicit Factor(float x) : f(x), six(6.f * x) {}
};

// The scale of a group whose largest magnitude has the bits `top`, and what its elements are
// multiplied by.  A factor that puts the step out of the normal numbers stores zeros.
struct Group {
  uint32_t byte;
  float inverse;  // 0: all codes are 0
  __device__ __forceinline__ Group(uint32_t top, const Factor& x) {
    const float g = fminf(x.six(__uint_as_float(top)), 448.f);
    byte = __nv_cvt_float_to_fp8(g, __NV_SATFINITE, __NV_E4M3);
    const float step = __fmul_rn(scale1(byte), x.f);
    const bool number = step >= 0x1p-126f && step <= 0x1p126f;
    inverse = number ? __frcp_rn(step) : 0.f;
    if (!number) byte = 0;
    if (top >= 0x7f800000u) {  // an infinity or a NaN in the group
      byte = 0x7f;
      inverse = 0.f;
    }
  }
};

// Eight elements of one group -> a word of codes.
__device__ __forceinline__ uint32_t encode8(const float* x, const Group& g) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(__fmul_rn(x[0], g.inverse)), "f"(__fmul_rn(x[1], g.inverse)), "f"(__fmul_rn(x[2], g.inverse)),
        "f"(__fmul_rn(x[3], g.inverse)), "f"(__fmul_rn(x[4], g.inverse)), "f"(__fmul_rn(x[5], g.inverse)),
        "f"(__fmul_rn(x[6], g.inverse)), "f"(__fmul_rn(x[7], g.inverse)));
  return g.inverse != 0.f ? w : 0u;
}

}  // namespace e2m1
}  // namespace pkv
