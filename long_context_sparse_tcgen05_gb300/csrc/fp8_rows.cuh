// Row arithmetic shared by the kernels that norm, rotate and quantise: unpacking and packing of
// bf16, e4m3 rounding, magnitudes that keep a NaN, and the quotients by a row's scale.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

namespace dsa {

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
// two fp32 -> two e4m3 codes (lo in the low byte), round to nearest even, saturate finite
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// max(|a|, |b|, |c|), NaN if one of them is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// y / s for many y of a row, rounded as IEEE division rounds: with r the rounded reciprocal of s and
// a = fl(y r), the remainder y - a s is exact in one fma, and fl(a + r (y - a s)) is the rounded
// quotient (Markstein 1990, "Computation of elementary functions on the IBM RISC System/6000
// processor", theorem on division) -- three instructions a value.  It needs a quotient and a
// remainder inside the normal range: scales outside [2^-60, 2^60] (and NaN) divide; a quotient small
// enough for its remainder to be subnormal is far below the least e4m3 value.
// (with_quotient picks one of the two for a whole row.)
struct FastQuotient {
  float s, r;
  __device__ __forceinline__ float operator()(float y) const {
    const float a = y * r;
    return fmaf(fmaf(-a, s, y), r, a);
  }
};
struct PlainQuotient {
  float s;
  __device__ __forceinline__ float operator()(float y) const { return y / s; }
};
template <class F>
__device__ __forceinline__ void with_quotient(float s, F&& f) {
  if (s >= 0x1p-60f && s <= 0x1p60f) f(FastQuotient{s, 1.f / s});
  else f(PlainQuotient{s});
}

}  // namespace dsa
