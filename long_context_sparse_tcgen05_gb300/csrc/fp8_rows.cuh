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

// ---- pairs of fp32 in one 64-bit register: one instruction for two values ---------------------
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float lo_of(f32x2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(f32x2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ f32x2 swapped(f32x2 v) { return pair(hi_of(v), lo_of(v)); }
__device__ __forceinline__ f32x2 mul_2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add_2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma_2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// the two bf16 of a word
__device__ __forceinline__ f32x2 unpack_bf16(uint32_t v) { return pair(bf_lo(v), bf_hi(v)); }

// y / s for many y of a row, rounded as IEEE division rounds: with r the rounded reciprocal of s and
// a = fl(y r), the remainder y - a s is exact in one fma, and fl(a + r (y - a s)) is the rounded
// quotient (Markstein 1990, "Computation of elementary functions on the IBM RISC System/6000
// processor", theorem on division) -- three instructions a pair.  It needs a quotient and a remainder
// inside the normal range, and gives NaN where the quotient is infinite.  So it is for values that the
// row's scale bounds, and for scales in [2^-60, 2^60] (others, and NaN, divide): of those a quotient too
// small for its remainder is far below the least e4m3 value.  Values that the scale does not bound go
// through any_quotient.  (with_quotient picks one of the two for a whole row.)
struct FastQuotient {
  f32x2 minus_s, r;
  __device__ __forceinline__ explicit FastQuotient(float s) : minus_s(pair(-s, -s)) {
    const float q = 1.f / s;
    r = pair(q, q);
  }
  __device__ __forceinline__ f32x2 operator()(f32x2 y) const {
    const f32x2 a = mul_2(y, r);
    return fma_2(fma_2(a, minus_s, y), r, a);
  }
};
struct PlainQuotient {
  float s;
  __device__ __forceinline__ f32x2 operator()(f32x2 y) const { return pair(lo_of(y) / s, hi_of(y) / s); }
};
template <class F>
__device__ __forceinline__ void with_quotient(float s, F&& f) {
  if (s >= 0x1p-60f && s <= 0x1p60f) f(FastQuotient(s));
  else f(PlainQuotient{s});
}
// y / s where s does not bound y: the division itself for a pair that has a value outside [2^-60, 2^60]
// (zeros, infinities and NaN among them), whose quotient may pass the range the correction needs.
template <class Q>
__device__ __forceinline__ f32x2 any_quotient(const Q& q, f32x2 y, float s) {
  const float lo = fabsf(lo_of(y)), hi = fabsf(hi_of(y));
  return max_nan(lo, hi) <= 0x1p60f && fminf(lo, hi) >= 0x1p-60f ? q(y) : PlainQuotient{s}(y);
}
// four quotients as e4m3 codes
template <class Q>
__device__ __forceinline__ uint32_t codes4(const Q& q, f32x2 a, f32x2 b) {
  const f32x2 x = q(a), y = q(b);
  return pack_e4m3(lo_of(x), hi_of(x)) | pack_e4m3(lo_of(y), hi_of(y)) << 16;
}

// Row r of a grid-stride walk over [B, n] rows as (sequence, row in it), without a division a step.
struct RowWalk {
  uint32_t b, i, db, di, n;
  __device__ __forceinline__ RowWalk(uint32_t r, uint32_t step, uint32_t rows_per_seq)
      : b(r / rows_per_seq), i(r - b * rows_per_seq), db(step / rows_per_seq), di(step - db * rows_per_seq), n(rows_per_seq) {}
  __device__ __forceinline__ void next() {
    b += db;
    i += di;
    if (i >= n) i -= n, ++b;
  }
};

// 16 bytes from global to shared memory behind the thread's back (zeros where !in), groups of them,
// and the wait for all but the newest N groups.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

}  // namespace dsa
