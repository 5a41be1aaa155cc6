// Addressing and decoding of the paged latent cache, FP8 or 4-bit, on the device.
#pragma once
#include <cuda_fp16.h>

#include "dsa_internal.cuh"

namespace dsa {

// Flat cache row of position pos >= 0 of sequence b, in two steps, so that a caller may put work between
// the load of the table entry and its use.
// The page (of a contiguous cache: the sequence) and the position in it; off = -1: past the sequence's rows.
__device__ __forceinline__ int latent_page(const LatentCacheView& c, int b, int64_t pos, int& off) {
  if (pos >= c.cap) {
    off = -1;
    return -1;
  }
  if (!c.table) {
    off = (int)pos;
    return b;
  }
  const uint32_t p = (uint32_t)pos, in_seq = p / (uint32_t)c.page_size;
  off = (int)(p - in_seq * (uint32_t)c.page_size);
  return __ldg(c.table + (int64_t)b * c.table_ld + in_seq);
}
// Its row, or -1: a block table entry that is no page.
__device__ __forceinline__ int64_t latent_row_of(const LatentCacheView& c, int page, int off) {
  if (c.table && (page < 0 || page >= c.n_pages)) return -1;
  return (int64_t)page * c.page_size + off;
}
__device__ __forceinline__ int64_t latent_row(const LatentCacheView& c, int b, int64_t pos) {
  int off;
  const int page = latent_page(c, b, pos, off);
  return off < 0 ? -1 : latent_row_of(c, page, off);
}

// Two e4m3 codes (low byte first) as floats; every e4m3 value is an f16 value.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// ---- the 4-bit cache: e2m1 codes (sign, two bits of exponent, one of fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6) under a
// group's byte b = e + 127, -5 <= e <= 6.  Every code times 2^e is an e4m3 value: of the magnitudes above 0.5 to 6 the
// e4m3 codes are c - 8, c, c + 4, c + 8, c + 12, c + 16, c + 20, with c = 8 (e + 7) the code of 2^e itself (their
// exponents go by steps of 8, their halves by 4; c - 8 >= 8, so all of them are normal).

// Eight e2m1 codes (low four bits first) as pairs of f16.
__device__ __forceinline__ void unpack_e2m1(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}
// Four pairs of floats as eight codes (the nearest, ties to even, at most 6).
__device__ __forceinline__ uint32_t pack_e2m1(const float2 (&z)[4]) {
  uint32_t codes;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(codes)
      : "f"(z[0].x), "f"(z[0].y), "f"(z[1].x), "f"(z[1].y), "f"(z[2].x), "f"(z[2].y), "f"(z[3].x), "f"(z[3].y));
  return codes;
}
// Eight e2m1 codes (low four bits first) to the e4m3 codes of what they stand for: the eight magnitudes are a table in
// two registers that a byte permutation looks up, four codes at a time.
struct ExpandFour {
  uint32_t lo, hi;  // magnitudes 0-3 and 4-7
  __device__ __forceinline__ explicit ExpandFour(uint32_t group) {
    // (four bits of the byte count: any byte gives finite values)
    const uint32_t c = ((group - 122u) & 15u) * 0x08080808u + 0x10101010u;
    lo = (c & 0xffffff00u) + 0x03fff800u;  // [0, c - 8, c, c + 4]
    hi = c + 0x14100c08u;                  // [c + 8, c + 12, c + 16, c + 20]
  }
  __device__ __forceinline__ uint2 operator()(uint32_t w) const {
    const uint32_t m = w & 0x77777777u, t = w << 4;  // magnitudes; the even codes' signs at their bytes' tops
    return make_uint2(__byte_perm(lo, hi, m) | (__byte_perm(t, w, 0x5140) & 0x80808080u),
                      __byte_perm(lo, hi, m >> 16) | (__byte_perm(t, w, 0x7362) & 0x80808080u));
  }
};

}  // namespace dsa
