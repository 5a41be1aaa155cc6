// Addressing and decoding of the paged FP8 latent cache on the device.
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

}  // namespace dsa
