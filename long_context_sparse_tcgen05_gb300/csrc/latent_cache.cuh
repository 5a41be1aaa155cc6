// Addressing and decoding of the paged FP8 latent cache on the device.
#pragma once
#include <cuda_fp16.h>

#include "dsa_internal.cuh"

namespace dsa {

// Flat cache row of position pos >= 0 of sequence b, or -1: past the sequence's rows, or a block
// table entry that is no page.
__device__ __forceinline__ int64_t latent_row(const LatentCacheView& c, int b, int64_t pos) {
  if (pos >= c.cap) return -1;
  if (!c.table) return (int64_t)b * c.page_size + pos;
  const uint32_t p = (uint32_t)pos, in_seq = p / (uint32_t)c.page_size;
  const int page = __ldg(c.table + (int64_t)b * c.table_ld + in_seq);
  if (page < 0 || page >= c.n_pages) return -1;
  return (int64_t)page * c.page_size + (p - in_seq * (uint32_t)c.page_size);
}

// Two e4m3 codes (low byte first) as floats; every e4m3 value is an f16 value.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

}  // namespace dsa
