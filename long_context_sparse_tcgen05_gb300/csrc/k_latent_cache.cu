// The paged FP8 latent cache: appending rows (norm, rotation, quantisation and the write through
// the block table in one pass) and reading rows back.  A warp takes a token: 16 latent values per
// lane (two 16-byte loads) and one rotated pair, so the sum of squares and the largest magnitude
// are warp shuffles.  HBM-bound: 1,152 bytes in and 644 out per appended token (the other way
// round to read), plus a 256-byte table row.
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_internal.cuh"
#include "latent_cache.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr float kMinScale = 0x1p-60f;  // rope / scale stays finite in bf16 for any sane rope value

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

__global__ void __launch_bounds__(kThreads) k_latent_append(LatentAppendLaunch p) {
  const int lane = threadIdx.x & 31;
  float w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = p.weight ? __ldg(p.weight + (e < 8 ? 0 : 256) + lane * 8 + (e & 7)) : 1.f;
  const int64_t toks = (int64_t)p.B * p.n;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t tok = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); tok < toks; tok += step) {
    const int b = (int)(tok / p.n), i = (int)(tok - (int64_t)b * p.n);
    const int64_t pos = p.positions ? p.positions[tok] : p.pos0 + i;
    if (pos == -1) continue;
    const int64_t row = pos >= 0 && (!p.cos || pos < p.max_pos) ? latent_row(p.cache, b, pos) : -1;
    if (row < 0) {
      if (lane == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
      continue;
    }
    const uint16_t* x = p.x + b * p.x_sb + i * p.x_st;
    const uint4 r0 = __ldg(reinterpret_cast<const uint4*>(x) + lane);
    const uint4 r1 = __ldg(reinterpret_cast<const uint4*>(x) + 32 + lane);
    // rope pair `lane`: values (2 lane, 2 lane + 1) or (lane, lane + 32)
    const uint16_t* xr = x + kLatentDim;
    float a, c;
    if (p.interleaved) {
      const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(xr) + lane);
      a = bf_lo(v);
      c = bf_hi(v);
    } else {
      a = bf_lo(__ldg(xr + lane));
      c = bf_lo(__ldg(xr + 32 + lane));
    }
    float cs = 1.f, sn = 0.f;
    if (p.cos) {
      cs = __ldg(p.cos + pos * 32 + lane);
      sn = __ldg(p.sin + pos * 32 + lane);
    }
    float y[16] = {bf_lo(r0.x), bf_hi(r0.x), bf_lo(r0.y), bf_hi(r0.y), bf_lo(r0.z), bf_hi(r0.z), bf_lo(r0.w), bf_hi(r0.w),
                   bf_lo(r1.x), bf_hi(r1.x), bf_lo(r1.y), bf_hi(r1.y), bf_lo(r1.z), bf_hi(r1.z), bf_lo(r1.w), bf_hi(r1.w)};
    if (p.weight) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss += y[e] * y[e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float f = rsqrtf(ss * (1.f / kLatentDim) + p.eps);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = y[e] * f * w[e];
    }
    uint32_t amax = 0;  // magnitude bits: a NaN is above every number and so is kept
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = max(amax, __float_as_uint(y[e]) & 0x7fffffffu);
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float q = __uint_as_float(amax) / 448.f;
    const float scale = q < kMinScale ? kMinScale : q;  // (a NaN stays)
    uint32_t k[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      k[e] = e4m3x2(y[4 * e] / scale, y[4 * e + 1] / scale) | e4m3x2(y[4 * e + 2] / scale, y[4 * e + 3] / scale) << 16;
    uint8_t* codes = p.cache.codes + row * kLatentDim;
    *reinterpret_cast<uint2*>(codes + lane * 8) = make_uint2(k[0], k[1]);
    *reinterpret_cast<uint2*>(codes + 256 + lane * 8) = make_uint2(k[2], k[3]);
    const float ra = (a * cs - c * sn) / scale, rc = (c * cs + a * sn) / scale;
    uint16_t* rope = p.cache.rope + row * kLatentRope;
    if (p.interleaved) {
      reinterpret_cast<uint32_t*>(rope)[lane] = pack2(ra, rc);
    } else {
      rope[lane] = (uint16_t)pack2(ra, 0.f);
      rope[32 + lane] = (uint16_t)pack2(rc, 0.f);
    }
    if (lane == 0) p.cache.scales[row] = scale;
  }
}

// Eight codes (two words) times the scale, as bf16.
__device__ __forceinline__ uint4 dequant8(uint2 c, float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_to_float2((uint16_t)((i < 2 ? c.x : c.y) >> ((i & 1) * 16)));
    o[i] = pack2(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kThreads) k_latent_read(LatentReadLaunch p) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)p.B * p.n;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += step) {
    const int b = (int)(r / p.n), i = (int)(r - (int64_t)b * p.n);
    const int64_t pos = p.idx ? (int64_t)__ldg(p.idx + r) : p.pos0 + i;
    const int64_t row = pos >= 0 ? latent_row(p.cache, b, pos) : -1;
    uint4* out = reinterpret_cast<uint4*>(p.out + r * (kLatentDim + kLatentRope));
    if (row < 0) {
      if (pos != -1 && lane == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
      out[lane] = out[32 + lane] = make_uint4(0, 0, 0, 0);
      if (lane < 8) out[64 + lane] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint2* codes = reinterpret_cast<const uint2*>(p.cache.codes + row * kLatentDim);
    const uint2 c0 = __ldg(codes + lane), c1 = __ldg(codes + 32 + lane);
    uint4 rp = make_uint4(0, 0, 0, 0);
    if (lane < 8) rp = __ldg(reinterpret_cast<const uint4*>(p.cache.rope + row * kLatentRope) + lane);
    const float s = __ldg(p.cache.scales + row);
    out[lane] = dequant8(c0, s);
    out[32 + lane] = dequant8(c1, s);
    if (lane < 8)
      out[64 + lane] = make_uint4(pack2(bf_lo(rp.x) * s, bf_hi(rp.x) * s), pack2(bf_lo(rp.y) * s, bf_hi(rp.y) * s),
                                  pack2(bf_lo(rp.z) * s, bf_hi(rp.z) * s), pack2(bf_lo(rp.w) * s, bf_hi(rp.w) * s));
  }
}

int grid_of(int64_t rows) {
  return (int)std::min<int64_t>((rows + kThreads / 32 - 1) / (kThreads / 32), (int64_t)device_sm_count() * 8);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendLaunch& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.n;
  if (rows == 0) return cudaSuccess;
  TraceScope trace(kTraceCache, st);
  k_latent_append<<<grid_of(rows), kThreads, 0, st>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_latent_read(const LatentReadLaunch& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.n;
  if (rows == 0) return cudaSuccess;
  TraceScope trace(kTraceCache, st);
  k_latent_read<<<grid_of(rows), kThreads, 0, st>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dsa
