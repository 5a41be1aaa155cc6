// The paged FP8 latent cache: appending rows (norm, rotation, quantisation and the write through
// the block table in one pass) and reading rows back.  A warp takes a token: 16 latent values per
// lane (two 16-byte loads) and one rotated pair, so the sum of squares and the largest magnitude
// are warp shuffles.  HBM-bound: 1,152 bytes in and 644 out per appended token (the other way
// round to read), plus a 256-byte table row.
#include <algorithm>

#include "dsa_internal.cuh"
#include "fp8_rows.cuh"
#include "latent_cache.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr float kMinScale = 0x1p-60f;  // rope / scale stays finite in bf16 for any sane rope value

__global__ void __launch_bounds__(kThreads) k_latent_append(LatentAppendLaunch p) {
  const int lane = threadIdx.x & 31;
  const uint32_t toks = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (kThreads / 32);
  uint32_t tok = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  RowWalk at_row(tok, step, p.n);
  // the next token's position is on its way while a token is worked on
  int64_t next = p.positions && tok < toks ? __ldg(p.positions + tok) : 0;
  for (; tok < toks; tok += step, at_row.next()) {
    const int b = (int)at_row.b, i = (int)at_row.i;
    // the row's values do not wait for its position and its page
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
    const int64_t pos = p.positions ? next : p.pos0 + i;
    if (p.positions && tok + step < toks) next = __ldg(p.positions + tok + step);
    if (pos == -1) continue;
    const int64_t row = pos >= 0 && (!p.cos || pos < p.max_pos) ? latent_row(p.cache, b, pos) : -1;
    if (row < 0) {
      if (lane == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
      continue;
    }
    float cs = 1.f, sn = 0.f;
    if (p.cos) {
      cs = __ldg(p.cos + pos * 32 + lane);
      sn = __ldg(p.sin + pos * 32 + lane);
    }
    f32x2 y[8] = {unpack_bf16(r0.x), unpack_bf16(r0.y), unpack_bf16(r0.z), unpack_bf16(r0.w),
                  unpack_bf16(r1.x), unpack_bf16(r1.y), unpack_bf16(r1.z), unpack_bf16(r1.w)};
    if (p.weight) {
      f32x2 s2 = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) s2 = fma_2(y[e], y[e], s2);
      float ss = lo_of(s2) + hi_of(s2);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float f = rsqrtf(ss * (1.f / kLatentDim) + p.eps);
      const f32x2 f2 = pair(f, f);
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {  // (from L1: 16 registers held for them cost a CTA per SM)
        const float4 w = __ldg(reinterpret_cast<const float4*>(p.weight + (e4 >> 1) * 256 + lane * 8) + (e4 & 1));
        y[2 * e4] = mul_2(mul_2(y[2 * e4], f2), pair(w.x, w.y));
        y[2 * e4 + 1] = mul_2(mul_2(y[2 * e4 + 1], f2), pair(w.z, w.w));
      }
    }
    float amax = 0.f;  // (a NaN stays)
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max3_abs(amax, lo_of(y[e]), hi_of(y[e]));
    // (the bits of a magnitude, NaN on top, order as integers)
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    const float q = amax / 448.f;
    const float scale = q < kMinScale ? kMinScale : q;  // (a NaN stays)
    with_quotient(scale, [&](auto div) {
      uint8_t* codes = p.cache.codes + row * kLatentDim;
      *reinterpret_cast<uint2*>(codes + lane * 8) = make_uint2(codes4(div, y[0], y[1]), codes4(div, y[2], y[3]));
      *reinterpret_cast<uint2*>(codes + 256 + lane * 8) = make_uint2(codes4(div, y[4], y[5]), codes4(div, y[6], y[7]));
      const f32x2 r = div(pair(a * cs - c * sn, c * cs + a * sn));
      const uint32_t rr = pack_bf16(lo_of(r), hi_of(r));
      uint16_t* rope = p.cache.rope + row * kLatentRope;
      if (p.interleaved) {
        reinterpret_cast<uint32_t*>(rope)[lane] = rr;
      } else {
        rope[lane] = (uint16_t)rr;
        rope[32 + lane] = (uint16_t)(rr >> 16);
      }
    });
    if (lane == 0) p.cache.scales[row] = scale;
  }
}

// Eight codes (two words) times the scale, as bf16.
__device__ __forceinline__ uint4 dequant8(uint2 c, float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_to_float2((uint16_t)((i < 2 ? c.x : c.y) >> ((i & 1) * 16)));
    o[i] = pack_bf16(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kThreads) k_latent_read(LatentReadLaunch p) {
  const int lane = threadIdx.x & 31;
  const uint32_t rows = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (kThreads / 32);
  for (uint32_t r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += step) {
    const int b = (int)(r / (uint32_t)p.n), i = (int)(r - (uint32_t)b * (uint32_t)p.n);
    const int64_t pos = p.idx ? (int64_t)__ldg(p.idx + r) : p.pos0 + i;
    const int64_t row = pos >= 0 ? latent_row(p.cache, b, pos) : -1;
    uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)r * (kLatentDim + kLatentRope));
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
      out[64 + lane] = make_uint4(pack_bf16(bf_lo(rp.x) * s, bf_hi(rp.x) * s), pack_bf16(bf_lo(rp.y) * s, bf_hi(rp.y) * s),
                                  pack_bf16(bf_lo(rp.z) * s, bf_hi(rp.z) * s), pack_bf16(bf_lo(rp.w) * s, bf_hi(rp.w) * s));
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
