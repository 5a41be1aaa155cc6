// Sparse attention over selected rows of the paged FP8 latent cache.
//
// One CTA per (query, eight heads): a warp holds a head.  Blocks of 32 selected rows are
// dequantised into shared memory; each lane forms its head's score with one row, the warp takes
// the block's maximum and sum (running maximum, fp32), and each thread accumulates two of the 512
// value columns for the eight heads.
#include <cuda_bf16.h>

#include "dsa_internal.cuh"
#include "latent_cache.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256, kHeads = 8, kKeys = 32, kD = kLatentDim + kLatentRope;
constexpr int kLd = kD + 1;  // row pitch in floats: lanes reading one column of 32 rows hit 32 banks
constexpr size_t kSmem = (size_t)(kKeys * kLd + kHeads * kD + kHeads * kKeys + 2 * kHeads) * 4;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__global__ void __launch_bounds__(kThreads) k_latent_attn(LatentAttnLaunch p) {
  extern __shared__ float sm[];
  float* rows = sm;                     // [kKeys][kLd]
  float* q = rows + kKeys * kLd;        // [kHeads][kD]
  float* prob = q + kHeads * kD;        // [kHeads][kKeys]
  float* alpha = prob + kHeads * kKeys; // [kHeads]
  float* rsum = alpha + kHeads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int b = (int)(blockIdx.x / p.T), t = (int)(blockIdx.x % p.T), h0 = blockIdx.y * kHeads;
  const int32_t* idx = p.idx + b * p.idx_sb + t * p.idx_st;
  const uint16_t* qg = p.q + b * p.q_sb + t * p.q_st;
  for (int i = tid; i < kHeads * kD; i += kThreads) q[i] = h0 + i / kD < p.H ? bf(qg[(int64_t)h0 * kD + i]) : 0.f;
  float m = -INFINITY, l = 0.f;
  float acc[kHeads][2] = {};
  for (int j0 = 0; j0 < p.kk; j0 += kKeys) {
    __syncthreads();
    uint32_t valid = 0;
    {
      const int e = j0 + lane;
      const int id = e < p.kk ? idx[e] : -1;
      const int64_t row = id >= 0 && id < p.S ? latent_row(p.cache, b, id) : -1;
      if (row < 0 && id != -1 && warp == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
      valid = __ballot_sync(0xffffffffu, row >= 0);
      for (int r = warp; r < kKeys; r += kThreads / 32) {
        const int64_t rr = __shfl_sync(0xffffffffu, row, r);
        float* dst = rows + r * kLd;
        if (rr < 0) {
          for (int c = lane; c < kD; c += 32) dst[c] = 0.f;
          continue;
        }
        const float s = p.cache.scales[rr];
        for (int c = lane; c < kLatentDim / 2; c += 32) {
          const float2 f = e4m3x2_to_float2(reinterpret_cast<const uint16_t*>(p.cache.codes + rr * kLatentDim)[c]);
          dst[2 * c] = f.x * s;
          dst[2 * c + 1] = f.y * s;
        }
        for (int c = lane; c < kLatentRope; c += 32) dst[kLatentDim + c] = bf(p.cache.rope[rr * kLatentRope + c]) * s;
      }
    }
    __syncthreads();
    if (valid == 0) continue;  // the same in every warp
    float s = 0.f;
    for (int c = 0; c < kD; ++c) s += q[warp * kD + c] * rows[lane * kLd + c];
    s = (valid >> lane) & 1u ? s * p.scale : -INFINITY;
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float a = __expf(m - mu), pr = (valid >> lane) & 1u ? __expf(s - mu) : 0.f;
    float sum = pr;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * a + sum;
    m = mn;
    prob[warp * kKeys + lane] = pr;
    if (lane == 0) alpha[warp] = a;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      acc[h][0] *= alpha[h];
      acc[h][1] *= alpha[h];
    }
    for (int r = 0; r < kKeys; ++r) {
      if (!((valid >> r) & 1u)) continue;
      const float v0 = rows[r * kLd + tid], v1 = rows[r * kLd + tid + 256];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        acc[h][0] += prob[h * kKeys + r] * v0;
        acc[h][1] += prob[h * kKeys + r] * v1;
      }
    }
  }
  if (lane == 0) {
    rsum[warp] = l == 0.f ? 0.f : 1.f / l;
    if (p.lse && h0 + warp < p.H) p.lse[(int64_t)blockIdx.x * p.H + h0 + warp] = l == 0.f ? -INFINITY : m + logf(l);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (h0 + h >= p.H) break;
    uint16_t* o = p.out + ((int64_t)blockIdx.x * p.H + h0 + h) * kLatentDim;
    const float r = rsum[h];
    o[tid] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[h][0] * r));
    o[tid + 256] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[h][1] * r));
  }
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnLaunch& p, cudaStream_t st) {
  TraceScope trace(kTraceAttention, st);
  cudaError_t e = cudaFuncSetAttribute(k_latent_attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  k_latent_attn<<<dim3((unsigned)(p.B * p.T), (unsigned)((p.H + kHeads - 1) / kHeads)), kThreads, kSmem, st>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dsa
