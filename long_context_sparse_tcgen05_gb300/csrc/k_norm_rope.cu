// Per-head norm and rotary rotation in one pass, to bf16 or to e4m3 codes with one scale per token.
//
// A head row of d values is held by G lanes of a warp (G = 4, 8, 16 or 32 by d), 8 values (16
// bytes) per lane and unit, so the mean, the variance and the sum of squares are log2(G) shuffles
// of fp32 partial sums.  The rotation needs each value's partner: interleaved pairs lie inside a
// unit, half-split pairs rope_dim / 2 values apart, whose unit is read a second time (an L1 hit)
// and normed with the same statistics -- one load in place of eight shuffles.
// HBM-bound: x read once, the result written once; the tables and weights are read from L1.
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_internal.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ Vec8 unpack8(uint4 r) {
  return {{bf_lo(r.x), bf_hi(r.x), bf_lo(r.y), bf_hi(r.y), bf_lo(r.z), bf_hi(r.z), bf_lo(r.w), bf_hi(r.w)}};
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ Vec8 load_f8(const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Position of token (b, i); < 0 when the token is skipped.  limit: rows that a position may name
// (0: positions only mark padding).
__device__ __forceinline__ int64_t token_pos(const NormRopeLaunch& p, int b, int i, bool lead) {
  const int64_t pos = p.positions ? p.positions[(int64_t)b * p.n + i] : p.pos0 + i;
  if (pos == -1) return -1;
  if (pos < 0 || (p.limit > 0 && pos >= p.limit)) {
    if (lead) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
    return -1;
  }
  return pos;
}

// Values of a lane's units: where each unit starts within the head, and whether it exists.
template <int G, int U>
struct Lane {
  int l;  // lane within the head's group
  __device__ __forceinline__ int at(int u) const { return (u * G + l) * 8; }
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, G);
  return v;
}

// (mean, factor) with y = (x - mean) * factor * weight + bias.  raw: the lane's units, zero where
// there is none.
template <int G, int U>
__device__ __forceinline__ float2 head_stats(const NormRopeLaunch& p, const uint4 (&raw)[U], Lane<G, U> ln) {
  if (p.norm == DSA_NORM_NONE) return make_float2(0.f, 1.f);
  float mean = 0.f;
  if (p.norm == DSA_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Vec8 x = unpack8(raw[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x.v[e];
    }
    mean = group_sum<G>(s) / (float)p.d;
  }
  float ss = 0.f;  // squares about the mean: no cancellation between mean^2 and the second moment
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (ln.at(u) < p.d) {
      const Vec8 x = unpack8(raw[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += (x.v[e] - mean) * (x.v[e] - mean);
    }
  }
  ss = group_sum<G>(ss);
  return make_float2(mean, rsqrtf(ss / (float)p.d + p.eps));
}

__device__ __forceinline__ Vec8 normed(const NormRopeLaunch& p, uint4 raw, float2 st, int at) {
  Vec8 y = unpack8(raw);
  if (p.norm == DSA_NORM_NONE) return y;
#pragma unroll
  for (int e = 0; e < 8; ++e) y.v[e] = (y.v[e] - st.x) * st.y;
  if (p.weight) {
    const Vec8 w = load_f8(p.weight + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] *= w.v[e];
  }
  if (p.bias) {
    const Vec8 b = load_f8(p.bias + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] += b.v[e];
  }
  return y;
}

// Rotates the normed unit at `at` of a head whose row starts at xrow.  partner: the raw unit that
// holds the other halves of its pairs (half-split only).
__device__ __forceinline__ void rotate(const NormRopeLaunch& p, Vec8& y, uint4 partner, float2 st, int at, int64_t pos) {
  const int j = at - p.rope_off, half = p.rope_dim >> 1;
  if (p.interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + pos * half + (j >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + pos * half + (j >> 1)));
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = y.v[2 * e], b = y.v[2 * e + 1];
      y.v[2 * e] = a * cv[e] - b * sv[e];
      y.v[2 * e + 1] = b * cv[e] + a * sv[e];
    }
  } else {
    const bool first = j < half;
    const Vec8 o = normed(p, partner, st, first ? at + half : at - half);
    const int t = first ? j : j - half;
    const Vec8 c = load_f8(p.cos + pos * half + t), s = load_f8(p.sin + pos * half + t);
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] = y.v[e] * c.v[e] + (first ? -o.v[e] : o.v[e]) * s.v[e];
  }
}

__device__ __forceinline__ bool in_rope(const NormRopeLaunch& p, int at) {
  return at >= p.rope_off && at < p.rope_off + p.rope_dim;
}
__device__ __forceinline__ int partner_at(const NormRopeLaunch& p, int at) {
  const int half = p.rope_dim >> 1;
  return at - p.rope_off < half ? at + half : at - half;
}

// bf16 out.  A warp takes one token and 32 / G heads at a time, R passes of heads whose loads are
// issued together.
template <int G, int U, int R>
__global__ void __launch_bounds__(kThreads) k_norm_rope_bf16(NormRopeLaunch p) {
  constexpr int kHeads = 32 / G;
  const int lane = threadIdx.x & 31;
  const Lane<G, U> ln{lane % G};
  const int hsub = lane / G;
  const int chunks = (p.H + kHeads * R - 1) / (kHeads * R);
  const int64_t tasks = (int64_t)p.B * p.n * chunks;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t task = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks; task += step) {
    const int64_t tok = task / chunks;
    const int h0 = (int)(task - tok * chunks) * kHeads * R + hsub;
    const int b = (int)(tok / p.n), i = (int)(tok - (int64_t)b * p.n);
    const int64_t pos = token_pos(p, b, i, lane == 0 && h0 == 0);
    if (pos < 0) continue;  // uniform over the warp
    const uint16_t* x = p.x + b * p.x_sb + i * p.x_st;
    uint4 raw[R][U], par[R][U];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + r * kHeads, at = ln.at(u);
        const bool in = h < p.H && at < p.d;
        // plain loads: out may be x
        raw[r][u] = in ? *reinterpret_cast<const uint4*>(x + h * p.x_sh + at) : make_uint4(0, 0, 0, 0);
        par[r][u] = in && !p.interleaved && in_rope(p, at)
                        ? *reinterpret_cast<const uint4*>(x + h * p.x_sh + partner_at(p, at))
                        : make_uint4(0, 0, 0, 0);
      }
    __syncwarp();  // in place: every load of these heads comes before their stores
    uint16_t* out = p.out + b * p.o_sb + i * p.o_st;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = h0 + r * kHeads;
      const float2 st = head_stats<G, U>(p, raw[r], ln);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = ln.at(u);
        if (h >= p.H || at >= p.d) continue;
        Vec8 y = normed(p, raw[r][u], st, at);
        if (in_rope(p, at)) rotate(p, y, par[r][u], st, at, pos);
        *reinterpret_cast<uint4*>(out + h * p.o_sh + at) =
            make_uint4(pack2(y.v[0], y.v[1]), pack2(y.v[2], y.v[3]), pack2(y.v[4], y.v[5]), pack2(y.v[6], y.v[7]));
      }
    }
  }
}

// e4m3 out.  A token belongs to a team: a group of G lanes (one head), a warp (all its heads in
// one pass) or the CTA (NP passes over the heads); the team holds the whole result in registers,
// takes its largest magnitude and divides.
template <int G, int U, int NP, int kTeam>
__global__ void __launch_bounds__(kThreads) k_norm_rope_e4m3(NormRopeLaunch p) {
  __shared__ float team_max[kThreads / 32];
  const int lane = threadIdx.x & 31;
  constexpr int kTeams = kThreads / kTeam;  // tokens per CTA
  constexpr int kHeads = kTeam / G;         // heads per pass
  const int t = threadIdx.x % kTeam;
  const Lane<G, U> ln{t % G};
  const int hsub = t / G;
  const int64_t toks = (int64_t)p.B * p.n;
  // every thread of a warp runs the same number of steps: the shuffles below take whole warps
  const int64_t step = (int64_t)gridDim.x * kTeams;
  for (int64_t base = (int64_t)blockIdx.x * kTeams; base < toks; base += step) {
    const int64_t tok = base + threadIdx.x / kTeam;
    const bool live = tok < toks;
    const int b = live ? (int)(tok / p.n) : 0, i = live ? (int)(tok - (int64_t)b * p.n) : 0;
    const int64_t pos = live ? token_pos(p, b, i, t == 0) : -1;
    const uint16_t* x = p.x + b * p.x_sb + i * p.x_st;
    uint4 raw[NP][U], par[NP][U];
#pragma unroll
    for (int s = 0; s < NP; ++s)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hsub + s * kHeads, at = ln.at(u);
        const bool in = pos >= 0 && h < p.H && at < p.d;
        raw[s][u] = in ? __ldg(reinterpret_cast<const uint4*>(x + h * p.x_sh + at)) : make_uint4(0, 0, 0, 0);
        par[s][u] = in && !p.interleaved && in_rope(p, at)
                        ? __ldg(reinterpret_cast<const uint4*>(x + h * p.x_sh + partner_at(p, at)))
                        : make_uint4(0, 0, 0, 0);
      }
    Vec8 y[NP][U];
    uint32_t amax = 0;  // magnitude bits: a NaN is above every number and so is kept
#pragma unroll
    for (int s = 0; s < NP; ++s) {
      const float2 st = head_stats<G, U>(p, raw[s], ln);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = ln.at(u);
        if (pos >= 0 && hsub + s * kHeads < p.H && at < p.d) {
          y[s][u] = normed(p, raw[s][u], st, at);
          if (in_rope(p, at)) rotate(p, y[s][u], par[s][u], st, at, pos);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(y[s][u].v[e]) & 0x7fffffffu);
        }
      }
    }
    constexpr int kShfl = kTeam < 32 ? kTeam : 32;
#pragma unroll
    for (int o = kShfl / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o, kShfl));
    if (kTeam > 32) {
      __syncthreads();  // the previous token's maxima have been read
      if (lane == 0) team_max[threadIdx.x >> 5] = __uint_as_float(amax);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) amax = max(amax, __float_as_uint(team_max[w]));
    }
    if (pos < 0) continue;  // (uniform over the team; a CTA-wide team agrees before its barriers)
    const float q = __uint_as_float(amax) / 448.f;
    const float scale = q == 0.f ? 1.f : q;  // (a NaN stays)
    const int64_t dst = (int64_t)b * p.S_cap + (p.at_position ? pos : i);
    uint8_t* codes = p.codes + dst * (int64_t)p.H * p.d;
#pragma unroll
    for (int s = 0; s < NP; ++s)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hsub + s * kHeads, at = ln.at(u);
        if (h >= p.H || at >= p.d) continue;
        const float* v = y[s][u].v;
        const uint32_t lo = e4m3x2(v[0] / scale, v[1] / scale) | e4m3x2(v[2] / scale, v[3] / scale) << 16;
        const uint32_t hi = e4m3x2(v[4] / scale, v[5] / scale) | e4m3x2(v[6] / scale, v[7] / scale) << 16;
        *reinterpret_cast<uint2*>(codes + (int64_t)h * p.d + at) = make_uint2(lo, hi);
      }
    if (t == 0) p.scales[dst] = scale;
  }
}

template <int G, int U>
void launch_e4m3(const NormRopeLaunch& p, int64_t cap, cudaStream_t st) {
  const int64_t toks = (int64_t)p.B * p.n;
  const int lanes = p.H * G;
  auto grid = [&](int64_t per_cta) { return (int)std::min<int64_t>((toks + per_cta - 1) / per_cta, cap); };
  if (p.H == 1) k_norm_rope_e4m3<G, U, 1, G><<<grid(kThreads / G), kThreads, 0, st>>>(p);
  else if (lanes <= 32) k_norm_rope_e4m3<G, U, 1, 32><<<grid(kThreads / 32), kThreads, 0, st>>>(p);
  else if (lanes <= 256) k_norm_rope_e4m3<G, U, 1, 256><<<grid(1), kThreads, 0, st>>>(p);
  else if (lanes <= 512) k_norm_rope_e4m3<G, U, 2, 256><<<grid(1), kThreads, 0, st>>>(p);
  else if constexpr (U <= 2) {
    if (lanes <= 1024) k_norm_rope_e4m3<G, U, 4, 256><<<grid(1), kThreads, 0, st>>>(p);
    else if constexpr (U == 1) k_norm_rope_e4m3<G, U, 8, 256><<<grid(1), kThreads, 0, st>>>(p);
  }
}

template <int G, int U, int R>
void launch_bf16(const NormRopeLaunch& p, int64_t cap, cudaStream_t st) {
  const int per = (32 / G) * R;
  const int64_t tasks = (int64_t)p.B * p.n * ((p.H + per - 1) / per);
  const int grid = (int)std::min<int64_t>((tasks + kThreads / 32 - 1) / (kThreads / 32), cap);
  k_norm_rope_bf16<G, U, R><<<grid, kThreads, 0, st>>>(p);
}

}  // namespace

// 8-value units of a head, padded: lanes x units per lane that hold it.
int norm_rope_units(int d) {
  return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : d <= 512 ? 64 : 128;
}

cudaError_t launch_norm_rope(const NormRopeLaunch& p, cudaStream_t st) {
  if (p.B == 0 || p.n == 0) return cudaSuccess;
  TraceScope trace(kTraceCache, st);
  const int64_t cap = (int64_t)device_sm_count() * 16;
  if (p.out) {
    if (p.d <= 32) launch_bf16<4, 1, 4>(p, cap, st);
    else if (p.d <= 64) launch_bf16<8, 1, 4>(p, cap, st);
    else if (p.d <= 128) launch_bf16<16, 1, 4>(p, cap, st);
    else if (p.d <= 256) launch_bf16<32, 1, 4>(p, cap, st);
    else if (p.d <= 512) launch_bf16<32, 2, 2>(p, cap, st);
    else launch_bf16<32, 4, 1>(p, cap, st);
  } else {
    switch (norm_rope_units(p.d)) {
      case 4: launch_e4m3<4, 1>(p, cap, st); break;
      case 8: launch_e4m3<8, 1>(p, cap, st); break;
      case 16: launch_e4m3<16, 1>(p, cap, st); break;
      case 32: launch_e4m3<32, 1>(p, cap, st); break;
      case 64: launch_e4m3<32, 2>(p, cap, st); break;
      default: launch_e4m3<32, 4>(p, cap, st); break;
    }
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dsa
