// Per-head norm and rotary rotation in one pass, to bf16 or to e4m3 codes with one scale per token.
//
// A head row of d values is held by G lanes of a warp (G = 8, 16 or 32 by d), 8 values (16 bytes)
// per lane and unit, so the mean, the variance and the sum of squares are log2(G) shuffles of fp32
// partial sums.  The rotation needs each value's partner: interleaved pairs lie inside a unit;
// half-split pairs lie rope_dim / 2 values apart, in another lane of the group (heads up to 256
// wide), or are read a second time and normed with the same statistics (wider heads).
// HBM-bound: x read once, the result written once; the tables and weights are read from L1, once
// per lane for all the heads of a token.
#include <algorithm>

#include "dsa_internal.cuh"
#include "fp8_rows.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
static_assert(DSA_NORM_NONE == 0 && DSA_NORM_RMS == 1 && DSA_NORM_LAYER == 2, "kNorm below");

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 unpack8(uint4 r) {
  return {{bf_lo(r.x), bf_hi(r.x), bf_lo(r.y), bf_hi(r.y), bf_lo(r.z), bf_hi(r.z), bf_lo(r.w), bf_hi(r.w)}};
}
__device__ __forceinline__ Vec8 load_f8(const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// A token's position, or -1 when the token is skipped.  p.limit: rows that a position may name (0:
// positions only mark padding).
__device__ __forceinline__ int64_t checked_pos(const NormRopeLaunch& p, int64_t pos, bool lead) {
  if (pos == -1) return -1;
  if (pos < 0 || (p.limit > 0 && pos >= p.limit)) {
    if (lead) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
    return -1;
  }
  return pos;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, G);
  return v;
}

// (mean, factor) with y = (x - mean) * factor * weight + bias, over a head held by G lanes as U units
// each, unit u of lane l at (u G + l) 8.  raw: zero where there is no unit.
template <int kNorm, int G, int U>
__device__ __forceinline__ float2 head_stats(const NormRopeLaunch& p, const uint4 (&raw)[U], int l) {
  float mean = 0.f;
  if (kNorm == DSA_NORM_LAYER) {
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
    if ((u * G + l) * 8 < p.d) {
      const Vec8 x = unpack8(raw[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += (x.v[e] - mean) * (x.v[e] - mean);
    }
  }
  ss = group_sum<G>(ss);
  return make_float2(mean, rsqrtf(ss / (float)p.d + p.eps));
}

// What a lane needs of a unit whatever its head: the norm's weights, and the cosines and sines of
// the unit's pairs (interleaved: four of each).
template <int kNorm>
struct UnitTables {
  float w[kNorm ? 8 : 1], b[kNorm == DSA_NORM_LAYER ? 8 : 1];
  Vec8 c, s;
  __device__ __forceinline__ void affine(const NormRopeLaunch& p, int at) {
    if constexpr (kNorm != DSA_NORM_NONE) {
      const Vec8 one{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
      const Vec8 wv = p.weight ? load_f8(p.weight + at) : one;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = wv.v[e];
    }
    if constexpr (kNorm == DSA_NORM_LAYER) {
      const Vec8 bv = p.bias ? load_f8(p.bias + at) : Vec8{};
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = bv.v[e];
    }
  }
  __device__ __forceinline__ void angles(const NormRopeLaunch& p, int at, int64_t pos) {
    const int j = at - p.rope_off, half = p.rope_dim >> 1;
    if (p.interleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos + pos * half + (j >> 1)));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin + pos * half + (j >> 1)));
      c.v[0] = cv.x, c.v[1] = cv.y, c.v[2] = cv.z, c.v[3] = cv.w;
      s.v[0] = sv.x, s.v[1] = sv.y, s.v[2] = sv.z, s.v[3] = sv.w;
    } else {
      const int64_t at_t = pos * half + (j < half ? j : j - half);
      c = load_f8(p.cos + at_t);
      s = load_f8(p.sin + at_t);
      if (j < half) {  // the first of a pair takes its partner's sine part away
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[e] = -s.v[e];
      }
    }
  }
};

template <int kNorm>
__device__ __forceinline__ Vec8 normed(uint4 raw, float2 st, const UnitTables<kNorm>& t) {
  Vec8 y = unpack8(raw);
  if constexpr (kNorm == DSA_NORM_RMS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] = y.v[e] * st.y * t.w[e];
  } else if constexpr (kNorm == DSA_NORM_LAYER) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] = (y.v[e] - st.x) * st.y * t.w[e] + t.b[e];
  }
  return y;
}

__device__ __forceinline__ bool in_rope(const NormRopeLaunch& p, int at) {
  return at >= p.rope_off && at < p.rope_off + p.rope_dim;
}
// Where the unit with the other halves of this unit's half-split pairs starts.
__device__ __forceinline__ int partner_at(const NormRopeLaunch& p, int at) {
  const int half = p.rope_dim >> 1;
  return at - p.rope_off < half ? at + half : at - half;
}

// Rotates a unit.  o: the (normed) values of its partner unit (half-split only).
template <int kNorm>
__device__ __forceinline__ void rotate(const NormRopeLaunch& p, Vec8& y, const Vec8& o, const UnitTables<kNorm>& t) {
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = y.v[2 * e], b = y.v[2 * e + 1];
      y.v[2 * e] = a * t.c.v[e] - b * t.s.v[e];
      y.v[2 * e + 1] = b * t.c.v[e] + a * t.s.v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] = y.v[e] * t.c.v[e] + o.v[e] * t.s.v[e];
  }
}

// The result of one unit of a head whose units are all in registers (U = 1): the partner comes from
// its lane.  A whole warp calls it; lanes without a unit get what they do not use.
template <int G, int kNorm>
__device__ __forceinline__ Vec8 unit_result(const NormRopeLaunch& p, uint4 raw, float2 st, int l, const UnitTables<kNorm>& t) {
  const int at = l * 8;
  Vec8 y = normed<kNorm>(raw, st, t), o{};
  if (p.rope_dim > 0) {
    const bool in = in_rope(p, at);
    if (!p.interleaved) {
      const int src = in ? partner_at(p, at) >> 3 : l;
      if constexpr (kNorm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = __shfl_sync(0xffffffffu, y.v[e], src, G);
      } else {  // as the packed values they came in
        uint4 q;
        q.x = __shfl_sync(0xffffffffu, raw.x, src, G);
        q.y = __shfl_sync(0xffffffffu, raw.y, src, G);
        q.z = __shfl_sync(0xffffffffu, raw.z, src, G);
        q.w = __shfl_sync(0xffffffffu, raw.w, src, G);
        o = unpack8(q);
      }
    }
    if (in) rotate<kNorm>(p, y, o, t);
  }
  return y;
}
// The same for a head of several units a lane: the partner unit is read again.
template <int kNorm>
__device__ __forceinline__ Vec8 unit_result_wide(const NormRopeLaunch& p, uint4 raw, uint4 partner, float2 st, int at,
                                                 int64_t pos) {
  UnitTables<kNorm> t;
  t.affine(p, at);
  Vec8 y = normed<kNorm>(raw, st, t);
  if (p.rope_dim > 0 && in_rope(p, at)) {
    t.angles(p, at, pos);
    Vec8 o{};
    if (!p.interleaved) {
      UnitTables<kNorm> pt;
      pt.affine(p, partner_at(p, at));
      o = normed<kNorm>(partner, st, pt);
    }
    rotate<kNorm>(p, y, o, t);
  }
  return y;
}

// bf16 out.  A warp takes one token and R passes of 32 / G heads, whose loads are issued together.
template <int G, int U, int R, int kNorm>
__global__ void __launch_bounds__(kThreads, U == 1 ? 4 : 2) k_norm_rope_bf16(NormRopeLaunch p) {
  constexpr int kHeads = 32 / G;
  const int lane = threadIdx.x & 31, l = lane % G, hsub = lane / G;
  const uint32_t chunks = (uint32_t)(p.H + kHeads * R - 1) / (kHeads * R);
  const uint32_t tasks = (uint32_t)p.B * p.n * chunks;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (kThreads / 32);
  UnitTables<kNorm> tab;
  if (U == 1 && l * 8 < p.d) tab.affine(p, l * 8);
  for (uint32_t task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks; task += step) {
    const uint32_t tok = task / chunks;
    const int h0 = (int)(task - tok * chunks) * kHeads * R + hsub;
    const int b = (int)(tok / (uint32_t)p.n), i = (int)(tok - (uint32_t)b * (uint32_t)p.n);
    const uint16_t* x = p.x + b * p.x_sb + i * p.x_st;
    uint4 raw[R][U], par[R][U];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + r * kHeads, at = (u * G + l) * 8;
        const bool in = h < p.H && at < p.d;
        // plain loads: out may be x
        raw[r][u] = in ? *reinterpret_cast<const uint4*>(x + h * p.x_sh + at) : make_uint4(0, 0, 0, 0);
        par[r][u] = U > 1 && in && !p.interleaved && in_rope(p, at)
                        ? *reinterpret_cast<const uint4*>(x + h * p.x_sh + partner_at(p, at))
                        : make_uint4(0, 0, 0, 0);
      }
    const int64_t pos = checked_pos(p, p.positions ? __ldg(p.positions + tok) : p.pos0 + i, lane == 0 && h0 == 0);
    if (pos < 0) continue;  // uniform over the warp
    if (U == 1 && p.rope_dim > 0 && in_rope(p, l * 8)) tab.angles(p, l * 8, pos);
    __syncwarp();  // in place: every load of these heads comes before their stores
    uint16_t* out = p.out + b * p.o_sb + i * p.o_st;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = h0 + r * kHeads;
      const float2 st = kNorm ? head_stats<kNorm, G, U>(p, raw[r], l) : make_float2(0.f, 1.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (u * G + l) * 8;
        Vec8 y;
        if constexpr (U == 1) y = unit_result<G, kNorm>(p, raw[r][u], st, l, tab);
        if (h >= p.H || at >= p.d) continue;
        if constexpr (U > 1) y = unit_result_wide<kNorm>(p, raw[r][u], par[r][u], st, at, pos);
        *reinterpret_cast<uint4*>(out + h * p.o_sh + at) = make_uint4(pack_bf16(y.v[0], y.v[1]), pack_bf16(y.v[2], y.v[3]),
                                                                      pack_bf16(y.v[4], y.v[5]), pack_bf16(y.v[6], y.v[7]));
      }
    }
  }
}

// e4m3 out.  A token belongs to a team: a group of G lanes (one head), a warp (all its heads in
// one pass) or the CTA (NP passes over the heads); the team holds the whole result in registers,
// takes its largest magnitude and divides.
template <int G, int U, int NP, int kTeam, int kNorm>
__global__ void __launch_bounds__(kThreads, NP * U >= 8 ? 1 : 3) k_norm_rope_e4m3(NormRopeLaunch p) {
  __shared__ float team_max[kThreads / 32];
  constexpr int kTeams = kThreads / kTeam;  // tokens per CTA
  constexpr int kHeads = kTeam / G;         // heads per pass
  const int lane = threadIdx.x & 31, t = threadIdx.x % kTeam, l = t % G, hsub = t / G;
  const uint32_t toks = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  UnitTables<kNorm> tab;
  if (U == 1 && l * 8 < p.d) tab.affine(p, l * 8);
  // every thread of a warp runs the same number of steps: the shuffles below take whole warps
  const uint32_t step = gridDim.x * kTeams;
  // the next token's position is on its way while a token is worked on
  auto position = [&](uint32_t tok) -> int64_t {
    if (tok >= toks) return -1;
    return p.positions ? __ldg(p.positions + tok) : p.pos0 + tok % (uint32_t)p.n;
  };
  int64_t next = position(blockIdx.x * kTeams + threadIdx.x / kTeam);
  for (uint32_t base = blockIdx.x * kTeams; base < toks; base += step) {
    const uint32_t tok = base + threadIdx.x / kTeam;
    const bool live = tok < toks;
    const int b = live ? (int)(tok / (uint32_t)p.n) : 0, i = live ? (int)(tok - (uint32_t)b * (uint32_t)p.n) : 0;
    const uint16_t* x = p.x + b * p.x_sb + i * p.x_st;
    uint4 raw[NP][U];
#pragma unroll
    for (int s = 0; s < NP; ++s)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hsub + s * kHeads, at = (u * G + l) * 8;
        const bool in = live && h < p.H && at < p.d;
        raw[s][u] = in ? __ldg(reinterpret_cast<const uint4*>(x + h * p.x_sh + at)) : make_uint4(0, 0, 0, 0);
      }
    const int64_t pos = checked_pos(p, next, t == 0);
    next = position(tok + step);
    if (U == 1 && pos >= 0 && p.rope_dim > 0 && in_rope(p, l * 8)) tab.angles(p, l * 8, pos);
    Vec8 y[NP][U];
    float amax = 0.f;  // (a NaN stays)
#pragma unroll
    for (int s = 0; s < NP; ++s) {
      const int h = hsub + s * kHeads;
      const float2 st = kNorm ? head_stats<kNorm, G, U>(p, raw[s], l) : make_float2(0.f, 1.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (u * G + l) * 8;
        const bool in = pos >= 0 && h < p.H && at < p.d;
        if constexpr (U == 1) y[s][u] = unit_result<G, kNorm>(p, raw[s][u], st, l, tab);
        if (!in) continue;
        if constexpr (U > 1) {
          const uint4 par = !p.interleaved && p.rope_dim > 0 && in_rope(p, at)
                                ? __ldg(reinterpret_cast<const uint4*>(x + h * p.x_sh + partner_at(p, at)))
                                : make_uint4(0, 0, 0, 0);
          y[s][u] = unit_result_wide<kNorm>(p, raw[s][u], par, st, at, pos);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) amax = max3_abs(amax, y[s][u].v[e], y[s][u].v[e + 1]);
      }
    }
    constexpr int kShfl = kTeam < 32 ? kTeam : 32;
#pragma unroll
    for (int o = kShfl / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o, kShfl));
    if (kTeam > 32) {
      __syncthreads();  // the previous token's maxima have been read
      if (lane == 0) team_max[threadIdx.x >> 5] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) amax = max_nan(amax, team_max[w]);
    }
    if (pos < 0) continue;  // (uniform over the team; a CTA-wide team agrees before its barriers)
    const float q = amax / 448.f;
    const float scale = q == 0.f ? 1.f : q;  // (a NaN stays)
    const int64_t dst = (int64_t)b * p.S_cap + (p.at_position ? pos : i);
    uint8_t* codes = p.codes + dst * (int64_t)p.H * p.d;
    with_quotient(scale, [&](auto div) {
#pragma unroll
      for (int s = 0; s < NP; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = hsub + s * kHeads, at = (u * G + l) * 8;
          if (h >= p.H || at >= p.d) continue;
          const float* v = y[s][u].v;
          const uint32_t lo = pack_e4m3(div(v[0]), div(v[1])) | pack_e4m3(div(v[2]), div(v[3])) << 16;
          const uint32_t hi = pack_e4m3(div(v[4]), div(v[5])) | pack_e4m3(div(v[6]), div(v[7])) << 16;
          *reinterpret_cast<uint2*>(codes + (int64_t)h * p.d + at) = make_uint2(lo, hi);
        }
    });
    if (t == 0) p.scales[dst] = scale;
  }
}

template <int G, int U, int kNorm>
void launch_e4m3(const NormRopeLaunch& p, int64_t cap, cudaStream_t st) {
  const int64_t toks = (int64_t)p.B * p.n;
  const int lanes = p.H * G;
  auto grid = [&](int64_t per_cta) { return (int)std::min<int64_t>((toks + per_cta - 1) / per_cta, cap); };
  if (p.H == 1) k_norm_rope_e4m3<G, U, 1, G, kNorm><<<grid(kThreads / G), kThreads, 0, st>>>(p);
  else if (lanes <= 32 && G < 32) k_norm_rope_e4m3<G, U, 1, G < 32 ? 32 : 256, kNorm><<<grid(kThreads / 32), kThreads, 0, st>>>(p);
  else if (lanes <= 256) k_norm_rope_e4m3<G, U, 1, 256, kNorm><<<grid(1), kThreads, 0, st>>>(p);
  else if (lanes <= 512) k_norm_rope_e4m3<G, U, 2, 256, kNorm><<<grid(1), kThreads, 0, st>>>(p);
  else if constexpr (U == 1) {
    if (lanes <= 1024) k_norm_rope_e4m3<G, U, 4, 256, kNorm><<<grid(1), kThreads, 0, st>>>(p);
    else k_norm_rope_e4m3<G, U, 8, 256, kNorm><<<grid(1), kThreads, 0, st>>>(p);
  }
}

template <int G, int U, int R, int kNorm>
void launch_bf16(const NormRopeLaunch& p, int64_t cap, cudaStream_t st) {
  const int per = (32 / G) * R;
  const int64_t tasks = (int64_t)p.B * p.n * ((p.H + per - 1) / per);
  const int grid = (int)std::min<int64_t>((tasks + kThreads / 32 - 1) / (kThreads / 32), cap);
  k_norm_rope_bf16<G, U, R, kNorm><<<grid, kThreads, 0, st>>>(p);
}

template <int kNorm>
void launch(const NormRopeLaunch& p, int64_t cap, cudaStream_t st) {
  if (p.out) {
    if (p.d <= 64) launch_bf16<8, 1, 4, kNorm>(p, cap, st);
    else if (p.d <= 128) launch_bf16<16, 1, 4, kNorm>(p, cap, st);
    else if (p.d <= 256) launch_bf16<32, 1, 4, kNorm>(p, cap, st);
    else if (p.d <= 512) launch_bf16<32, 2, 2, kNorm>(p, cap, st);
    else launch_bf16<32, 4, 1, kNorm>(p, cap, st);
  } else {
    if (p.d <= 64) launch_e4m3<8, 1, kNorm>(p, cap, st);
    else if (p.d <= 128) launch_e4m3<16, 1, kNorm>(p, cap, st);
    else if (p.d <= 256) launch_e4m3<32, 1, kNorm>(p, cap, st);
    else launch_e4m3<32, 4, kNorm>(p, cap, st);
  }
}

}  // namespace

// 8-value units of a head, padded: lanes x units per lane that hold it in the e4m3 kernels.
int norm_rope_units(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : 128; }

cudaError_t launch_norm_rope(const NormRopeLaunch& p, cudaStream_t st) {
  if (p.B == 0 || p.n == 0) return cudaSuccess;
  TraceScope trace(kTraceCache, st);
  const int64_t cap = (int64_t)device_sm_count() * 16;
  if (p.norm == DSA_NORM_NONE) launch<DSA_NORM_NONE>(p, cap, st);
  else if (p.norm == DSA_NORM_RMS) launch<DSA_NORM_RMS>(p, cap, st);
  else launch<DSA_NORM_LAYER>(p, cap, st);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dsa
