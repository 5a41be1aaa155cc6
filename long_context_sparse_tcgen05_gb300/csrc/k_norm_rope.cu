// Per-head norm and rotary rotation in one pass, to bf16 or to e4m3 codes with one scale per token.
//
// A head row of d values is held by G lanes of a warp (G = 8, 16 or 32 by d), 8 values (16 bytes)
// per lane and unit, so the mean, the variance and the sum of squares are log2(G) shuffles of fp32
// partial sums.  The rotation needs each value's partner: interleaved pairs lie inside a unit;
// half-split pairs lie rope_dim / 2 values apart, in another lane of the group (heads up to 256
// wide), or are read a second time and normed with the same statistics (wider heads).
// x is read once and the result written once; the tables and weights are read from L1, once per lane
// for all the heads of a token.  Measured (device time, inputs of 3 calls past L2):
//   16,384 tokens x 64 x 128 to e4m3, half-split rotation   101 us, 4.0 TB/s: issue (61% of the slots, 141
//       instructions for a lane's 8 values, 12 of them quotients) and, at 24 warps an SM, the loads' latency; 260 us before
//       the next token's values were copied ahead and two values went into an instruction
//   8,192 tokens x 64 x 64 to bf16 among 576-wide rows      25.6 us, 5.3 TB/s (53% of the issue slots)
//   6,455 tokens x 20 x 96, RMS norm                        19.3 us, 2.6 TB/s: issue (68%); heads of 96
//       leave 4 of 16 lanes idle
// A warp or a CTA per token in the e4m3 form: the scale needs every head's values before the first code, and
// they stay in registers, so nothing is read twice.
#include <algorithm>

#include "dsa_internal.cuh"
#include "fp8_rows.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
static_assert(DSA_NORM_NONE == 0 && DSA_NORM_RMS == 1 && DSA_NORM_LAYER == 2, "kNorm below");

// A unit's 8 values, as pairs.
struct Vec8 {
  f32x2 p[4];
};

__device__ __forceinline__ Vec8 unpack8(uint4 r) {
  return {{unpack_bf16(r.x), unpack_bf16(r.y), unpack_bf16(r.z), unpack_bf16(r.w)}};
}
__device__ __forceinline__ uint4 pack8(const Vec8& y) {
  return make_uint4(pack_bf16(lo_of(y.p[0]), hi_of(y.p[0])), pack_bf16(lo_of(y.p[1]), hi_of(y.p[1])),
                    pack_bf16(lo_of(y.p[2]), hi_of(y.p[2])), pack_bf16(lo_of(y.p[3]), hi_of(y.p[3])));
}
__device__ __forceinline__ Vec8 load_f8(const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  return {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
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
// each, unit u of lane l at (u G + l) 8.  raw: zero where there is no unit.  inv_d: 1 / d (a division a
// head is a tenth of the work; half a step of the reciprocal is 2^-24 of the variance).
template <int kNorm, int G, int U>
__device__ __forceinline__ float2 head_stats(const NormRopeLaunch& p, const uint4 (&raw)[U], int l, float inv_d) {
  float mean = 0.f;
  if (kNorm == DSA_NORM_LAYER) {
    f32x2 s = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Vec8 x = unpack8(raw[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = add_2(s, x.p[e]);
    }
    mean = group_sum<G>(lo_of(s) + hi_of(s)) * inv_d;
  }
  f32x2 ss = 0;  // squares about the mean: no cancellation between mean^2 and the second moment
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if ((u * G + l) * 8 < p.d) {
      const Vec8 x = unpack8(raw[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x2 c = kNorm == DSA_NORM_LAYER ? add_2(x.p[e], pair(-mean, -mean)) : x.p[e];
        ss = fma_2(c, c, ss);
      }
    }
  }
  return make_float2(mean, rsqrtf(fmaf(group_sum<G>(lo_of(ss) + hi_of(ss)), inv_d, p.eps)));
}

// What a lane needs of a unit whatever its head: the norm's weights, and the factors of its rotation
// y <- y c + partner s (half-split: s negative in the first of a pair; interleaved: the partners are
// the pairs' other values, c = (cos, cos) and s = (-sin, sin)).
template <int kNorm>
struct UnitTables {
  f32x2 w[kNorm ? 4 : 1], b[kNorm == DSA_NORM_LAYER ? 4 : 1];
  Vec8 c, s;
  __device__ __forceinline__ void affine(const NormRopeLaunch& p, int at) {
    const f32x2 one = pair(1.f, 1.f);
    if constexpr (kNorm != DSA_NORM_NONE) {
      const Vec8 wv = p.weight ? load_f8(p.weight + at) : Vec8{{one, one, one, one}};
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = wv.p[e];
    }
    if constexpr (kNorm == DSA_NORM_LAYER) {
      const Vec8 bv = p.bias ? load_f8(p.bias + at) : Vec8{};
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = bv.p[e];
    }
  }
  __device__ __forceinline__ void angles(const NormRopeLaunch& p, int at, int64_t pos) {
    const int j = at - p.rope_off, half = p.rope_dim >> 1;
    if (p.interleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos + pos * half + (j >> 1)));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin + pos * half + (j >> 1)));
      c = {{pair(cv.x, cv.x), pair(cv.y, cv.y), pair(cv.z, cv.z), pair(cv.w, cv.w)}};
      s = {{pair(-sv.x, sv.x), pair(-sv.y, sv.y), pair(-sv.z, sv.z), pair(-sv.w, sv.w)}};
    } else {
      const int64_t at_t = pos * half + (j < half ? j : j - half);
      c = load_f8(p.cos + at_t);
      s = load_f8(p.sin + at_t);
      const f32x2 sign = j < half ? pair(-1.f, -1.f) : pair(1.f, 1.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) s.p[e] = mul_2(s.p[e], sign);
    }
  }
};

template <int kNorm>
__device__ __forceinline__ Vec8 normed(uint4 raw, float2 st, const UnitTables<kNorm>& t) {
  Vec8 y = unpack8(raw);
  const f32x2 f = pair(st.y, st.y), m = pair(-st.x, -st.x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (kNorm == DSA_NORM_RMS) y.p[e] = mul_2(mul_2(y.p[e], f), t.w[e]);
    if constexpr (kNorm == DSA_NORM_LAYER) y.p[e] = fma_2(mul_2(add_2(y.p[e], m), f), t.w[e], t.b[e]);
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

__device__ __forceinline__ void rotate(Vec8& y, const Vec8& partner, const Vec8& c, const Vec8& s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) y.p[e] = fma_2(partner.p[e], s.p[e], mul_2(y.p[e], c.p[e]));
}
__device__ __forceinline__ Vec8 swapped8(const Vec8& y) {
  return {{swapped(y.p[0]), swapped(y.p[1]), swapped(y.p[2]), swapped(y.p[3])}};
}

// The result of one unit of a head whose units are all in registers (U = 1): the partner comes from
// lane `src` of the group.  A whole warp calls it; lanes without a unit get what they do not use.
// turn: the unit is rotated.
template <int G, int kNorm>
__device__ __forceinline__ Vec8 unit_result(const NormRopeLaunch& p, uint4 raw, float2 st, int src, bool turn,
                                            const UnitTables<kNorm>& t) {
  Vec8 y = normed<kNorm>(raw, st, t), o{};
  if (p.rope_dim > 0) {
    if (p.interleaved) {
      o = swapped8(y);
    } else if constexpr (kNorm != DSA_NORM_NONE) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o.p[e] = pair(__shfl_sync(0xffffffffu, lo_of(y.p[e]), src, G), __shfl_sync(0xffffffffu, hi_of(y.p[e]), src, G));
    } else {  // as the packed values they came in
      uint4 q;
      q.x = __shfl_sync(0xffffffffu, raw.x, src, G);
      q.y = __shfl_sync(0xffffffffu, raw.y, src, G);
      q.z = __shfl_sync(0xffffffffu, raw.z, src, G);
      q.w = __shfl_sync(0xffffffffu, raw.w, src, G);
      o = unpack8(q);
    }
    if (turn) rotate(y, o, t.c, t.s);
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
    Vec8 o = swapped8(y);
    if (!p.interleaved) {
      UnitTables<kNorm> pt;
      pt.affine(p, partner_at(p, at));
      o = normed<kNorm>(partner, st, pt);
    }
    rotate(y, o, t.c, t.s);
  }
  return y;
}

// bf16 out.  A warp takes one token and R passes of 32 / G heads, whose loads are issued together.
template <int G, int U, int R, int kNorm>
__global__ void __launch_bounds__(kThreads, U == 1 ? 4 : 2) k_norm_rope_bf16(NormRopeLaunch p) {
  constexpr int kHeads = 32 / G;
  const int lane = threadIdx.x & 31, l = lane % G, hsub = lane / G;
  const float inv_d = 1.f / (float)p.d;
  const uint32_t chunks = (uint32_t)(p.H + kHeads * R - 1) / (kHeads * R);
  const uint32_t tasks = (uint32_t)p.B * p.n * chunks;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (kThreads / 32);
  UnitTables<kNorm> tab;
  if (U == 1 && l * 8 < p.d) tab.affine(p, l * 8);
  const bool turn = p.rope_dim > 0 && in_rope(p, l * 8);  // (U = 1: of this lane's unit)
  const int src = turn ? partner_at(p, l * 8) >> 3 : l;
  for (uint32_t task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks; task += step) {
    const uint32_t tok = task / chunks;
    const int h0 = (int)(task - tok * chunks) * kHeads * R + hsub;
    const int b = (int)(tok / (uint32_t)p.n), i = (int)(tok - (uint32_t)b * (uint32_t)p.n);
    const uint16_t* x = p.x + b * p.x_sb + i * p.x_st + h0 * p.x_sh;
    uint4 raw[R][U], par[R][U];
#pragma unroll
    for (int r = 0; r < R; ++r, x += kHeads * p.x_sh)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (u * G + l) * 8;
        const bool in = h0 + r * kHeads < p.H && at < p.d;
        // plain loads: out may be x
        raw[r][u] = in ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0, 0, 0, 0);
        par[r][u] = U > 1 && in && !p.interleaved && in_rope(p, at)
                        ? *reinterpret_cast<const uint4*>(x + partner_at(p, at))
                        : make_uint4(0, 0, 0, 0);
      }
    const int64_t pos = checked_pos(p, p.positions ? __ldg(p.positions + tok) : p.pos0 + i, lane == 0 && h0 == 0);
    if (pos < 0) continue;  // uniform over the warp
    if (U == 1 && turn) tab.angles(p, l * 8, pos);
    __syncwarp();  // in place: every load of these heads comes before their stores
    uint16_t* out = p.out + b * p.o_sb + i * p.o_st + h0 * p.o_sh;
#pragma unroll
    for (int r = 0; r < R; ++r, out += kHeads * p.o_sh) {
      if (h0 - hsub + r * kHeads >= p.H) break;  // (uniform over the warp)
      const float2 st = kNorm ? head_stats<kNorm, G, U>(p, raw[r], l, inv_d) : make_float2(0.f, 1.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (u * G + l) * 8;
        Vec8 y;
        if constexpr (U == 1) y = unit_result<G, kNorm>(p, raw[r][u], st, src, turn, tab);
        if (h0 + r * kHeads >= p.H || at >= p.d) continue;
        if constexpr (U > 1) y = unit_result_wide<kNorm>(p, raw[r][u], par[r][u], st, at, pos);
        *reinterpret_cast<uint4*>(out + at) = pack8(y);
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
  // each thread's units of the next token, copied while a token is worked on (not for the widest
  // tokens, whose registers hold them off the SM anyway)
  constexpr bool kAhead = NP * U <= 4;
  __shared__ uint4 ahead[kAhead ? 2 : 1][kAhead ? NP * U : 1][kThreads];
  constexpr int kTeams = kThreads / kTeam;  // tokens per CTA
  constexpr int kHeads = kTeam / G;         // heads per pass
  const int lane = threadIdx.x & 31, t = threadIdx.x % kTeam, l = t % G, hsub = t / G;
  const uint32_t toks = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  const float inv_d = 1.f / (float)p.d;
  UnitTables<kNorm> tab;
  if (U == 1 && l * 8 < p.d) tab.affine(p, l * 8);
  const bool turn = p.rope_dim > 0 && in_rope(p, l * 8);  // (U = 1: of this lane's unit)
  const int src = turn ? partner_at(p, l * 8) >> 3 : l;
  // every thread of a warp runs the same number of steps: the shuffles below take whole warps
  const uint32_t step = gridDim.x * kTeams;
  RowWalk at_row(blockIdx.x * kTeams + threadIdx.x / kTeam, step, p.n);
  // the next token's position is on its way while a token is worked on
  auto position = [&](uint32_t tok, uint32_t i) -> int64_t {
    if (tok >= toks) return -1;
    return p.positions ? __ldg(p.positions + tok) : p.pos0 + i;
  };
  const uint32_t first = blockIdx.x * kTeams + threadIdx.x / kTeam;
  int64_t next = position(first, at_row.i);
  // this thread's first unit of the token at row w, and its unit (s, u)
  const uint16_t* const mine = p.x + hsub * p.x_sh + l * 8;
  auto units_of = [&](const RowWalk& w) { return mine + w.b * p.x_sb + w.i * p.x_st; };
  auto unit_at = [&](const uint16_t* x, int s, int u) { return x + s * kHeads * p.x_sh + u * G * 8; };
  auto has_unit = [&](uint32_t tok, int s, int u) { return tok < toks && hsub + s * kHeads < p.H && (u * G + l) * 8 < p.d; };
  auto fetch = [&](uint32_t tok, const RowWalk& w, int slot) {
    if constexpr (kAhead) {
      const uint16_t* x = units_of(w);
#pragma unroll
      for (int s = 0; s < NP; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool in = has_unit(tok, s, u);
          copy16_async(&ahead[slot][s * U + u][threadIdx.x], in ? unit_at(x, s, u) : p.x, in);
        }
      copies_commit();
    }
  };
  fetch(first, at_row, 0);
  int slot = 0;
  for (uint32_t base = blockIdx.x * kTeams; base < toks; base += step) {
    const uint32_t tok = base + threadIdx.x / kTeam;
    const bool live = tok < toks;
    const int b = live ? (int)at_row.b : 0, i = live ? (int)at_row.i : 0;
    uint4 raw[NP][U];
    if constexpr (!kAhead) {
      const uint16_t* x = units_of(at_row);
#pragma unroll
      for (int s = 0; s < NP; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u)
          raw[s][u] = has_unit(tok, s, u) ? __ldg(reinterpret_cast<const uint4*>(unit_at(x, s, u))) : make_uint4(0, 0, 0, 0);
    }
    at_row.next();
    const int64_t pos = checked_pos(p, next, t == 0);
    next = position(tok + step, at_row.i);
    if (U == 1 && pos >= 0 && turn) tab.angles(p, l * 8, pos);
    if constexpr (kAhead) {
      fetch(tok + step, at_row, slot ^ 1);
      copies_wait<1>();
#pragma unroll
      for (int s = 0; s < NP; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) raw[s][u] = ahead[slot][s * U + u][threadIdx.x];
      slot ^= 1;
    }
    Vec8 y[NP][U];
    float amax = 0.f;  // (a NaN stays)
#pragma unroll
    for (int s = 0; s < NP; ++s) {
      const int h = hsub + s * kHeads;
      const float2 st = kNorm ? head_stats<kNorm, G, U>(p, raw[s], l, inv_d) : make_float2(0.f, 1.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (u * G + l) * 8;
        const bool in = pos >= 0 && h < p.H && at < p.d;
        if constexpr (U == 1) y[s][u] = unit_result<G, kNorm>(p, raw[s][u], st, src, turn, tab);
        if (!in) continue;
        if constexpr (U > 1) {
          const uint4 par = !p.interleaved && p.rope_dim > 0 && in_rope(p, at)
                                ? __ldg(reinterpret_cast<const uint4*>(p.x + b * p.x_sb + i * p.x_st + h * p.x_sh + partner_at(p, at)))
                                : make_uint4(0, 0, 0, 0);
          y[s][u] = unit_result_wide<kNorm>(p, raw[s][u], par, st, at, pos);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max3_abs(amax, lo_of(y[s][u].p[e]), hi_of(y[s][u].p[e]));
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
    uint8_t* codes = p.codes + dst * (int64_t)p.H * p.d + (int64_t)hsub * p.d + l * 8;
    with_quotient(scale, [&](auto div) {
#pragma unroll
      for (int s = 0; s < NP; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = hsub + s * kHeads, at = (u * G + l) * 8;
          if (h >= p.H || at >= p.d) continue;
          const f32x2* v = y[s][u].p;
          *reinterpret_cast<uint2*>(codes + s * kHeads * p.d + u * G * 8) = make_uint2(codes4(div, v[0], v[1]), codes4(div, v[2], v[3]));
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
