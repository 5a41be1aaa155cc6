// The paged latent cache, FP8 or 4-bit: appending rows (norm, rotation, quantisation and the write through
// the block table in one pass) and reading rows back.  FP8:  a warp takes a token: 16 latent values per
// lane (two 16-byte loads) and one rotated pair, so the sum of squares and the largest magnitude
// are warp shuffles.  HBM-bound: 1,152 bytes in and 644 out per appended token (the other way
// round to read), plus a 256-byte table row.  Measured: 131,072 tokens appended in 55.6 us (4.9 TB/s;
// 75% of the issue slots, 370 instructions a token, 27 of them quotients) and read back in 41.2 us
// (5.7 TB/s); 32 x 2,048 selected rows read in 22.6 us (5.2 TB/s); one token each of 32 sequences appended
// in 3.5 us.
// 4-bit (404 bytes a row): 131,072 tokens appended in 47 us (5.0 TB/s, 69% of the issue slots, 295 instructions a token), read
// back in 34.6 us (5.9 TB/s), unpacked to FP8 rows in 24.6 us (5.6 TB/s); 32 x 2,048 selected rows read in 17.5 us (5.9 TB/s).
#include <algorithm>

#include "dsa_internal.cuh"
#include "fp8_rows.cuh"
#include "latent_cache.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr float kMinScale = 0x1p-60f;  // rope / scale stays finite in bf16 for any sane rope value

// Everything a token needs is on its way while the one before it is worked on: its 1,152 bytes in
// the warp's part of shared memory, its angles and block table entry in registers (its position one
// token earlier still).  Loaded when its turn came, a token took a warp three dependent loads.
// kTurn: with rotation tables.  (Without them the rope values stay as they are: an angle of zero, 1 and 0,
// would spread an infinity or NaN over its pair.  Chosen inside the kernel it cost 59.5, not 58.2 us.)
template <bool kTurn>
__global__ void __launch_bounds__(kThreads) k_latent_append(LatentAppendLaunch p) {
  constexpr int kRow = kLatentDim + kLatentRope;
  __shared__ alignas(16) uint16_t rows[2][kThreads / 32][kRow];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t toks = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (kThreads / 32), first = blockIdx.x * (kThreads / 32) + warp;
  struct Ahead {
    int64_t pos;      // -1: skipped, -2: to be flagged
    int64_t in_page;  // offset in the page (without a table: the cache row)
    int page;
    float cs, sn;
  };
  auto position = [&](uint32_t tok, uint32_t i) -> int64_t {
    if (tok >= toks) return -1;
    return p.positions ? __ldg(p.positions + tok) : p.pos0 + i;
  };
  auto fetch = [&](uint32_t tok, const RowWalk& w, int64_t pos, int slot) -> Ahead {
    Ahead a{pos, 0, 0, 1.f, 0.f};
    const uint16_t* x = tok < toks ? p.x + w.b * p.x_sb + w.i * p.x_st : p.x;
    uint16_t* dst = rows[slot][warp];
    copy16_async(dst + 8 * lane, x + 8 * lane, tok < toks);
    copy16_async(dst + 256 + 8 * lane, x + 256 + 8 * lane, tok < toks);
    if (lane < 8) copy16_async(dst + 512 + 8 * lane, x + 512 + 8 * lane, tok < toks);
    copies_commit();
    if (pos == -1) return a;
    if (pos < 0 || pos >= p.cache.cap || (kTurn && pos >= p.max_pos)) {
      a.pos = -2;
      return a;
    }
    if (p.cache.table) {
      const uint32_t in_seq = (uint32_t)pos / (uint32_t)p.cache.page_size;
      a.in_page = (uint32_t)pos - in_seq * (uint32_t)p.cache.page_size;
      a.page = __ldg(p.cache.table + (int64_t)w.b * p.cache.table_ld + in_seq);
    } else {
      a.page = (int)w.b;
      a.in_page = pos;
    }
    if (kTurn) {
      a.cs = __ldg(p.cos + pos * 32 + lane);
      a.sn = __ldg(p.sin + pos * 32 + lane);
    }
    return a;
  };
  RowWalk w(first, step, p.n);
  Ahead nxt = fetch(first, w, position(first, w.i), 0);
  w.next();
  int64_t pos_next = position(first + step, w.i);
  int slot = 0;
  for (uint32_t tok = first; tok < toks; tok += step, slot ^= 1) {
    const Ahead now = nxt;
    nxt = fetch(tok + step, w, pos_next, slot ^ 1);
    w.next();
    pos_next = position(tok + 2 * step, w.i);
    copies_wait<1>();
    __syncwarp();
    const uint16_t* x = rows[slot][warp];
    const uint4 r0 = *reinterpret_cast<const uint4*>(x + 8 * lane), r1 = *reinterpret_cast<const uint4*>(x + 256 + 8 * lane);
    // rope pair `lane`: values (2 lane, 2 lane + 1) or (lane, lane + 32)
    const uint16_t* xr = x + kLatentDim + (p.interleaved ? 2 * lane : lane);
    const float a = bf_lo(xr[0]), c = bf_lo(xr[p.interleaved ? 1 : 32]);
    __syncwarp();  // the slot may be filled again
    if (now.pos == -1) continue;
    if (now.pos < 0 || now.page < 0 || now.page >= p.cache.n_pages) {
      if (lane == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
      continue;
    }
    const int64_t row = (int64_t)now.page * p.cache.page_size + now.in_page;
    const float cs = now.cs, sn = now.sn;
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
      // (the scale is the latent values': it does not bound these)
      const f32x2 r = any_quotient(div, kTurn ? pair(a * cs - c * sn, c * cs + a * sn) : pair(a, c), scale);
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

constexpr float kTopFour = 384.f;  // 6 * 2^6: the largest e2m1 value under the largest group factor
// The byte of a group whose largest magnitude over the row's scale is m: b - 127 = e, the least of -5 .. 6 with
// 6 * 2^e = 1.5 * 2^(e + 2) >= m.  (A fraction above a half carries into the exponent.)
__device__ __forceinline__ uint32_t group_of(float m) {
  const int e = (int)((__float_as_uint(m) + 0x3fffffu) >> 23) - 127 - 2;
  return (uint32_t)(min(max(e, -5), 6) + 127);
}

// Into the 4-bit cache, two tokens a warp: a lane has the 32 values of one group of one of them, so a group's largest
// value is the lane's own, a row's sums and maximum take four shuffles, and what a token costs beside its values is paid
// once for two.  (A warp a token, as in the FP8 kernel: 62 us for 131,072 rows; this one 47.  Rows copied two or three turns
// ahead instead of one: no faster.)  As there, everything a token
// needs is on its way while the one before it is worked on.  The 16-byte pieces of a row lie in shared memory so that
// eight lanes, each reading from its own 64 bytes, meet all banks; so do the weights.
template <bool kTurn>
__global__ void __launch_bounds__(kThreads, 3) k_latent4_append(LatentAppendLaunch p) {
  constexpr int kRow = kLatentDim + kLatentRope, kWarps = kThreads / 32;
  __shared__ alignas(16) uint16_t rows[2][kWarps][2][kRow];
  __shared__ alignas(16) float weights[kLatentDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15, half = lane >> 4;
  if (p.weight) {  // (four floats c of group g at 8 g + (c ^ (g & 7)))
    for (int i = threadIdx.x; i < kLatentDim / 4; i += kThreads)
      reinterpret_cast<float4*>(weights)[(i & ~7) | ((i ^ (i >> 3)) & 7)] = __ldg(reinterpret_cast<const float4*>(p.weight) + i);
    __syncthreads();
  }
  const uint32_t toks = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (2 * kWarps), first = (blockIdx.x * kWarps + warp) * 2 + half;
  struct Ahead {
    int64_t pos;      // -1: skipped, -2: to be flagged
    int64_t in_page;  // offset in the page (without a table: the cache row)
    int page;
    float2 cs, sn;
  };
  auto position = [&](uint32_t tok, uint32_t i) -> int64_t {
    if (tok >= toks) return -1;
    return p.positions ? __ldg(p.positions + tok) : p.pos0 + i;
  };
  auto fetch = [&](uint32_t tok, const RowWalk& w, int64_t pos, int slot) -> Ahead {
    Ahead a{pos, 0, 0, make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
    const bool in = tok < toks;
    const uint16_t* x = in ? p.x + w.b * p.x_sb + w.i * p.x_st : p.x;
    uint16_t* dst = rows[slot][warp][half];
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // piece k = 4 g + c of the row, of group g
      const int k = 16 * q + l;
      copy16_async(dst + 8 * ((k & ~3) | ((k ^ (k >> 3)) & 3)), x + 8 * k, in);
    }
    if (l < 8) copy16_async(dst + kLatentDim + 8 * l, x + kLatentDim + 8 * l, in);
    copies_commit();
    if (pos == -1) return a;
    if (pos < 0 || pos >= p.cache.cap || (kTurn && pos >= p.max_pos)) {
      a.pos = -2;
      return a;
    }
    if (p.cache.table) {
      const uint32_t in_seq = (uint32_t)pos / (uint32_t)p.cache.page_size;
      a.in_page = (uint32_t)pos - in_seq * (uint32_t)p.cache.page_size;
      a.page = __ldg(p.cache.table + (int64_t)w.b * p.cache.table_ld + in_seq);
    } else {
      a.page = (int)w.b;
      a.in_page = pos;
    }
    if (kTurn) {
      a.cs = __ldg(reinterpret_cast<const float2*>(p.cos + pos * 32) + l);
      a.sn = __ldg(reinterpret_cast<const float2*>(p.sin + pos * 32) + l);
    }
    return a;
  };
  RowWalk w(first, step, p.n);
  Ahead nxt = fetch(first, w, position(first, w.i), 0);
  w.next();
  int64_t pos_next = position(first + step, w.i);
  int slot = 0;
  for (uint32_t base = first - half; base < toks; base += step, slot ^= 1) {  // (the same for both halves of a warp)
    const uint32_t tok = base + half;
    const Ahead now = nxt;
    nxt = fetch(tok + step, w, pos_next, slot ^ 1);
    w.next();
    pos_next = position(tok + 2 * step, w.i);
    copies_wait<1>();
    __syncwarp();
    const uint16_t* x = rows[slot][warp][half];
    f32x2 y[16];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + 8 * (4 * l + (c ^ ((l >> 1) & 3))));
      y[4 * c] = unpack_bf16(v.x);
      y[4 * c + 1] = unpack_bf16(v.y);
      y[4 * c + 2] = unpack_bf16(v.z);
      y[4 * c + 3] = unpack_bf16(v.w);
    }
    // rope pairs 2 l and 2 l + 1: values 4 l .. 4 l + 3, or (2 l, 2 l + 32) and (2 l + 1, 2 l + 33)
    const uint32_t* xr = reinterpret_cast<const uint32_t*>(x + kLatentDim);
    const uint32_t u = xr[p.interleaved ? 2 * l : l], v = xr[p.interleaved ? 2 * l + 1 : 16 + l];
    __syncwarp();  // the slot may be filled again
    bool bad = now.pos == -2;
    const bool live = now.pos >= 0 && now.page >= 0 && now.page < p.cache.n_pages;
    bad |= now.pos >= 0 && !live;
    if (bad && l == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
    if (p.weight) {  // (both halves, whether their tokens are stored or not: the shuffles want all lanes)
      f32x2 s2 = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) s2 = fma_2(y[e], y[e], s2);
      float ss = lo_of(s2) + hi_of(s2);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float f = rsqrtf(ss * (1.f / kLatentDim) + p.eps);
      const f32x2 f2 = pair(f, f);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 g = reinterpret_cast<const float4*>(weights)[8 * l + (c ^ (l & 7))];
        y[2 * c] = mul_2(mul_2(y[2 * c], f2), pair(g.x, g.y));
        y[2 * c + 1] = mul_2(mul_2(y[2 * c + 1], f2), pair(g.z, g.w));
      }
    }
    float top = 0.f;  // (a NaN stays)
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max3_abs(top, lo_of(y[e]), hi_of(y[e]));
    float amax = top;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!live) continue;
    const int64_t row = (int64_t)now.page * p.cache.page_size + now.in_page;
    const float q = amax / kTopFour;
    // (e2m1 has no infinity and no NaN to give a row: its scale is NaN)
    const float scale = !(amax < INFINITY) ? NAN : q < kMinScale ? kMinScale : q;
    with_quotient(scale, [&](auto div) {
      const uint32_t g = group_of(lo_of(div(pair(top, top))));
      const float f = __uint_as_float((254u - g) << 23);  // 2^-e
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x2 v = mul_2(div(y[4 * i + j]), pair(f, f));
          z[j] = make_float2(lo_of(v), hi_of(v));
        }
        o[i] = pack_e2m1(z);
      }
      reinterpret_cast<uint4*>(p.cache.codes + row * (kLatentDim / 2))[l] = make_uint4(o[0], o[1], o[2], o[3]);
      p.cache.groups[row * kLatentGroups + l] = (uint8_t)g;
      const float a0 = bf_lo(u), c0 = p.interleaved ? bf_hi(u) : bf_lo(v), a1 = p.interleaved ? bf_lo(v) : bf_hi(u), c1 = bf_hi(v);
      const f32x2 r0 = any_quotient(div, kTurn ? pair(a0 * now.cs.x - c0 * now.sn.x, c0 * now.cs.x + a0 * now.sn.x) : pair(a0, c0), scale);
      const f32x2 r1 = any_quotient(div, kTurn ? pair(a1 * now.cs.y - c1 * now.sn.y, c1 * now.cs.y + a1 * now.sn.y) : pair(a1, c1), scale);
      uint32_t* out = reinterpret_cast<uint32_t*>(p.cache.rope + row * kLatentRope);
      if (p.interleaved) {
        reinterpret_cast<uint2*>(out)[l] = make_uint2(pack_bf16(lo_of(r0), hi_of(r0)), pack_bf16(lo_of(r1), hi_of(r1)));
      } else {
        out[l] = pack_bf16(lo_of(r0), lo_of(r1));
        out[16 + l] = pack_bf16(hi_of(r0), hi_of(r1));
      }
    });
    if (l == 0) p.cache.scales[row] = scale;
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

// Eight e2m1 codes times s (the group's power of two in it), as bf16.
__device__ __forceinline__ uint4 dequant8(uint32_t c, float s) {
  uint32_t o[4], h[4];
  unpack_e2m1(c, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
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

// Rows of the 4-bit cache: as bf16, or (kUnpack) in the FP8 cache's form, under the same scale.  A half-warp takes a row,
// lane l its values 8 l + 128 k .. + 7 (k < 4), so that every store is of whole runs and what a row costs beside its
// values is paid once for two (a warp a row, 187 instructions each: 30.8 us to unpack 131,072 rows; this one, 121, 24.6).  The
// next row's page and the position after that are on their way meanwhile.
template <bool kUnpack>
__global__ void __launch_bounds__(kThreads, 8) k_latent4_read(LatentReadLaunch p) {
  const int lane = threadIdx.x & 31, l = lane & 15;
  const uint32_t rows = (uint32_t)p.B * p.n;  // (below 2^31: checked by the caller)
  const uint32_t step = gridDim.x * (kThreads / 16), first = (blockIdx.x * kThreads + threadIdx.x) / 16;
  auto position = [&](uint32_t r, uint32_t i) -> int64_t { return r >= rows ? -1 : p.idx ? (int64_t)__ldg(p.idx + r) : p.pos0 + i; };
  // (off -1: a position without a row; -2: to be flagged, too)
  auto look_up = [&](uint32_t b, int64_t pos, int& page, int& off) {
    page = 0;
    off = -1;
    if (pos == -1) return;
    if (pos >= 0) page = latent_page(p.cache, b, pos, off);
    if (off < 0) off = -2;
  };
  RowWalk w(first, step, p.n);
  int page, off;
  look_up(w.b, position(first, w.i), page, off);
  w.next();
  int64_t pos = position(first + step, w.i);
  for (uint32_t r = first; r < rows; r += step) {
    const int64_t row = off >= 0 ? latent_row_of(p.cache, page, off) : -1;
    if (row < 0 && off != -1 && l == 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
    // (a row that is none: zeros)
    uint32_t c[4] = {0, 0, 0, 0};
    uint4 g = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
    uint2 rp = make_uint2(0, 0);
    float s = 1.f;
    if (row >= 0) {
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(p.cache.codes + row * (kLatentDim / 2)) + l;
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = __ldg(codes + 16 * k);
      g = __ldg(reinterpret_cast<const uint4*>(p.cache.groups + row * kLatentGroups));
      rp = __ldg(reinterpret_cast<const uint2*>(p.cache.rope + row * kLatentRope) + l);
      s = __ldg(p.cache.scales + row);
    }
    look_up(w.b, pos, page, off);
    w.next();
    pos = position(r + 2 * step, w.i);
    const uint32_t gs[4] = {g.x, g.y, g.z, g.w};  // groups 4 k .. 4 k + 3
    if constexpr (kUnpack) {
      uint2* out = reinterpret_cast<uint2*>(p.out_codes + (int64_t)r * kLatentDim) + l;
#pragma unroll
      for (int k = 0; k < 4; ++k) out[16 * k] = ExpandFour(gs[k] >> (8 * (l >> 2)))(c[k]);
      reinterpret_cast<uint2*>(p.out_rope + (int64_t)r * kLatentRope)[l] = rp;
      if (l == 0) p.out_scales[r] = s;
    } else {
      uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)r * (kLatentDim + kLatentRope)) + l;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out[16 * k] = dequant8(c[k], s * __uint_as_float(((gs[k] >> (8 * (l >> 2))) & 0xffu) << 23));
      reinterpret_cast<uint2*>(out - l + 64)[l] =
          make_uint2(pack_bf16(bf_lo(rp.x) * s, bf_hi(rp.x) * s), pack_bf16(bf_lo(rp.y) * s, bf_hi(rp.y) * s));
    }
  }
}

// Blocks for as many warps as are wanted, up to a number per SM.
int grid_of(int64_t warps, int blocks_per_sm = 8) {
  return (int)std::min<int64_t>((warps + kThreads / 32 - 1) / (kThreads / 32), (int64_t)device_sm_count() * blocks_per_sm);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendLaunch& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.n;
  if (rows == 0) return cudaSuccess;
  TraceScope trace(kTraceCache, st);
  if (p.cache.groups) {
    auto kernel = p.cos ? k_latent4_append<true> : k_latent4_append<false>;
    kernel<<<grid_of((rows + 1) / 2, 3), kThreads, 0, st>>>(p);
  } else {
    auto kernel = p.cos ? k_latent_append<true> : k_latent_append<false>;
    kernel<<<grid_of(rows), kThreads, 0, st>>>(p);
  }
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_latent_read(const LatentReadLaunch& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.n;
  if (rows == 0) return cudaSuccess;
  TraceScope trace(kTraceCache, st);
  if (p.cache.groups) {
    auto kernel = p.out_codes ? k_latent4_read<true> : k_latent4_read<false>;
    kernel<<<grid_of((rows + 1) / 2, 16), kThreads, 0, st>>>(p);
  } else {
    k_latent_read<<<grid_of(rows), kThreads, 0, st>>>(p);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dsa
