// The paged FP8 latent cache: appending rows (norm, rotation, quantisation and the write through
// the block table in one pass) and reading rows back.  A warp takes a token: 16 latent values per
// lane (two 16-byte loads) and one rotated pair, so the sum of squares and the largest magnitude
// are warp shuffles.  HBM-bound: 1,152 bytes in and 644 out per appended token (the other way
// round to read), plus a 256-byte table row.  Measured: 131,072 tokens appended in 55.6 us (4.9 TB/s;
// 75% of the issue slots, 370 instructions a token, 27 of them quotients) and read back in 41.2 us
// (5.7 TB/s); 32 x 2,048 selected rows read in 22.6 us (5.2 TB/s); one token each of 32 sequences appended
// in 3.5 us.
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
// would spread an infinity or NaN over its pair.  Chosen inside the kernel, a call of 131,072 rows took 59.5,
// not 57.2 us.)
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
  if (p.cos) k_latent_append<true><<<grid_of(rows), kThreads, 0, st>>>(p);
  else k_latent_append<false><<<grid_of(rows), kThreads, 0, st>>>(p);
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
