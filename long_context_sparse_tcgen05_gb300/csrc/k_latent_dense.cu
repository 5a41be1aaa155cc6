// Attention over every row that a query sees of the paged latent cache, FP8 or 4-bit: the kernel of latent_attn.cuh
// walking runs of blocks, and the joins of tiles that a run ends in.
//   O = sum_j 2^x_j s_j c_j / sum_j 2^x_j over j < lens - T + 1 + t (causal) or j < lens.
// The lengths are device values, so every CTA finds its run from them (ShareCount); the host knows only how many runs
// there may be.  A part of a tile is left in memory as fp32 rows normalised by its own sum and their log sums, two parts a
// CTA at most: 40 MB of scratch at one CTA an SM, less where S says that there are fewer runs.  A second kernel weighs and adds them in order.
// A tile of few heads takes several tokens, which share its rows: 16 heads of a token fill a quarter of the 64.
//
// Measured (64 heads, 4-bit): one token over 131,072 rows 39 us (36 with the rows in L2: 28 the runs of 13.5 blocks, of which
// 7.5 to the first score product and 2 to leave the part, and 8 the join of 152 parts); 32 tokens over 1,024 to 32,768
// rows 95 us; 1,024 tokens over 32,768 rows 3.92 ms, 1,172 TFLOP/s; 4,096 tokens of a prompt 1.34 to 1.40 ms (FP8 1.15 to 1.20); two chunks of
// 301 tokens of 16 heads over 4,099 and 2,050 rows (FP8) 88 to 91 us; 608 tokens over 524,288 rows 38.6 ms (FP8 36.5).  Bounded like the sparse kernels (a block 2,200 cycles).
// Tried: the join launched early (griddepcontrol): 35.4 us either way; told early by the attention kernel: 40; blocks
// walked from a start of each CTA's own, against many CTAs asking for the same rows at once: 2% slower.
#include <algorithm>

#include "latent_attn.cuh"

namespace dsa {
namespace {

constexpr int kJoinThreads = 256;

// A split tile that block x of a join has to put together: the x-th of them.
struct SplitTile {
  int tile, run, parts, first_slot;
  // Part s is of run `run - 1 + s`; the first one's is its last tile, the others' their first.
  __device__ __forceinline__ const float* part(const LatentAttnLaunch& p, int s) const {
    return p.parts + (int64_t)(s == 0 ? first_slot : 2 * (run - 1 + s)) * kPartFloats;
  }
};
// Found by all threads of a block (parts = 0: there is none).
__device__ __forceinline__ SplitTile find_split(const LatentAttnLaunch& p, int ctas) {
  __shared__ int2 starts[kMaxRuns];  // of each run: its first tile (-1: none) and block in it
  __shared__ SplitTile found;
  const int t = threadIdx.x, lane = t & 31;
  for (int c = t; c < ctas; c += kJoinThreads) {
    const int4 s = p.shares[c];
    starts[c] = make_int2(s.x, s.y);
  }
  __syncthreads();
  if (t < 32) {  // the x-th run that starts inside a tile which the run before it starts at or before
    int left = blockIdx.x, run = -1, n = 1;
    for (int c0 = 1; c0 < ctas && run < 0; c0 += 32) {
      const int c = c0 + lane;
      const bool is = c < ctas && starts[c].x >= 0 && starts[c].y > 0 && (starts[c - 1].x != starts[c].x || starts[c - 1].y == 0);
      uint32_t bal = __ballot_sync(0xffffffffu, is);
      const int k = __popc(bal);
      if (left < k) {
        for (int i = 0; i < left; ++i) bal &= bal - 1;
        run = c0 + __ffs(bal) - 1;
      } else {
        left -= k;
      }
    }
    for (bool more = run > 0; more;) {  // it and the runs after it that start inside the tile: a part each
      const int c = run + n - 1 + lane;
      const uint32_t bal = __ballot_sync(0xffffffffu, c < ctas && starts[c].x == starts[run].x && starts[c].y > 0);
      const int k = bal == 0xffffffffu ? 32 : __ffs(~bal) - 1;
      n += k;
      more = k == 32;
    }
    if (t == 0) {
      found.run = run;
      found.parts = run > 0 ? n : 0;
      found.tile = run > 0 ? starts[run].x : 0;
      found.first_slot = run > 0 ? 2 * (run - 1) + (starts[run - 1].x != starts[run].x) : 0;
    }
  }
  __syncthreads();
  return found;
}

// Puts the parts of split tiles together: O = sum_s w_s O_s, w_s = e^(lse_s - lse), in the order of the parts.  Block
// (x, y) takes the x-th split tile and the y-th `heads` heads of it, a warp a quarter of a head's dims.
__global__ void __launch_bounds__(kJoinThreads) k_latent_join(LatentAttnLaunch p, int ctas, int heads) {
  const SplitTile f = find_split(p, ctas);
  if (f.parts == 0) return;
  const Item I = item_of<kAll>(p, f.tile);
  const int64_t out0 = (int64_t)I.row * p.H + I.h0;
  const int lane = threadIdx.x & 31, end = min((int)(blockIdx.y + 1) * heads, I.heads) * 4;
  for (int u = blockIdx.y * heads * 4 + (threadIdx.x >> 5); u < end; u += kJoinThreads / 32) {
    const int h = u >> 2, quarter = u & 3;
    auto piece = [&](int s) { return reinterpret_cast<const float4*>(f.part(p, s) + h * kLatentDim + quarter * (kLatentDim / 4)) + lane; };
    // four parts on their way together, the first four before their weights
    constexpr int kAtOnce = 4;
    float4 x[kAtOnce];
    auto load = [&](int s) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (s + i < f.parts) x[i] = __ldg(piece(s + i));
    };
    load(0);
    float mx = -INFINITY, sum = 0.f;
    for (int s = lane; s < f.parts; s += 32) mx = fmaxf(mx, f.part(p, s)[kHg * kLatentDim + h]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < f.parts; s0 += 32) {
      float w = 0.f;
      if (s0 + lane < f.parts) {
        const float v = f.part(p, s0 + lane)[kHg * kLatentDim + h];
        w = v == -INFINITY ? 0.f : expf(v - mx);  // (a NaN stays)
      }
      sum += w;
      for (int s = s0; s < min(s0 + 32, f.parts); s += kAtOnce) {
        if (s > 0) load(s);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const float ws = __shfl_sync(0xffffffffu, w, s - s0 + i);
          if (s + i < f.parts) {
            acc.x += ws * x[i].x;
            acc.y += ws * x[i].y;
            acc.z += ws * x[i].z;
            acc.w += ws * x[i].w;
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = sum == 0.f ? 0.f : 1.f / sum;
    reinterpret_cast<uint2*>(p.out + (out0 + h) * kLatentDim + quarter * (kLatentDim / 4))[lane] =
        make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
    if (p.lse && quarter == 0 && lane == 0) p.lse[out0 + h] = sum == 0.f ? -INFINITY : mx + logf(sum);
  }
}

// The same of few tiles, which may have a part on every SM: block (x, y) takes a quarter of one head's dims, each of its
// warps every eighth part.  (131,072 rows of one sequence, 152 parts: 8 us.)
__global__ void __launch_bounds__(kJoinThreads) k_latent_join_long(LatentAttnLaunch p, int ctas) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float lse[kMaxRuns];
  __shared__ float4 sums[kWarps][32];
  __shared__ float sum_s;
  const SplitTile f = find_split(p, ctas);
  if (f.parts == 0) return;
  const Item I = item_of<kAll>(p, f.tile);
  const int h = blockIdx.y >> 2, quarter = blockIdx.y & 3, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (h >= I.heads) return;
  // A warp's parts on their way together, all of them where there are up to 160 parts, before their weights.
  constexpr int kAtOnce = 20;
  float4 x[kAtOnce];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int s = s0 + i * kWarps;
      if (s < f.parts) x[i] = __ldg(reinterpret_cast<const float4*>(f.part(p, s) + h * kLatentDim + quarter * (kLatentDim / 4)) + lane);
    }
  };
  load(warp);
  for (int s = t; s < f.parts; s += kJoinThreads) lse[s] = f.part(p, s)[kHg * kLatentDim + h];
  __syncthreads();
  float mx = -INFINITY;
  for (int s = lane; s < f.parts; s += 32) mx = fmaxf(mx, lse[s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  auto weight = [&](int s) { return lse[s] == -INFINITY ? 0.f : expf(lse[s] - mx); };  // (a NaN stays)
  if (warp == 0) {
    float sum = 0.f;
    for (int s = lane; s < f.parts; s += 32) sum += weight(s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sum_s = sum;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = warp; s0 < f.parts; s0 += kAtOnce * kWarps) {
    if (s0 != warp) load(s0);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int s = s0 + i * kWarps;
      if (s < f.parts) {
        const float w = weight(s);
        acc.x += w * x[i].x;
        acc.y += w * x[i].y;
        acc.z += w * x[i].z;
        acc.w += w * x[i].w;
      }
    }
  }
  sums[warp][lane] = acc;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int i = 1; i < kWarps; ++i) {
    const float4 x = sums[i][lane];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const int64_t row = (int64_t)I.row * p.H + I.h0 + h;
  const float r = sum_s == 0.f ? 0.f : 1.f / sum_s;
  reinterpret_cast<uint2*>(p.out + row * kLatentDim + quarter * (kLatentDim / 4))[lane] =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (p.lse && quarter == 0 && lane == 0) p.lse[row] = sum_s == 0.f ? -INFINITY : mx + logf(sum_s);
}

template <bool kPoll, bool kFour>
auto dense_kernel(Form form) {
  if (form == kAllLong) return k_latent_attn<kPoll, kAllLong, kFour>;
  if constexpr (!kFour)
    if (form == kAllTiles) return k_latent_attn<kPoll, kAllTiles, kFour>;
  return k_latent_attn<kPoll, kAll, kFour>;
}
template <bool kFour>
auto dense_kernel(bool poll, Form form) {
  return poll ? dense_kernel<true, kFour>(form) : dense_kernel<false, kFour>(form);
}

// How a call's queries lie on tiles of 64 heads: of one token a group of 64, or, of few heads, several tokens.
void tile(LatentAttnLaunch& p) {
  p.groups = (p.H + kHg - 1) / kHg;
  p.tile_t = p.H <= kHg ? min(kHg / p.H, p.T) : 1;
  p.tiles_t = (p.T + p.tile_t - 1) / p.tile_t;
}
// CTAs of a call: one per SM, fewer where S says that there are not blocks enough for them.
int runs_of(const LatentAttnLaunch& p) {
  const int64_t blocks = (int64_t)p.B * p.tiles_t * p.groups * ((p.S - 1) / kNB + 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(device_sm_count(), kMaxRuns), blocks / kMinRun));
}

// Blocks of one tile that a CTA may walk, at most: of few tiles their equal parts, else all that a run holds (see ShareCount).
int64_t most_blocks(const LatentAttnLaunch& p, int runs) {
  const int64_t tiles = (int64_t)p.B * p.tiles_t * p.groups, blocks = (p.S - 1) / kNB + 1;
  return std::min(blocks, tiles * (blocks + kMostCost) / runs + 2 * (kMostCost + kMinRun));
}

template <bool kFour>
cudaError_t launch(LatentAttnLaunch p, cudaStream_t st) {
  TraceScope trace(kTraceAttention, st);
  static std::atomic<bool> ready[64];
  tile(p);
  const int runs = runs_of(p);
  p.wait = wait_limit();
  p.splits = 1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    for (int poll = 0; poll < 2; ++poll)
      for (Form form : {kAll, kAllTiles, kAllLong})
        if ((e = prepare_kernel<kFour>(dense_kernel<kFour>(poll, form))) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t cfg = launch_config<kFour>(runs, 1, st, &attr);
  const bool poll = p.wait < kDefaultWaitCycles;
  p.by_length = most_blocks(p, runs) > kMaxBlocks;
  if ((e = cudaLaunchKernelEx(&cfg, dense_kernel<kFour>(poll, p.causal && p.tile_t > 1 ? kAllTiles : kAll), p)) != cudaSuccess) return e;
  count_launches(1);
  if (p.by_length) {
    if ((e = cudaLaunchKernelEx(&cfg, dense_kernel<kFour>(poll, kAllLong), p)) != cudaSuccess) return e;
    count_launches(1);
  }
  if (runs > 1) {
    const int split = std::min(runs - 1, p.B * p.tiles_t * p.groups);  // split tiles, at most
    const int most = std::min(kHg, p.H * p.tile_t);
    // The join of many parts for up to three tiles, the short one with four heads a block for up to 64, us with the long one /
    // four / eight heads (single tokens of 64 heads, 131,072 rows unless said): 1 sequence 37 / 64 / 95, 2 60 / 70 / 86, 3 80 / 83 / 96,
    // 4 99 / 95 / 106, 8 of 65,536 108 / 90 / 95, 16 of 32,768 133 / 92 / 94, 32 of up to 32,768 172 / 95 / 98, 140 of up to 20,000
    // - / 210 / 208.  (Of 8 heads, 4 sequences: 85 / 93 / 102.)
    if (split <= 3) {
      k_latent_join_long<<<dim3(split, 4 * most), kJoinThreads, 0, st>>>(p, runs);
    } else {
      const int heads = split <= 64 ? 4 : 8;
      k_latent_join<<<dim3(split, (most + heads - 1) / heads), kJoinThreads, 0, st>>>(p, runs, heads);
    }
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace

size_t latent_dense_scratch(LatentAttnLaunch p) {
  tile(p);
  const size_t runs = runs_of(p);
  return runs * (sizeof(int4) + 2 * kPartFloats * sizeof(float));
}

cudaError_t launch_latent_dense(LatentAttnLaunch p, void* scratch, cudaStream_t st) {
  tile(p);
  p.shares = static_cast<int4*>(scratch);
  p.parts = reinterpret_cast<float*>(p.shares + runs_of(p));
  return p.cache.groups ? launch<true>(p, st) : launch<false>(p, st);
}
}  // namespace dsa
