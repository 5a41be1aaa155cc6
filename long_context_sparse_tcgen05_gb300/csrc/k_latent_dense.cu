// Attention over every row that a query sees of the paged latent cache, FP8 or 4-bit.
#include <algorithm>

#include "latent_attn.cuh"

namespace dsa {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kMaxRuns = 1024;  // CTAs of a call

// Puts the parts of split tiles together: O = sum_s w_s O_s, w_s = e^(lse_s - lse), in a fixed order.  Block (x, y)
// takes the x-th split tile and the y-th `heads` heads of it (kQuarter: the y-th quarter of one head's dims): threads of a
// row take four dims each, the rows of threads share the parts.
template <bool kQuarter>
__global__ void __launch_bounds__(kJoinThreads) k_latent_join(LatentAttnLaunch p, int ctas, int heads) {
  constexpr int kCols = kQuarter ? kLatentDim / 16 : kLatentDim / 4, kGroups = kJoinThreads / kCols;
  __shared__ float wgt[kMaxRuns];
  __shared__ float4 sums[kGroups][kCols];
  __shared__ int2 starts[kMaxRuns];  // of each run: its first tile (-1: none) and block in it
  __shared__ int found_run, found_parts;
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
      found_run = run;
      found_parts = n;
    }
  }
  __syncthreads();
  const int run = found_run, parts = found_parts;
  if (run < 0) return;
  const int tile = starts[run].x;
  const Item I = item_of<kAll>(p, tile);
  // Part s is of run `run - 1 + s`; the first one's is its last tile, the others' their first.
  const int first_slot = 2 * (run - 1) + (starts[run - 1].x != tile);
  auto part = [&](int s) -> const float* { return p.parts + (int64_t)(s == 0 ? first_slot : 2 * (run - 1 + s)) * kPartFloats; };
  const int64_t out0 = (int64_t)I.row * p.H + I.h0;
  const int group = t / kCols, col = t % kCols, col0 = kQuarter ? blockIdx.y % 4 * kCols : 0;
  const int h0 = kQuarter ? blockIdx.y / 4 : blockIdx.y * heads;
  for (int h = h0; h < min(h0 + (kQuarter ? 1 : heads), I.heads); ++h) {
    if (t < 32) {
      float mx = -INFINITY, sum = 0.f;
      for (int s = lane; s < parts; s += 32) {
        const float v = part(s)[kHg * kLatentDim + h];
        wgt[s] = v;
        mx = fmaxf(mx, v);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      for (int s = lane; s < parts; s += 32) sum += wgt[s] = wgt[s] == -INFINITY ? 0.f : expf(wgt[s] - mx);  // (a NaN stays)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      for (int s = lane; s < parts; s += 32) wgt[s] = sum == 0.f ? 0.f : wgt[s] / sum;
      if (t == 0 && p.lse && col0 == 0) p.lse[out0 + h] = sum == 0.f ? -INFINITY : mx + logf(sum);
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = group; s < parts; s += kGroups) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(part(s) + h * kLatentDim) + col0 + col);
      const float w = wgt[s];
      acc.x += w * x.x;
      acc.y += w * x.y;
      acc.z += w * x.z;
      acc.w += w * x.w;
    }
    sums[group][col] = acc;
    __syncthreads();
    if (!group) {
      for (int i = 1; i < min(kGroups, parts); ++i) {
        const float4 x = sums[i][col];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      reinterpret_cast<uint2*>(p.out + (out0 + h) * kLatentDim)[col0 + col] = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
    __syncthreads();  // (wgt and sums are free)
  }
}

template <bool kFour>
auto dense_kernel(bool poll) {
  return poll ? k_latent_attn<true, kAll, kFour> : k_latent_attn<false, kAll, kFour>;
}

// How a call's queries lie on tiles of 64 heads: of one token a group of 64, or, of few heads, several tokens.
void tile(LatentAttnLaunch& p) {
  p.groups = (p.H + kHg - 1) / kHg;
  p.tile_t = p.H <= kHg ? min(kHg / p.H, p.T) : 1;
  p.tiles_t = (p.T + p.tile_t - 1) / p.tile_t;
}
// CTAs of a call: one per SM, fewer where S says that there are not blocks enough for them.
int runs_of(const LatentAttnLaunch& p) {
  const int64_t blocks = (int64_t)p.B * p.tiles_t * p.groups * ((p.S + kNB - 1) / kNB);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(device_sm_count(), kMaxRuns), blocks / kMinRun));
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
      if ((e = prepare_kernel<kFour>(dense_kernel<kFour>(poll))) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t cfg = launch_config<kFour>(runs, 1, st, &attr);
  if ((e = cudaLaunchKernelEx(&cfg, dense_kernel<kFour>(p.wait < kDefaultWaitCycles), p)) != cudaSuccess) return e;
  count_launches(1);
  if (runs > 1) {
    const int split = std::min(runs - 1, p.B * p.tiles_t * p.groups);  // split tiles, at most
    const int most = std::min(kHg, p.H * p.tile_t);
    if (split <= 8) {  // few tiles of many parts: more blocks a tile
      k_latent_join<true><<<dim3(split, 4 * most), kJoinThreads, 0, st>>>(p, runs, 1);
    } else {
      const int heads = split <= 64 ? 2 : 8;
      k_latent_join<false><<<dim3(split, (most + heads - 1) / heads), kJoinThreads, 0, st>>>(p, runs, heads);
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
