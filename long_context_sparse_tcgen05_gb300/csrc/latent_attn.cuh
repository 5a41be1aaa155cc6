// Attention over rows of the paged latent cache, FP8 or 4-bit, on tcgen05 tensor cores that read e4m3
// codes: over selected rows (index rows), or over every row that a query sees.
//
// An FP8 cache row j stands for s_j [c_j | r_j]: 512 e4m3 codes and 64 bf16 rope values under one fp32
// scale.  For a head with query q, in base-2 units (a = softmax scale * log2 e):
//   x_j = a s_j (q_c . c_j + q_r . r_j),   O = sum_j 2^x_j s_j c_j / sum_j 2^x_j.
// Both products take the codes as FP8 operands, so no row is dequantised; the other operand is
// made of two FP8 terms that together keep bf16's precision:
//   * q: a power of two 2^k per head brings its largest value to [128, 256); then
//     q 2^k = hi + lo / 16 with hi = e4m3(q 2^k) and lo = e4m3(16 (q 2^k - hi)).  A bf16 value has 8
//     significant bits, hi takes 4 and lo the other 4: exact down to 2^-21 of the head's largest.
//     The rope part stays bf16 (times 2^k, exact).  S has a hi and a lo row per head (M = 128 for
//     64 heads): hi . c + r . r and lo . c, added by the softmax.
//   * the weights: y_j = x_j + log2 s_j carries the row's scale.  A block of 64 keys takes its own
//     power of two, E = ceil(max y) - 8 per head: p_j = 2^(y_j - E) <= 256, and p_j = hi + lo in
//     e4m3 (each rounded to nearest): relative error 2^-8, at most 2^-10 absolute where p_j is
//     small, 2^-17 of the block's largest.  The value product is block-scaled, the B scale 2^(E - E0) per
//     head, E0 being the head's E at its first block, so blocks of any size add into the same O
//     without rescaling it (before, each rise of a running maximum had to rescale O between two
//     products: in ten of a row's 32 blocks, a third of a decode step).  Only when E passes
//     E0 + 40 is O rescaled and E0 moved.  Row sums take p_j / s_j, times 2^(E - E0), in fp32.
// FP8 products accumulate exactly enough in fp32 (sums of 2,048 products of mixed size came out
// equal to the 64-bit sum; those of millions do not, see kMaxBlocks).
//
// A row of the 4-bit cache has 512 e2m1 codes, a power of two for 32 of them, and the same scale and rope
// values: each code times its power of two is an e4m3 value (see latent_cache.cuh), so the gather warps expand
// the codes on their way into shared memory and all that follows is the same, bit for bit.  The tensor cores
// could read e2m1 codes with a power of two for 32 values of a dot product, which serves the scores; in the value
// product a row's powers vary along the other axis, so they have to be in the operand.
//
// Persistent CTAs, one per SM, walk items (query, group of 64 heads, part of the row's blocks of 64
// keys).  24 warps:
//   6-7    take the blocks in turn, up to six ahead: resolve positions through the block table and
//          read the rows' scales
//   0-3    copy the rows (16-byte cp.async) into three stages of 40 KB, five 128-byte-swizzled atoms
//          each, as soon as the products have released them.  4-bit: with 24-27, eight warps, from registers; a
//          block needs 2,150 warp instructions more, half of them byte permutations and logic that run at half
//          rate, and four warps took 3.1 ms for what eight do in 1.2
//   4      S (hi and lo rows, 128 x 64) = Q K^T: A is Q in tensor memory, so the product reads only
//          the codes from shared memory; 16 FP8 steps and 4 bf16 steps for the rope part
//   5      O^T (512 x 64) += V^T P^T: four chunks of 128 dims, 2 key steps, hi and lo
//   8-15   softmax: a warp holds 8 heads whole (their hi and lo rows lie in one 16-lane half of a
//          lane quarter), so maxima and sums never leave a quad of lanes and no barrier joins warps
//   16-19  put a block's scales into tensor memory (every lane quarter wants a copy); rescale O^T
//          when a head's E0 moves
//   20-23  convert the next item's queries while the present one runs, and put them into tensor
//          memory when its last score product is done
//   16-23  normalise an item's O, while the softmax already runs the next item: bf16 rows go to the
//          room of the converted queries (free at that time) and out by bulk copies
// The issuing warps run as whole warps on warp-uniform values and elect the issuing lane: operand
// descriptors then stay in uniform registers.  Issued from a lane-0 branch, every product took 60
// cycles whatever its shape; this way 32 (A in tensor memory) and 48 (A in shared memory: 6 KB of
// operands at 128 bytes a cycle).
// With few items of long index rows each is split into up to 8 parts of about 128 keys or more, one to each
// CTA of a cluster, and the parts are joined over the cluster's shared memory.
// Over all rows, an item is a tile of 64 heads of one or (few heads) several tokens, or 2^18 rows of a longer one, and a
// CTA walks a run of blocks over tiles: see ShareCount, kMaxBlocks and k_latent_dense.cu.
// Waits are bounded (DSA_FLAG_TIMEOUT).
//
// Measured (64 heads, k = 2,048, FP8 / 4-bit): 4,096 queries over 131,072 rows 0.98 / 1.20 ms, 1,195 / 973 TFLOP/s, the
// tensor pipe 51 / 43% busy; 32 single tokens over 200,000 rows 27.3 / 28.3 us; one over 20,000 rows 18.3 / 19.2 us.
// What bounds the 4-bit form: the gather warps' instructions (a block 2,400 cycles; without half of the products it
// takes 3% less) and, where rows are at random, 2,000 cycles to their codes.  What bounds the FP8 form: a
// block's products need 1,360 cycles of the tensor pipe, a block takes 2,000: a softmax warp's waits
// (200), loads (170), scores and maxima (680), exponentials and stores (740) follow one another, and
// tensor memory (512 columns in use) has no room for a second score buffer to overlap them with.  A
// row's start and end cost 4,000 more (O must leave tensor memory before the next row's first product).
// Several roles share each scheduler and their loops compete for the instruction caches: a smaller loop
// often beat one with more in flight.  A decode step is a chain of latencies: 4 us to the first rows,
// 1 us a block, 1.7 us to leave a part, 4.5 us to join the parts.
#pragma once
#include <cuda_bf16.h>

#include <atomic>
#include <climits>
#include <type_traits>

#include "dsa_internal.cuh"
#include "fp8_rows.cuh"
#include "latent_cache.cuh"
#include "sm100.cuh"

namespace dsa {
namespace {
using namespace sm100;

constexpr int kHg = 64;                      // heads of an item
constexpr int kNB = 64;                      // keys of a block
constexpr int kStages = 3;
constexpr int kD = kLatentDim + kLatentRope;
constexpr uint32_t kAtom = kNB * 128;        // 64 rows of 128 bytes
constexpr uint32_t kStage = 5 * kAtom;       // four atoms of codes, one of rope values
constexpr uint32_t kPBytes = kHg * 128;      // P: per head 64 hi bytes, then 64 lo bytes
// Converted queries: 128 rows (hi and lo of 64 heads) of 512 codes, then of 64 bf16 rope values, the
// 16-byte words of a row permuted by the row's low bits (a lane reads its row word by word).
constexpr uint32_t kQCodes = 128 * kLatentDim, kQBytes = kQCodes + 128 * kLatentRope * 2;
constexpr int kGatherWarps = 4, kSWarp = 4, kPvWarp = 5, kIxWarp0 = 6, kSmWarp0 = 8, kSmWarps = 8, kOWarp0 = 16, kQWarp0 = 20;
constexpr int kRing = 6;                     // blocks the index warps may be ahead
constexpr int kWarps = 24, kMoreGather0 = kWarps;
// The 4-bit kernels have four gather warps more, behind the others: theirs expand the codes.
template <bool kFour>
constexpr int kThreads = (kWarps + (kFour ? kGatherWarps : 0)) * 32;
// Registers by warpgroup (warps 0-3, 4-7, ..), moved at the start from the kernel's own each; the softmax warps
// spilled in their block loop at that.
template <bool kFour>
struct Regs {
  static constexpr int kLaunch = kLatentAttnRegs, kGather = 56, kIssue = 64, kSm = 104, kEpi = 72;
  static_assert(kGather + kIssue + 2 * kSm + 2 * kEpi <= 6 * kLaunch, "registers the block is launched with");
};
template <>
struct Regs<true> {
  static constexpr int kLaunch = kLatent4AttnRegs, kGather = 64, kIssue = 56, kSm = 96, kEpi = 64;
  static_assert(2 * kGather + kIssue + 2 * kSm + 2 * kEpi <= 7 * kLaunch, "registers the block is launched with");
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColQ = 256, kColQR = 384, kColSfA = 416, kColSfB = 424, kColS = 448;
constexpr int64_t kPartFloats = kHg * kLatentDim + kHg;  // of a part in memory: O by head, then lse
constexpr int kMinRun = 2;                   // blocks of a CTA's run, where there are few
constexpr int kTileCost = 10, kMostCost = kTileCost + 3;  // of a tile beside its blocks, in blocks: see ShareCount
constexpr int kSlack = 20;                   // see ShareCount
constexpr int kMaxRuns = 1024;               // CTAs of a call over all rows
// Of a call over all rows, blocks that go into one O in tensor memory.  A CTA walks a longer tile in several items and adds
// their O's in memory, in fp32: each of a block's four additions may lose a last place (2^-23), and they lose in one direction.
// FP8 rows of one sign in one O came out short by (beside bf16's rounding, 2e-3 norm-wise) 2^18 rows 2e-4, 2^20 1.6e-3, 2^22
// 1.1e-2, equal ones by up to 1.8e-2.  2^18 rows, 2^14 additions, stay within 2^-9.  And a wait, which may last an item, stays
// far below its limit however long the rows are.
constexpr int kMaxBlocks = 4096;
// What is told of an item: its blocks and, of kAllLong, whether its tile goes on in the CTA's next item, or began in an
// earlier one.
constexpr int kBlocksMask = 0xffff, kGoesOn = 1 << 16, kBegan = 1 << 17;
static_assert(kMaxBlocks <= kBlocksMask);
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// E0 moves when a block's E passes it by this.  A row sum holds up to 1,024 blocks of 64 weights
// p_j / s_j <= 2^8 / 2^-60 (the append's least scale), times 2^(E - E0): 2^(10 + 6 + 8 + 60 + 40) = 2^124,
// within fp32 (with 60 it passed 2^128).  Over all rows there may be 2^25 blocks: 2^(25 + 6 + 8 + 60 + 24) = 2^123.
constexpr float kMove = 40.f, kMoveAll = 24.f;
constexpr int kInfoReaders = kGatherWarps + 2 + kSmWarps + 4 + 4;  // (4-bit: kGatherWarps more)
constexpr int kEpiThreads = 256;             // O and query warps store an item's O together
constexpr uint32_t kOPitch = 2 * kLatentDim + 16;  // a staged O row: 8 heads' 16-byte pieces in 32 banks
static_assert(kHg * kOPitch <= kQBytes, "O is staged in the queries' room");
static_assert(kHg * kLatentDim * sizeof(float) <= kStages * kStage + 2 * kPBytes, "a part is left over the stages and P");
static_assert(kHg * kMaxLatentSplits * sizeof(float) <= kQBytes, "the parts' weights in the queries' room");

// What a kernel walks.  kRows: whole index rows; kRowParts: parts of index rows, one a CTA, joined over a
// cluster; kAll: all rows that the queries see, divided into equal runs of blocks; kAllTiles: the same of FP8 rows some of
// which not every token of a tile sees.  (In a kernel of its own: what it does about NaN codes costs calls without such tiles
// 6%, a prompt of 4,096 tokens of 64 heads 1,147 -> 1,218 us, and its own calls 2 to 4%, of 16 heads 323 -> 329 to 336.)  kAllLong: any of
// these calls of which a CTA may have more than kMaxBlocks of one tile (3 to 6% slower a block, so a kernel of its own, too:
// where S leaves it open whether any tile is that long, both are launched, and one of them finds that the work is not its own).
enum Form { kRows, kRowParts, kAll, kAllTiles, kAllLong };

struct Bars {
  uint64_t q_full, q_empty, qs_full[2];
  // kv_empty[st][c]: atoms of stage st that may be refilled (0, 1: two of codes, after the value
  // product's dim chunks 1 and 3; 2: the rope values, after the score product)
  uint64_t kv_full[kStages], kv_empty[kStages][3];
  uint64_t ix_row[kRing], ix_full[kRing], ix_empty[kRing];  // a block's rows; its scales too
  uint64_t s_full, s_empty;
  uint64_t p_full[2], p_empty[2];
  uint64_t o_full, o_empty, m_full[2], sf_full[2];
  uint64_t l_full[2], l_empty[2];
  uint64_t info_full[2], info_empty[2];
  uint64_t drain[2];
};
// A CTA's run of blocks in a call over all rows: from block first_j0 of tile `first` to block last_end of tile `last`.
struct DenseShare {
  int first, first_j0, last, last_end, last_whole;
  // Room of a tile that this CTA has a part of (two at most: its first and its last); -1: it has the whole tile.
  __device__ __forceinline__ int slot(int tile) const {
    const bool begun = tile == first && first_j0 > 0;
    if (!begun && (tile != last || last_whole)) return -1;
    return 2 * blockIdx.x + (tile != first);
  }
};
struct Small {
  alignas(16) float4 sc[kRing][kNB / 2]; // of two rows of a block: their scales, log2 of them (0 and -inf: skipped)
  alignas(16) float isc[kRing][kNB];     // 1 / scale (0: skipped)
  int32_t row[kRing][kNB];               // cache row (-1: skipped); 2^31 rows would not fit in memory
  int valid[kRing];                      // some row of the block counts
  alignas(16) float alpha[2][kHg];       // by block parity: factor of O where `need` is set
  uint32_t sf[2][kHg];                   // by block parity: a block's scale, as exponent + 127 in each byte
  alignas(16) float lsum[2][kHg];        // reciprocal row sums, by item parity (of a tile that goes on: 1, or 0 without weights)
  float part_lse[kHg];                   // of a part of a row
  float qs[2][kHg], qnext[kHg];          // 2^-k of the item's heads, and of the converted next one's
  alignas(8) uint8_t need[2][8];         // by block parity and group of 8 heads: O must be rescaled
  Bars bar;
  uint32_t tmem;
  int abort;
  int nb[2];                             // blocks of the item (and flags), by item parity
  // of a call over all rows: the item's first block and the positions that its last token sees, by item
  // parity; this CTA's share of the tiles
  int j0[2], sees[2];
  DenseShare share;
  float carry[2][kHg];                   // of a tile that began before, by item parity: factor of the O's so far
};
constexpr size_t kSmem = 1024 + kStages * kStage + 2 * kPBytes + kQBytes + sizeof(Small);
static_assert(kSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void mma_fp8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
// Block-scaled: B's column n and 32 values of K count times 2^(sf[n] - 127), the byte that the
// instruction descriptor picks of the words at `sfb`; A's rows likewise at `sfa`.
__device__ __forceinline__ void mma_mxfp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
      : "memory");
}
// Its instruction descriptor: e4m3 operands, A (128 dims) MN-major, N = 64, ue8m0 scales, byte 0 of
// A's and of B's scale words.
__host__ __device__ constexpr uint32_t idesc_mx() {
  return (1u << 15) | ((uint32_t)(64 >> 3) << 17) | (1u << 23) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x2(uint32_t taddr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};\n" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 lanes x 64 columns: thread t receives, for j < 8, lane t/4 at columns 8j + 2(t%4) + {0, 1}
// (r[4j], r[4j + 1]) and lane t/4 + 8 at the same columns (r[4j + 2], r[4j + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// 16 lanes x 32 columns, distributed the same way.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// Before the asynchronous proxy (a product, a bulk copy) reads what threads wrote to shared memory.  The order
// of the write before the read wants one proxy fence anywhere between them, so the reading thread makes it,
// after the barrier that the writers arrived at: one a block instead of one in each writing warp (with a
// second load of O in flight, 1.02 -> 0.99 ms a 4,096-query chunk).
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
// mbar_wait in few instructions: 24 warps of seven kinds run at a time, and their loops compete for
// the instruction caches.  The abort word and the bound are read at each wake.
template <bool kPoll>
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* abort, long long limit) {
  if constexpr (kPoll) return mbar_wait<true>(b, parity, abort, limit);
  if (mbar_try_wait_sleep(b, parity, kSuspendNs)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_try_wait_sleep(b, parity, kSuspendNs)) {
    if (*abort) return false;
    if (clock64() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// One look at three phases: their latencies overlap.
__device__ __forceinline__ bool try_wait3(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6, %7;\n\t"
      "and.pred p, p, q;\n\tand.pred p, p, r;\n\tselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(a)), "r"(pa), "r"(smem_addr(b)), "r"(pb), "r"(smem_addr(c)), "r"(pc), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Other CTAs of the cluster: a meeting of all their threads (each comes, since every wait of its own is
// bounded), and loads from the place in rank's shared memory that p has in this CTA's.
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float cluster_ld(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(const float* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Named barrier of n threads that ORs a predicate over them: the answer is the same for all, so a
// decision to leave (a wait ran out in some warp) leaves no warp behind at a later barrier.
__device__ __forceinline__ bool named_sync_or(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void named_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// Zeros in the place of NaN among the sixteen e4m3 codes at `at` in shared memory.
__device__ __forceinline__ void drop_nan_codes(uint32_t at) {
  uint32_t w[4], any = 0;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t hit = ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // (0x7f alone carries into its top bit)
    any |= hit;
    w[i] &= ~((hit >> 7) * 0xffu);
  }
  if (any) st_shared16(at, make_uint4(w[0], w[1], w[2], w[3]));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// two floats as f16 (a in the low half), f16 pair to e4m3 pair (nearest, saturating) and back
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h) : "f"(b), "f"(a));
  return h;
}
__device__ __forceinline__ uint16_t e4m3_of_f16x2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(c) : "r"(h));
  return c;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(c));
  return h;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// An item: head group and part of query row (b, t).  Of a call over all rows: a tile, the heads of p.tile_t
// tokens from t on, or of one token a group of 64; `heads` counts those of all its tokens, `last` its last token.
struct Item {
  int row, b, t, h0, heads, split, last;
};
template <Form kForm>
__device__ __forceinline__ Item item_of(const LatentAttnLaunch& p, int item) {
  Item r;
  if constexpr (kForm >= kAll) {
    const int u = item / p.groups;
    r.h0 = (item - u * p.groups) * kHg;
    r.b = u / p.tiles_t;
    r.t = (u - r.b * p.tiles_t) * p.tile_t;
    r.last = min(r.t + p.tile_t, p.T) - 1;
    r.heads = p.groups > 1 ? min(kHg, p.H - r.h0) : (r.last + 1 - r.t) * p.H;
    r.row = r.b * p.T + r.t;
    r.split = 0;
    return r;
  }
  r.last = 0;
  const int lrow = item / p.splits;
  r.split = item - lrow * p.splits;
  r.row = lrow / p.groups;
  r.h0 = (lrow - r.row * p.groups) * kHg;
  r.heads = min(kHg, p.H - r.h0);
  r.b = r.row / p.T;
  r.t = r.row - r.b * p.T;
  return r;
}

// Positions that token t sees, of a sequence that holds len (what is out of [0, S] is taken as the
// nearer end, and flagged), and their blocks: one at least, so that a token that sees none still has an item.
__device__ __forceinline__ int dense_sees(const LatentAttnLaunch& p, int t, int len) {
  len = max(0, min(len, p.S));
  return p.causal ? max(0, len - (p.T - 1 - t)) : len;
}
__device__ __forceinline__ int dense_blocks(int sees) { return sees < 1 ? 1 : (sees - 1) / kNB + 1; }

// This CTA's share of a call over all rows: a run of blocks of one tile or of several, one after another.  Runs that
// end inside tiles leave parts, which k_latent_join puts together.
//   Few tiles: each is cut into equal parts of at most L blocks, a part a CTA, if some L up to kSlack above the mean gives no
// more parts than there are CTAs, since a run over a tile's end has a second segment, which costs more than its blocks
// (queries, O).  Up to 20 above, against up to 4 (8 and 12 alike), us: two chunks of 301 tokens of 16 heads over 4,099 and
// 2,050 rows 91 / 98 (FP8 87 / 92; parts of 65 blocks at a mean of 47, so only 20 admits them); but 32 sequences of 1,024 to
// 32,768 rows 95 / 92, 60 of up to 20,000 rows 110 / 101, and within 1 for eight shapes of shorter rows.  (The slack is a
// number of blocks whatever the mean: one row of 4,000 among 99 of up to 64 34.6 / 33.7.)
//   Otherwise all tiles, one after another, are divided into runs of equal cost, so sequences of any lengths keep the SMs
// evenly busy.  A tile costs its blocks (1.15 us each) and own() more: ten, and up to three more where it has fewer than
// twelve.  (Measured alone, 6 us beside its blocks where it is long, 11 us where it has one, a chain of latencies; ten
// blocks are 11.)  A run that ends among those ends with the tile before.  A prompt of 4,096 tokens, 64 heads: by blocks alone
// 3.7 ms (the first CTA had 330 short tiles), with 5 more a tile 1.86 (FP8 1.69), 10 more 1.37 (1.15), own() 1.35 (1.15), 13
// more 1.34 (1.19).  Tiles of up to eight blocks would rather have ten: 1,216 tokens over 512 rows 126 us, with own() 140.
// Every CTA counts all tiles (a few instructions each, over its threads; a tile's own work is thousands of cycles): each
// thread its tiles' blocks, then, all threads having met, find() places the run's ends.
struct ShareRoom {
  int64_t warp_sum[32];
  int parts[kSlack + 1];  // that the tiles make at each L
  int blocks[kMaxRuns];   // of each tile, where there are few
};
template <int kThreads>
struct ShareCount {
  const LatentAttnLaunch& p;
  int64_t sum, upto;  // cost of this thread's tiles; of its warp's threads up to it
  // A tile's own cost beside its n blocks.
  __device__ __forceinline__ static int own(int n) { return max(kTileCost, kMostCost - n / 4); }
  int tiles, lo, hi;
  bool longer;  // one of this thread's tiles has more than kMaxBlocks
  __device__ __forceinline__ int blocks(int tile) const {
    const Item I = item_of<kAll>(p, tile);
    return dense_blocks(dense_sees(p, I.last, __ldg(p.lens + I.b)));
  }
  __device__ __forceinline__ bool few() const { return tiles <= (int)gridDim.x; }  // (at most kMaxRuns)
  __device__ __forceinline__ ShareCount(const LatentAttnLaunch& p, ShareRoom& room) : p(p) {
    tiles = p.B * p.tiles_t * p.groups;
    const int per = (tiles + kThreads - 1) / kThreads;
    lo = min((int)threadIdx.x * per, tiles);
    hi = min(lo + per, tiles);
    sum = 0;
    longer = false;
    for (int i = lo; i < hi; ++i) {
      const int n = blocks(i);
      longer |= n > kMaxBlocks;
      if (few()) room.blocks[i] = n;
      sum += n + own(n);
    }
    upto = sum;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) room.warp_sum[threadIdx.x >> 5] = upto;
  }
  // false: nothing to do.  (All threads meet in it.)
  __device__ __forceinline__ bool find(DenseShare& s, ShareRoom& room) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t upto_warp = lane < kThreads / 32 ? room.warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto_warp, o);
      if (lane >= o) upto_warp += v;
    }
    const int64_t total = __shfl_sync(0xffffffffu, upto_warp, 31);
    const int64_t above = __shfl_sync(0xffffffffu, upto_warp, warp > 0 ? warp - 1 : 0);
    const int64_t before = (warp > 0 ? above : 0) + upto - sum;
    const int c = blockIdx.x;
    if (few() && total >> 32 == 0) {
      int all = 0;
      for (int i = lane; i < tiles; i += 32) all += room.blocks[i];
      all = __reduce_add_sync(0xffffffffu, all);
      const int L0 = max(kMinRun, (int)(((uint32_t)all + gridDim.x - 1) / gridDim.x));
      if (warp <= kSlack) {
        int n = 0;
        for (int i = lane; i < tiles; i += 32) n += (room.blocks[i] + L0 + warp - 1) / (L0 + warp);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) room.parts[warp] = n;
      }
      __syncthreads();
      int L = 0;
#pragma unroll
      for (int i = kSlack; i >= 0; --i)
        if (room.parts[i] <= (int)gridDim.x) L = L0 + i;
      if (L > 0) {
        if (warp == 0) {
          int at = 0, tile = -1, n = 0, part = 0, k = 1;
          for (int i0 = 0; i0 < tiles && tile < 0; i0 += 32) {
            const int mine = i0 + lane < tiles ? room.blocks[i0 + lane] : 0, parts = (mine + L - 1) / L;
            int upto = parts;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
              const int v = __shfl_up_sync(0xffffffffu, upto, o);
              if (lane >= o) upto += v;
            }
            const uint32_t bal = __ballot_sync(0xffffffffu, at + upto > c);
            if (bal) {
              const int w = __ffs(bal) - 1;
              tile = i0 + w;
              n = __shfl_sync(0xffffffffu, mine, w);
              k = __shfl_sync(0xffffffffu, parts, w);
              part = c - (at + __shfl_sync(0xffffffffu, upto, w) - k);
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
          }
          if (lane == 0) {
            s.first = s.last = tile;
            s.first_j0 = (int)((int64_t)n * part / k);
            s.last_end = (int)((int64_t)n * (part + 1) / k);
            s.last_whole = part == k - 1;
            p.shares[c] = make_int4(tile, s.first_j0, tile, s.last_whole);
          }
        }
        __syncthreads();
        return s.first >= 0;
      }
    }
    // run c: costs [from, to) (one division, in 32 bits where they suffice); longer than a tile's own cost
    const int ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, total / (own(0) + kMinRun)));
    if (c >= ctas) {
      if (threadIdx.x == 0) p.shares[c] = make_int4(-1, 0, -1, 0);
      return false;
    }
    const int64_t each = total >> 32 ? total / ctas : (int64_t)((uint32_t)total / (uint32_t)ctas);
    const int rest = (int)(total - each * ctas);
    const int64_t from = each * c + min(c, rest), to = each * (c + 1) + min(c + 1, rest);
    if (from < before + sum && to > before) {  // the run has some of this thread's tiles
      int64_t at = before;
      for (int i = lo; i < hi && at < to; ++i) {
        const int n = blocks(i), mine = own(n), cost = n + mine;
        if (from >= at && from < at + cost) {
          s.first = i;
          s.first_j0 = max((int)(from - at) - mine, 0);
        }
        if (to > at && to <= at + cost) {
          const int end = (int)(to - at) - mine;
          s.last = end > 0 ? i : i - 1;
          s.last_end = end > 0 ? end : blocks(i - 1);
          s.last_whole = end <= 0 || end == n;
        }
        at += cost;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) p.shares[c] = make_int4(s.first, s.first_j0, s.last, s.last_whole);
    return true;
  }
};

// kPoll: a wait limit below the default.  kParts: an item is a part of a row, one a CTA.  (A kernel of its
// own: the loops of a chunk run at the pace of their instruction fetches, 1.09 against 0.99 ms with the
// joining code beside them.)
template <bool kPoll, Form kForm, bool kFour>
__global__ void __launch_bounds__(kThreads<kFour>, 1) k_latent_attn(LatentAttnLaunch p) {
  constexpr bool kParts = kForm == kRowParts, kDense = kForm >= kAll, kLong = kForm == kAllLong;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kv_s = base;
  uint8_t* p_s = kv_s + kStages * kStage;
  uint8_t* q_s = p_s + 2 * kPBytes;
  Small* sm = reinterpret_cast<Small*>(q_s + kQBytes);
  Bars& bar = sm->bar;
  volatile int* abort_flag = &sm->abort;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  int first = blockIdx.x, items = p.B * p.T * p.groups * p.splits;
  const int G = kDense ? 1 : (int)gridDim.x;
  // of what is told of an item: its blocks, and how far on the next item is
  auto blocks_told = [](int told) { return kLong ? told & kBlocksMask : told; };
  auto step = [&](int told) { return kLong && (told & kGoesOn) ? 0 : G; };
  // a wait that every lane of a warp makes, with one answer for the warp
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bar_wait<kPoll>(b, parity, abort_flag, p.wait));
  };

  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 4);
    mbar_init(&bar.q_empty, 1);
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.s_empty, kSmWarps);
    mbar_init(&bar.o_full, 1);
    mbar_init(&bar.o_empty, 8);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.kv_full[i], kFour ? 2 * kGatherWarps : kGatherWarps * 32);
      for (int c = 0; c < 3; ++c) mbar_init(&bar.kv_empty[i][c], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar.ix_row[i], 1);
      mbar_init(&bar.ix_full[i], 1);
      mbar_init(&bar.ix_empty[i], kSmWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.qs_full[i], 4);
      mbar_init(&bar.p_full[i], kSmWarps);
      mbar_init(&bar.p_empty[i], 1);
      mbar_init(&bar.m_full[i], kSmWarps);
      mbar_init(&bar.sf_full[i], 4);
      mbar_init(&bar.l_full[i], kSmWarps);
      mbar_init(&bar.l_empty[i], 8);
      mbar_init(&bar.info_full[i], 1);
      mbar_init(&bar.info_empty[i], kInfoReaders + (kFour ? kGatherWarps : 0));
      mbar_init(&bar.drain[i], 1);
    }
    sm->abort = 0;
    fence_barrier_init();
  }
  if (warp == kSWarp) {
    tmem_alloc(&sm->tmem, kTmemCols);
    tmem_relinquish();
  }
  ShareRoom& room = *reinterpret_cast<ShareRoom*>(kv_s);  // (no stage is in use yet)
  using Count = std::conditional_t<kDense, ShareCount<kThreads<kFour>>, int>;
  const Count count = [&] {
    if constexpr (kDense) return Count(p, room);
    else return 0;
  }();
  tc_fence_before();
  bool other = false;  // the work is the other kernel's
  if constexpr (kDense) other = (__syncthreads_or(count.longer) != 0) != kLong && p.by_length;
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm->tmem, 0);
  if constexpr (kDense) {
    if (other || !count.find(sm->share, room)) {
      if (warp == kSWarp) tmem_dealloc(tmem, kTmemCols);
      return;
    }
    first = sm->share.first;
    items = sm->share.last + 1;
  }

  // Every n-th head of an item's queries, from w on, to hi and lo rows in shared memory (so few heads are
  // spread over the warps too; zeros where there is none).  Two heads at a time, 16 latent values and 2
  // rope values of each a lane.  Row of head h's hi codes: row_of(h); its lo codes 8 rows on, so that a
  // softmax thread's one load gives it both.
  auto row_of = [](int h) -> uint32_t { return 32 * (h >> 4) + 16 * ((h >> 3) & 1) + (h & 7); };
  auto convert = [&](int item, int w, int n) {
    const Item I = item_of<kForm>(p, item);
    const uint16_t* q0 = p.q + I.b * p.q_sb + I.t * p.q_st + (int64_t)I.h0 * kD;
    auto head_at = [&](int h) -> const uint16_t* {
      if (!kDense || p.tile_t == 1) return q0 + (int64_t)h * kD;
      const int t = h / p.H;
      return q0 + t * p.q_st + (int64_t)(h - t * p.H) * kD;
    };
    const uint32_t sixteen = 0x4c004c00u;  // f16 16.0 twice
    uint4 nx[2][2];
    uint32_t nr[2];
    auto load = [&](int h) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool live = h + k * n < I.heads;
        const uint4* q = reinterpret_cast<const uint4*>(head_at(kDense && !live ? 0 : h + k * n));
        nx[k][0] = live ? __ldg(q + lane) : make_uint4(0, 0, 0, 0);
        nx[k][1] = live ? __ldg(q + 32 + lane) : make_uint4(0, 0, 0, 0);
        nr[k] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + kLatentDim / 8) + lane) : 0u;
      }
    };
    auto one = [&](int h, const uint4 (&v)[2], uint32_t rp) {
      // largest magnitude, as bf16 bits (a NaN is above every number)
      uint32_t top = rp & 0x7fff7fffu;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        top = __vmaxu2(top, __vmaxu2(v[u].x & 0x7fff7fffu, v[u].y & 0x7fff7fffu));
        top = __vmaxu2(top, __vmaxu2(v[u].z & 0x7fff7fffu, v[u].w & 0x7fff7fffu));
      }
      top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
      // the largest value's exponent e (not below -100): 2^(7 - e) brings it to [128, 256)
      const int e = max((int)(top >> 7) - 127, -100);
      const bool finite = (top >> 7) < 255;
      const float mul = finite ? __uint_as_float((uint32_t)(7 - e + 127) << 23) : __uint_as_float(0x7fc00000u);
      if (lane == 0) sm->qnext[h] = finite ? __uint_as_float((uint32_t)(e - 7 + 127) << 23) : 1.f;
      const uint32_t row = row_of(h);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t f = f16x2(__uint_as_float(w[x] << 16) * mul, __uint_as_float(w[x] & 0xffff0000u) * mul);
          const uint32_t c = e4m3_of_f16x2(f);
          const uint32_t r = e4m3_of_f16x2(mul_f16x2(sub_f16x2(f, f16x2_of_e4m3((uint16_t)c)), sixteen));
          if (x & 1) hi[x >> 1] |= c << 16, lo[x >> 1] |= r << 16;
          else hi[x >> 1] = c, lo[x >> 1] = r;
        }
        const uint32_t word = 16 * u + (lane >> 1);  // (row and row + 8 permute alike)
        uint8_t* dst = q_s + row * kLatentDim + ((word ^ (row & 7)) << 4) + (lane & 1) * 8;
        *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(dst + 8 * kLatentDim) = make_uint2(lo[0], lo[1]);
      }
      // the lo row's rope part: 2^-40 of the hi row's, nothing beside it, so that an infinite rope
      // value of a key gives both rows the same infinity (zeros would make it a NaN)
      const float a = __uint_as_float(rp << 16) * mul, b = __uint_as_float(rp & 0xffff0000u) * mul;
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b), l2 = __floats2bfloat162_rn(a * 0x1p-40f, b * 0x1p-40f);
      uint8_t* dst = q_s + kQCodes + row * (2 * kLatentRope) + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4;
      *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(&h2);
      *reinterpret_cast<uint32_t*>(dst + 8 * 2 * kLatentRope) = *reinterpret_cast<const uint32_t*>(&l2);
    };
    load(w);
#pragma unroll 1
    for (int h = w; h < I.heads; h += 2 * n) {
      const uint4 a[2] = {nx[0][0], nx[0][1]}, b[2] = {nx[1][0], nx[1][1]};
      const uint32_t ra = nr[0], rb = nr[1];
      load(h + 2 * n);
      one(h, a, ra);
      one(h + n, b, rb);  // (a place below 64: an even number of them a warp)
    }
    if (I.heads == kHg) return;
#pragma unroll 1
    for (int h = w; h < kHg; h += n) {
      if (h < I.heads) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<uint4*>(q_s + (row_of(h) + 8 * k) * kLatentDim + lane * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint32_t*>(q_s + kQCodes + (row_of(h) + 8 * k) * (2 * kLatentRope) + lane * 4) = 0u;
      }
      if (lane == 0) sm->qnext[h] = 1.f;
    }
  };

  // A row's queries into L2, while the item before it is worked on: converting them waits for their loads, which shows where
  // the items are short.  6 x 300 tokens of 64 heads, k 50 / 250: 130 -> 114, 160 -> 150 us, FP8 129 -> 108, 147 -> 131.  Not
  // behind an item of more than four blocks (nothing to win), nor for rows of up to 16 heads, which are loaded at once (one
  // head: 79 -> 82).  Nor over all rows: tiles of one block gain (1,216 tokens over 64 rows: 102 -> 93), but a prompt of 4,096
  // tokens loses (FP8 1,167 -> 1,184) and 1,024 tokens of 128 heads over 8,192 rows, too (1,962 -> 1,977).
  constexpr int kFetchBlocks = 4, kFetchHeads = 16;
  auto fetch = [&](int item) {
    const Item I = item_of<kForm>(p, item);
    const uint16_t* q = p.q + I.b * p.q_sb + I.t * p.q_st + (int64_t)I.h0 * kD;
    if (lane == 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(q), "r"(I.heads * kD * 2) : "memory");
  };

  // An item's O, once its sums and its last value product are there: dim chunks 0 and 2 by the O warps,
  // 1 and 3 by the query warps.  false: a wait ran out in one of them, and all eight leave.
  // These warps meet at barrier 1 in step, and once more (meet_last) when they are done or leave for
  // a wait of their own, so none waits there for one that has left.
  bool met_failure = false;
  auto meet_last = [&](bool ok) {
    if (!met_failure) named_sync_or(1, kEpiThreads, !ok);
  };
  auto epilogue = [&](int item, int oc, int told) -> bool {
    const int q4 = warp & 3, cw = warp < kQWarp0 ? 0 : 1;
    const Item I = item_of<kForm>(p, item);
    const float* ls = sm->lsum[oc & 1];
    const uint32_t o_addr = tmem + ((uint32_t)(q4 * 32) << 16) + kColO + cw * kHg;
    const bool ok = wait(&bar.l_full[oc & 1], (oc >> 1) & 1) && wait(&bar.o_full, oc & 1);
    // (here the query warps are past the read of their converted queries)
    if (named_sync_or(1, kEpiThreads, !ok)) {
      met_failure = true;
      return false;
    }
    tc_fence_after();
    // (a head without weights, sum 0, gives zeros whatever its products left)
    const bool none = __any_sync(0xffffffffu, ls[lane] == 0.f || ls[32 + lane] == 0.f);
    const int part = kDense ? sm->share.slot(item) : -1;
    // (a tile that the CTA has whole, in several items, passes through the room of its last part, which comes later)
    const bool several = kLong && (told & (kGoesOn | kBegan)) != 0;
    const int slot = several && part < 0 ? 2 * (int)blockIdx.x + 1 : part;
    if (several) {  // (a thread reads what it wrote itself)
      float* rows = p.parts + (int64_t)slot * kPartFloats;
#pragma unroll 1
      for (int i = 0; i < kHg / 4; ++i) {
        const int c = i & 1, h0 = 8 * (i >> 1);
        if (h0 >= I.heads) break;
        const int dim = (2 * c + cw) * 128 + q4 * 32 + lane;
        uint32_t r[8];
        tmem_ld_x8(o_addr + 2 * c * kHg + h0, r);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float* at = rows + (h0 + u) * kLatentDim + dim;
          const float a = ls[h0 + u];
          float v = __uint_as_float(r[u]);
          if (told & kBegan) v = fmaf(*at, sm->carry[oc & 1][h0 + u], v);
          v = a == 0.f ? 0.f : v * a;
          if ((told & kGoesOn) || part >= 0) *at = v;
          else if (h0 + u < I.heads) reinterpret_cast<__nv_bfloat16*>(p.out)[((int64_t)I.row * p.H + I.h0 + h0 + u) * kLatentDim + dim] = __float2bfloat16_rn(v);
        }
      }
    } else if (kParts || slot >= 0) {  // fp32 rows over the stages, which the last products have read, or to memory; 32 dims of a head a store
      float* rows = kParts ? reinterpret_cast<float*>(kv_s) : p.parts + (int64_t)slot * kPartFloats;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int c = i >> 1, h0 = 32 * (i & 1);
        if (h0 >= I.heads) continue;
        float* out = rows + h0 * kLatentDim + (2 * c + cw) * 128 + q4 * 32 + lane;
        uint32_t r[32];
        tmem_ld32(o_addr + 2 * c * kHg + h0, r);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          const float4 f = *reinterpret_cast<const float4*>(ls + h0 + u);
          const float a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            out[(u + x) * kLatentDim] = none && a[x] == 0.f ? 0.f : __uint_as_float(r[u + x]) * a[x];
        }
      }
    } else {
      // 16 dims x 32 heads at a time, as 8 x 8 tiles (rows: dims) that stmatrix stores transposed.
      // (A small loop: unrolled, this code ran at the pace of its instruction fetches.)
#pragma unroll 1
      for (int h0 = 0; h0 < I.heads; h0 += 32) {
        const uint32_t dst = smem_addr(q_s) + (h0 + 8 * (lane >> 4) + (lane & 7)) * kOPitch +
                             2 * (cw * 128 + q4 * 32 + 8 * ((lane >> 3) & 1));
        f32x2 f[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) f[t] = *reinterpret_cast<const f32x2*>(ls + h0 + 8 * t + 2 * (lane & 3));
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {  // this warp's chunks: dims 0-15 and 16-31 of its quarter together
          uint32_t r[2][16], w[8];
#pragma unroll
          for (int x = 0; x < 2; ++x) tmem_ld_16x256b_x4(o_addr + 2 * c * kHg + h0 + (x << 20), r[x]);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (none) {
#pragma unroll
              for (int u = 0; u < 16; ++u)
                if ((u & 1 ? hi_of(f[u >> 2]) : lo_of(f[u >> 2])) == 0.f) r[x][u] = 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const f32x2 v = mul_2(pair(__uint_as_float(r[x][2 * u]), __uint_as_float(r[x][2 * u + 1])), f[u >> 1]);
              w[u] = pack_bf16(lo_of(v), hi_of(v));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
              asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(dst + 16 * k * kOPitch + 32 * x + 512 * c),
                           "r"(w[4 * k]), "r"(w[4 * k + 1]), "r"(w[4 * k + 2]), "r"(w[4 * k + 3])
                           : "memory");
          }
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bar.l_empty[oc & 1]);
      mbar_arrive(&bar.o_empty);
    }
    if (!kParts && slot < 0) {
      if (warp < kQWarp0) {
        named_arrive(4, kEpiThreads);  // (the next arrival here comes after the next meeting at barrier 1)
      } else {
        named_sync(4, kEpiThreads);
        async_fence();  // the staged rows, all warps', are read by bulk copies
        const int h = threadIdx.x - kQWarp0 * 32;
        if (h < I.heads) {
          bulk_store(p.out + ((int64_t)I.row * p.H + I.h0 + h) * kLatentDim, smem_addr(q_s) + h * kOPitch, 2 * kLatentDim);
          asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
        }
        named_sync(2, 128);  // the room may hold converted queries again
      }
    }
    return true;
  };

  // Joins the parts of a row, one in each CTA of a cluster: O = sum_s w_s O_s, w_s = e^(lse_s - lse).  The
  // O and query warps of each take a share of the heads, over every CTA's shared memory: 128 KB at the
  // 15 bytes a cycle that such loads move.  (Parts in global memory, joined by a second kernel, took the same
  // 29 us for a 32-sequence decode step and 16.5, not 19, for a single sequence in 16 parts, but 28, not
  // 20, on the host, whose time is what a caller outside a graph waits for: a launch more, and room.)
  auto join = [&]() {
    const Item I = item_of<kForm>(p, blockIdx.x);
    const int t = threadIdx.x - kOWarp0 * 32, h0 = kHg * I.split / p.splits, share = kHg * (I.split + 1) / p.splits - h0;
    float* wgt = reinterpret_cast<float*>(q_s);  // [head of the share][part]: the queries' room is free
    if (t < share) {
      float mx = -INFINITY, sum = 0.f, v[kMaxLatentSplits];
#pragma unroll
      for (int s = 0; s < kMaxLatentSplits; ++s) {
        v[s] = s < p.splits ? cluster_ld(&sm->part_lse[h0 + t], s) : -INFINITY;
        mx = fmaxf(mx, v[s]);
      }
#pragma unroll
      for (int s = 0; s < kMaxLatentSplits; ++s) {
        v[s] = v[s] == -INFINITY ? 0.f : expf(v[s] - mx);  // (a NaN stays)
        sum += v[s];
      }
#pragma unroll
      for (int s = 0; s < kMaxLatentSplits; ++s) wgt[t * kMaxLatentSplits + s] = sum == 0.f ? 0.f : v[s] / sum;
      if (p.lse && h0 + t < I.heads) p.lse[(int64_t)I.row * p.H + I.h0 + h0 + t] = sum == 0.f ? -INFINITY : mx + logf(sum);
    }
    named_sync(1, kEpiThreads);
#pragma unroll 1
    for (int i = t; i < share * (kLatentDim / 4); i += kEpiThreads) {
      const int h = i / (kLatentDim / 4), d = i % (kLatentDim / 4) * 4;
      if (h0 + h >= I.heads) break;
      const float* mine = reinterpret_cast<const float*>(kv_s) + (h0 + h) * kLatentDim + d;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), x[kMaxLatentSplits];
#pragma unroll
      for (int s = 0; s < kMaxLatentSplits; ++s)
        if (s < p.splits) x[s] = s == I.split ? *reinterpret_cast<const float4*>(mine) : cluster_ld4(mine, s);
#pragma unroll
      for (int s = 0; s < kMaxLatentSplits; ++s) {
        const float w = wgt[h * kMaxLatentSplits + s];
        if (w == 0.f) continue;  // (an empty part wrote no values)
        acc.x += w * x[s].x;
        acc.y += w * x[s].y;
        acc.z += w * x[s].z;
        acc.w += w * x[s].w;
      }
      reinterpret_cast<uint2*>(p.out + ((int64_t)I.row * p.H + I.h0 + h0 + h) * kLatentDim + d)[0] =
          make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
  };
  // Every warp's end: with parts, all of a cluster's CTAs meet before they are joined and after.
  auto finish = [&](bool joins) {
    if constexpr (kParts) {
      cluster_meet();
      if (joins) join();
      cluster_meet();
    }
  };

  // The converted rows' columns 32 s0 .. 32 s1 into tensor memory (the rope columns follow the codes').
  auto copy_q = [&](int s0, int s1) {
    const int row = 32 * (warp & 3) + lane;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {  // eight words at a time
      const uint8_t* src = s < 4 ? q_s + row * kLatentDim + 128 * s : q_s + kQCodes + row * (2 * kLatentRope);
      uint32_t r[32];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + ((u ^ (row & 7)) << 4));
        r[4 * u] = v.x;
        r[4 * u + 1] = v.y;
        r[4 * u + 2] = v.z;
        r[4 * u + 3] = v.w;
      }
      tmem_st_x32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColQ + 32 * s, r);
    }
    tmem_wait_stores();
    tc_fence_before();
  };
  // The first item's queries: sixteen warps that have nothing else to do yet convert four heads each,
  // eight of them store the rows (a single decode step waits for nothing longer).
  if (warp >= kSmWarp0 && warp < kWarps) {
    convert(first, warp - kSmWarp0, 16);
    named_sync(3, 512);
    if (warp >= kOWarp0) {
      copy_q(warp < kQWarp0 ? 0 : 3, warp < kQWarp0 ? 3 : 5);
      named_sync(1, kEpiThreads);
    }
  }

  if (warp < kGatherWarps || (kFour && warp >= kMoreGather0)) {
    reg_dec<Regs<kFour>::kGather>();
    // ================= gather =================
    int it = 0;
    uint32_t g = 0;  // blocks so far
    bool ok = true;
    const uint8_t* const codes = p.cache.codes;
    const uint8_t* const rope = reinterpret_cast<const uint8_t*>(p.cache.rope);
    for (int item = first, told = 0; ok && item < items; item += step(told), ++it) {
      if (!(ok = wait(&bar.info_full[it & 1], (it >> 1) & 1))) break;
      told = sm->nb[it & 1];
      const int nb = blocks_told(told);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.info_empty[it & 1]);
      if constexpr (kFour) {
        // A warp has eight rows of a block, a lane 16 bytes of codes (a group of 32 values) of each of four of them.  They
        // wait in registers: a block's loads are made while the one before it is expanded, before a stage is free;
        // so are the copies of its rope values.  Of a skipped row the first row's codes are taken (whatever they are,
        // they stand for finite values, which its weights of 0 make nothing of) and zeros for rope values: loads under a
        // condition were waited for at once, a latency each.
        // Eight lanes have four groups of two neighbouring rows, so that their stores meet all banks.
        const int w0 = 8 * (warp < kGatherWarps ? warp : warp - kMoreGather0 + kGatherWarps);
        const int r0 = w0 + ((lane >> 2) & 1), c = (lane & 3) + 4 * (lane >> 3);
        uint4 raw[4];
        uint32_t grp[4];
        const uint8_t* const codes_c = codes + 16 * c;
        const uint8_t* const groups_c = p.cache.groups + c;
        auto load = [&](int pass, const int32_t* rows) {
          const uint32_t row = (uint32_t)max(rows[r0 + 2 * pass], 0);
          raw[pass] = __ldg(reinterpret_cast<const uint4*>(codes_c + (uint64_t)row * (kLatentDim / 2)));
          grp[pass] = __ldg(groups_c + (uint64_t)row * kLatentGroups);
        };
        auto copy_rope = [&](uint32_t st, const int32_t* rows) {
#pragma unroll
          for (int pass = 0; pass < 2; ++pass) {
            const int r = w0 + pass * 4 + (lane >> 3), cc = lane & 7, row = rows[r];
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(kv_s) + st * kStage + 4 * kAtom + r * 128 + ((cc ^ (r & 7)) << 4)),
                         "l"(rope + (uint64_t)(uint32_t)max(row, 0) * (2 * kLatentRope) + cc * 16), "r"(row < 0 ? 0 : 16)
                         : "memory");
          }
        };
        if (nb) {
          const uint32_t ri = g % kRing, st = g % kStages;
          if (!(ok = wait(&bar.ix_row[ri], (g / kRing) & 1) && wait(&bar.kv_empty[st][2], ((g / kStages) & 1) ^ 1))) break;
          copy_rope(st, sm->row[ri]);
          copies_commit();
#pragma unroll
          for (int pass = 0; pass < 4; ++pass) load(pass, sm->row[ri]);
        }
        for (int j = 0; j < nb; ++j, ++g) {
          const uint32_t st = g % kStages, sn = (g + 1) % kStages, rn = (g + 1) % kRing;
          // The whole stage (its value products end last), the next block's rows, the next stage's rope atom.
          uint64_t* const bs[3] = {&bar.kv_empty[st][1], &bar.ix_row[rn], &bar.kv_empty[sn][2]};
          const uint32_t ph[3] = {((g / kStages) & 1) ^ 1, ((g + 1) / kRing) & 1, (((g + 1) / kStages) & 1) ^ 1};
          const bool more = j + 1 < nb;
          if (kPoll || !more || !__all_sync(0xffffffffu, try_wait3(bs[0], ph[0], bs[1], ph[1], bs[2], ph[2])))
            if (!(ok = wait(bs[0], ph[0]) && (!more || (wait(bs[1], ph[1]) && wait(bs[2], ph[2]))))) break;
          if (more) copy_rope(sn, sm->row[rn]);
          copies_commit();
          const uint32_t at = smem_addr(kv_s) + st * kStage + (c >> 2) * kAtom + r0 * 128 + (((2 * (c & 3)) ^ (r0 & 1)) << 4);
#pragma unroll
          for (int pass = 0; pass < 4; ++pass) {
            const ExpandFour x(grp[pass]);
            const uint2 v0 = x(raw[pass].x), v1 = x(raw[pass].y), v2 = x(raw[pass].z), v3 = x(raw[pass].w);
            const uint32_t to = (at + 256 * pass) ^ (32 * pass);  // (row & 7 = 2 pass + its low bit)
            st_shared16(to, make_uint4(v0.x, v0.y, v1.x, v1.y));
            st_shared16(to ^ 16, make_uint4(v2.x, v2.y, v3.x, v3.y));
            if (more) load(pass, sm->row[rn]);
          }
          copies_wait<1>();  // this block's rope values
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.kv_full[st]);
        }
      } else {
        for (int j = 0; j < nb; ++j, ++g) {
          const int st = (int)(g % kStages), ri = (int)(g % kRing);
          if (!(ok = wait(&bar.ix_row[ri], (g / kRing) & 1))) break;
          const int cc = lane & 7;
          uint8_t* stage = kv_s + st * kStage;
          // atom by atom, 8 lanes per row, 4 rows per pass; the rope atom is free first.  (Waits and commits
          // for each atom of codes cost more than they bring: 1.05 against 0.99 ms a 4,096-query chunk; one
          // for all four: 1.00.)
          int64_t row[4];
          uint32_t dst[4], n[4];
#pragma unroll
          for (int pass = 0; pass < 4; ++pass) {
            const int r = warp * 16 + pass * 4 + (lane >> 3);
            row[pass] = sm->row[ri][r];
            n[pass] = row[pass] >= 0 ? 16 : 0;  // a skipped row is filled with zeros
            if (row[pass] < 0) row[pass] = 0;
            dst[pass] = smem_addr(stage + r * 128 + ((cc ^ (r & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < 5; ++i) {
            const int a = i == 0 ? 4 : i - 1;
            if (i == 0 || i == 1 || i == 3)
              ok &= bar_wait<kPoll>(&bar.kv_empty[st][i == 0 ? 2 : i >> 1], ((g / kStages) & 1) ^ 1, abort_flag, p.wait);
#pragma unroll
            for (int pass = 0; pass < 4; ++pass)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst[pass] + a * kAtom),
                           "l"(a < 4 ? codes + row[pass] * kLatentDim + (a * 128 + cc * 16) : rope + row[pass] * (2 * kLatentRope) + cc * 16),
                           "r"(n[pass])
                           : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_addr(&bar.kv_full[st])) : "memory");
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
      }
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    finish(false);
  } else if (warp < kSmWarp0) {
    reg_dec<Regs<kFour>::kIssue>();
    if (warp == kSWarp) {
      // ================= score product =================
      const uint32_t id8 = idesc_mn(0, 0, 128, kNB), id16 = idesc_mn(1, 1, 128, kNB);
      const uint64_t kv_desc = desc_sw128(smem_addr(kv_s));
      int it = 0, oc = 0;
      uint32_t g = 0;
      bool ok = true;
      for (int item = first, told = 0; ok && item < items; item += step(told), ++it) {
        if (!(ok = wait(&bar.info_full[it & 1], (it >> 1) & 1))) break;
        told = __shfl_sync(0xffffffffu, sm->nb[it & 1], 0);
        const int nb = blocks_told(told);
        if (lane == 0) mbar_arrive(&bar.info_empty[it & 1]);
        if (nb == 0) continue;
        if (!(ok = wait(&bar.q_full, oc & 1))) break;
        for (int j = 0; j < nb; ++j, ++g) {
          const int st = (int)(g % kStages);
          if (!(ok = wait(&bar.s_empty, (g & 1) ^ 1) && wait(&bar.kv_full[st], (g / kStages) & 1))) break;
          async_fence();  // the stage was written by cp.async
          tc_fence_after();
          if (elect_lane()) {
            const uint64_t kd = kv_desc + (uint64_t)((st * kStage) >> 4);
#pragma unroll 1
            for (int a = 0; a < 4; ++a)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_fp8_ts(tmem + kColS, tmem + kColQ + 32 * a + 8 * k, kd + (uint64_t)((a * kAtom + k * 32) >> 4), id8, (a | k) != 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16_ts(tmem + kColS, tmem + kColQR + 8 * k, kd + (uint64_t)((4 * kAtom + k * 32) >> 4), id16, 1);
            mma_commit(&bar.s_full);
            mma_commit(&bar.kv_empty[st][2]);
            if (j == nb - 1) mma_commit(&bar.q_empty);
          }
          __syncwarp();
        }
        ++oc;
      }
      if (elect_lane()) {  // the products issued here end before tensor memory is freed
        mma_commit(&bar.drain[0]);
        mbar_wait_drain(&bar.drain[0], 0);
      }
      __syncwarp();
    } else if (warp == kPvWarp) {
      // ================= value product =================
      const uint64_t v_desc = desc_sw128(smem_addr(kv_s)), p_desc = desc_sw128(smem_addr(p_s));
      int it = 0, oc = 0;
      uint32_t g = 0;
      bool ok = true;
      for (int item = first, told = 0; ok && item < items; item += step(told), ++it) {
        if (!(ok = wait(&bar.info_full[it & 1], (it >> 1) & 1))) break;
        told = __shfl_sync(0xffffffffu, sm->nb[it & 1], 0);
        const int nb = blocks_told(told);
        if (lane == 0) mbar_arrive(&bar.info_empty[it & 1]);
        if (nb == 0) continue;
        if (!(ok = wait(&bar.o_empty, (oc & 1) ^ 1))) break;
        for (int j = 0; j < nb; ++j, ++g) {
          const int st = (int)(g % kStages), pb = (int)(g & 1);
          if (!(ok = wait(&bar.kv_full[st], (g / kStages) & 1) && wait(&bar.sf_full[pb], (g >> 1) & 1) &&
                     wait(&bar.p_full[pb], (g >> 1) & 1)))
            break;
          async_fence();  // P was written by plain stores, the stage by cp.async
          tc_fence_after();
          if (elect_lane()) {
            const uint64_t vd = v_desc + (uint64_t)((st * kStage) >> 4), pd = p_desc + (uint64_t)((pb * kPBytes) >> 4);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int k = 0; k < 4; ++k)  // keys 0-31 and 32-63 by the hi terms, then by the lo terms
                mma_mxfp8(tmem + kColO + c * kHg, vd + (uint64_t)((c * kAtom + (k & 1) * 4096) >> 4),
                          pd + (uint64_t)((k * 32) >> 4), idesc_mx(), tmem + kColSfA, tmem + kColSfB + 4 * pb, (j | k) != 0);
              if (c & 1) mma_commit(&bar.kv_empty[st][c >> 1]);
            }
            mma_commit(&bar.p_empty[pb]);
            if (j == nb - 1) mma_commit(&bar.o_full);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++oc;
      }
      if (elect_lane()) {
        mma_commit(&bar.drain[1]);
        mbar_wait_drain(&bar.drain[1], 0);
      }
      __syncwarp();
    } else {
      // ================= index: positions to cache rows and scales =================
      struct Blocks {  // of an item: its row's ids, its sequence, its first block and their number
        const int32_t* ids;
        int b, j0, nb;
        int sees;  // of a call over all rows: the positions that the tile's last token sees
      };
      // Of a call over all rows, where this CTA's blocks of a tile begin and end.
      auto tile_begin = [&](int tile) { return tile == first ? sm->share.first_j0 : 0; };
      auto tile_end = [&](int tile, int sees) { return tile == sm->share.last ? sm->share.last_end : dense_blocks(sees); };
      auto blocks_of = [&](int item) -> Blocks {
        const Item I = item_of<kForm>(p, item);
        if constexpr (kDense) {
          const int sees = dense_sees(p, I.last, __ldg(p.lens + I.b)), j0 = tile_begin(item), nb = tile_end(item, sees) - j0;
          return {nullptr, I.b, j0, kLong ? min(nb, kMaxBlocks) : nb, sees};
        }
        const int32_t* ids = p.idx + I.b * p.idx_sb + I.t * p.idx_st;
        // blocks of the row = 1 + (last entry other than -1) / 64, searched from the end
        int last = -1;
        for (int e0 = p.kk - 1; e0 >= 0 && last < 0; e0 -= 32 * 8) {
          int v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int e = e0 - u * 32 - lane;
            v[u] = e >= 0 ? __ldg(ids + e) : -1;
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint32_t bal = __ballot_sync(0xffffffffu, v[u] != -1);
            if (last < 0 && bal) last = e0 - u * 32 - (__ffs(bal) - 1);
          }
        }
        const int nbr = (last + kNB) / kNB;
        const int j0 = (int)((int64_t)I.split * nbr / p.splits);
        return {ids, I.b, j0, (int)((int64_t)(I.split + 1) * nbr / p.splits) - j0, 0};
      };
      Blocks cur{}, next{};
      // The blocks behind `cur` of a tile that goes on.  (Chosen inside blocks_of, or in a function around both, a prompt of 4,096
      // FP8 rows took 2% longer.)
      auto rest_of = [&](int tile) -> Blocks {
        const int j0 = cur.j0 + cur.nb;
        return {nullptr, cur.b, j0, min(tile_end(tile, cur.sees) - j0, kMaxBlocks), cur.sees};
      };
      // (Of a part the row is taken to be full while its end is looked for: its ids are then there a latency earlier, 29.5 ->
      // 28.3 us a 32-sequence decode step out of L2.  In the kernel that walks many rows the code cost 3%.)
      int id_0[2], id_2[2], id[2];
      bool guessed = false;
      // Below, block j >= cur.nb is the next item's block j - cur.nb.
      auto load_ids = [&](int j, int (&id)[2]) {
        const bool here = j < cur.nb;
        const int32_t* ids = here ? cur.ids : next.ids;
        const int jb = here ? j : j - cur.nb, e0 = (int)((uint32_t)((here ? cur.j0 : next.j0) + jb) * kNB) + lane;
        const bool in = jb < (here ? cur.nb : next.nb);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (kDense) id[u] = in && e0 + u * 32 < (here ? cur.sees : next.sees) ? e0 + u * 32 : -1;
          else id[u] = in && e0 + u * 32 < p.kk ? __ldg(ids + e0 + u * 32) : -1;
        }
      };
      auto load_pages = [&](int j, const int (&id)[2], int (&page)[2], int (&off)[2]) {
        const int b = j < cur.nb ? cur.b : next.b;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          off[u] = -1;
          if (id[u] >= 0 && id[u] < p.S) page[u] = latent_page(p.cache, b, id[u], off[u]);
          if (off[u] < 0 && id[u] != -1) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
        }
      };
      auto resolve = [&](const int (&page)[2], const int (&off)[2], int (&row)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          row[u] = off[u] >= 0 ? (int)latent_row_of(p.cache, page[u], off[u]) : -1;
          if (row[u] < 0 && off[u] >= 0) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
        }
      };
      // (Bringing the rows' lines to L2 from here cost more in the load pipe than it saved: 1.15 against
      // 1.09 ms a 4,096-query chunk.)
      auto load_scales = [&](const int (&row)[2], float (&scale)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) scale[u] = row[u] >= 0 ? __ldg(p.cache.scales + row[u]) : 0.f;
      };
      // The four loads behind a block, each on the last one's result (its ids, their pages, the rows'
      // scales; the copies wait for the rows only), are made one of this warp's blocks apart, so a block
      // costs one latency, not all; and so across items.  (One latency after the other took 2,400 cycles
      // a block in a decode step, and 9,000 at the start of every row.)  Only where the item had three
      // blocks or more for this warp; the first blocks of the others' successors wait.
      if constexpr (!kParts) {
        cur = blocks_of(first);
      } else {
        const int first_j = warp - kIxWarp0;  // of this warp
        const Item I = item_of<kForm>(p, first);
        const int most = (p.kk + kNB - 1) / kNB, j0 = (int)((int64_t)I.split * most / p.splits);
        cur = {p.idx + I.b * p.idx_sb + I.t * p.idx_st, I.b, j0, (int)((int64_t)(I.split + 1) * most / p.splits) - j0, 0};
        load_ids(first_j, id_0);
        load_ids(first_j + 2, id_2);
        load_ids(first_j + 4, id);
        const Blocks found = blocks_of(first);
        guessed = found.j0 == cur.j0 && found.nb == cur.nb;
        cur = found;
      }
      int page[2], off[2], row[2];
      float scale[2];
      int it = 0;
      uint32_t g = 0;
      bool ok = true, ahead = false;  // ahead: id, page, off, row and scale are the item's
      for (int item = first, told = 0; ok && item < items; item += step(told), ++it) {
        if constexpr (kLong)
          told = (cur.j0 + cur.nb < tile_end(item, cur.sees) ? kGoesOn : 0) | (cur.j0 > tile_begin(item) ? kBegan : 0);
        if (warp == kIxWarp0) {
          if (!(ok = wait(&bar.info_empty[it & 1], ((it >> 1) & 1) ^ 1))) break;
          if (lane == 0) {
            sm->nb[it & 1] = cur.nb | told;
            if constexpr (kDense) {
              sm->j0[it & 1] = cur.j0;
              sm->sees[it & 1] = cur.sees;
              const int len = __ldg(p.lens + cur.b);
              if (len < 0 || len > p.S) atomicOr(p.flags, DSA_FLAG_BAD_INDEX);
            }
            mbar_arrive(&bar.info_full[it & 1]);
          }
        }
        int j = (int)((g ^ (uint32_t)(warp - kIxWarp0)) & 1u);  // this warp's blocks: g + j even or odd
        if (!ahead && j < cur.nb) {
          if (!kParts || !guessed) {
            load_ids(j, id_0);
            load_ids(j + 2, id_2);
            load_ids(j + 4, id);
          }
          load_pages(j, id_0, page, off);
          resolve(page, off, row);
          load_scales(row, scale);
          load_pages(j + 2, id_2, page, off);
        }
        guessed = false;
        int known = item + step(told) < items ? 0 : 3;  // the last loads that saw the blocks of this or the next item
        bool seen = known != 0;                // the next item's blocks are known
        next.nb = 0;
        for (; j < cur.nb; j += 2) {
          const int ri = (int)((g + j) % kRing);
          if (!(ok = wait(&bar.ix_empty[ri], (((g + j) / kRing) & 1) ^ 1))) break;
          sm->row[ri][lane] = row[0];
          sm->row[ri][32 + lane] = row[1];
          const bool some = __any_sync(0xffffffffu, row[0] >= 0 || row[1] >= 0);
          if (lane == 0) sm->valid[ri] = some;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.ix_row[ri]);  // the copies do not wait for the scales
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = u * 32 + lane;
            float* sc = reinterpret_cast<float*>(&sm->sc[ri][r >> 1]) + (r & 1);
            sc[0] = row[u] >= 0 ? scale[u] : 0.f;
            sc[2] = row[u] >= 0 ? log2f(scale[u]) : -INFINITY;
            const float inv = row[u] >= 0 ? 1.f / scale[u] : 0.f;
            // (always finite, the largest float instead of a NaN: it leaves the zero weights of a tile's tokens that do not see
            // the row at zero, and those that do have a NaN weight by its scale alone)
            sm->isc[ri][r] = kDense ? fminf(inv, 0x1.fffffep127f) : inv;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.ix_full[ri]);
          resolve(page, off, row);
          load_scales(row, scale);
          load_pages(j + 4, id, page, off);
          load_ids(j + 6, id);
          known = j + 6 < cur.nb || seen ? known + 1 : 0;
          if (!seen && j + 8 >= cur.nb) {
            if (kLong && (told & kGoesOn)) next = rest_of(item);
            else next = blocks_of(item + G);
            seen = true;
          }
        }
        if (kLong && !seen && (told & kGoesOn)) next = rest_of(item);
        else if (!seen) next = blocks_of(item + G);
        ahead = known >= 3;
        g += cur.nb;
        cur = next;
      }
    }
    finish(false);
  } else if (warp < kOWarp0) {
    reg_inc<Regs<kFour>::kSm>();
    // ================= softmax =================
    const int hgp = 2 * (warp & 3) + ((warp - kSmWarp0) >> 2);  // this warp's 8 heads
    const int hl = hgp * 8 + (lane >> 2), m = lane & 3;         // this thread's head; keys 8j + 2m + {0, 1}
    const uint32_t s_addr = tmem + kColS + ((uint32_t)((warp & 3) * 32 + ((warp - kSmWarp0) >> 2) * 16) << 16);
    int it = 0, oc = 0;
    uint32_t g = 0;
    bool ok = true;
    // of this thread's head, of a tile in several items: what the loop over its blocks keeps from one to the next, and the power
    // of two that O was held under when it was last added to memory
    [[maybe_unused]] float kept_E0, kept_l, kept_lost, E_added;
    [[maybe_unused]] int kept_valid;
    for (int item = first, told = 0; ok && item < items; item += step(told), ++it) {
      if (!(ok = wait(&bar.info_full[it & 1], (it >> 1) & 1))) break;
      told = sm->nb[it & 1];
      const int nb = blocks_told(told);
      // Of a tile of several tokens: the keys of the item's first block on that this thread's head sees (its last
      // token's are all there are).
      int left = INT_MAX;
      if constexpr (kDense) {
        const Item I = item_of<kForm>(p, item);
        if (p.causal && p.tile_t > 1) left = sm->sees[it & 1] - (I.last - I.t - min(hl / p.H, I.last - I.t)) - sm->j0[it & 1] * kNB;
      }
      float cq = 0.f;
      if (nb) {
        if (!(ok = wait(&bar.qs_full[oc & 1], (oc >> 1) & 1))) break;
        cq = sm->qs[oc & 1][hl] * (p.scale * kLog2e);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.info_empty[it & 1]);
      if (nb == 0) continue;
      float E0 = -INFINITY, l = 0.f, lost = 0.f;
      int any_valid = 0;
      if constexpr (kLong)
        if (told & kBegan) E0 = kept_E0, l = kept_l, lost = kept_lost, any_valid = kept_valid;
      for (int j = 0; j < nb; ++j, ++g) {
        const int ri = (int)(g % kRing), pb = (int)(g & 1);
        // the block's scales, the release of P(g - 2) (and with it of its scales), the scores.  (Uniform
        // waits, one by one: a barrier per lane, for one latency in all, took 2,530 cycles a block, not 2,170.)
        if (kPoll || !__all_sync(0xffffffffu, try_wait3(&bar.ix_full[ri], (g / kRing) & 1, &bar.p_empty[pb], ((g >> 1) & 1) ^ 1,
                                                        &bar.s_full, g & 1)))
          if (!(ok = wait(&bar.ix_full[ri], (g / kRing) & 1) && wait(&bar.p_empty[pb], ((g >> 1) & 1) ^ 1) && wait(&bar.s_full, g & 1)))
            break;
        uint32_t r[32];
        tc_fence_after();
        tmem_ld_16x256b_x8(s_addr, r);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_empty);
        any_valid |= sm->valid[ri];
        f32x2 y[8];
        float ymax = -INFINITY;
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          const float4 s = sm->sc[ri][4 * jj + m];
          const f32x2 t = fma_2(pair(__uint_as_float(r[4 * jj + 2]), __uint_as_float(r[4 * jj + 3])), pair(0.0625f, 0.0625f),
                                pair(__uint_as_float(r[4 * jj]), __uint_as_float(r[4 * jj + 1])));
          y[jj] = fma_2(t, mul_2(pair(cq, cq), pair(s.x, s.y)), pair(s.z, s.w));
          if constexpr (!kDense) ymax = max3(ymax, lo_of(y[jj]), hi_of(y[jj]));
        }
        if constexpr (kDense) {
          if (__any_sync(0xffffffffu, left < kNB)) {
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
              const int k0 = 8 * jj + 2 * m;
              y[jj] = pair(k0 < left ? lo_of(y[jj]) : -INFINITY, k0 + 1 < left ? hi_of(y[jj]) : -INFINITY);
            }
          }
          left -= left == INT_MAX ? 0 : kNB;
#pragma unroll
          for (int jj = 0; jj < 8; ++jj) ymax = max3(ymax, lo_of(y[jj]), hi_of(y[jj]));
        }
        ymax = fmaxf(ymax, __shfl_xor_sync(0xffffffffu, ymax, 1));
        ymax = fmaxf(ymax, __shfl_xor_sync(0xffffffffu, ymax, 2));
        const float E = ceilf(ymax) - 8.f;  // -inf: no weight in this block
        const bool move = E > E0 + (kDense ? kMoveAll : kMove);  // (E0 starts at -inf)
        const float alpha = move ? ex2(E0 - E) : 1.f;
        const int any = __any_sync(0xffffffffu, move);
        E0 = move ? E : E0;
        const float d = fmaxf(E - E0, -120.f);  // beside 2^0, nothing is left of 2^-120
        if (m == 0) {
          sm->sf[pb][hl] = (uint32_t)(127 + (int)d) * 0x01010101u;  // of all four key steps
          if (any) sm->alpha[pb][hl] = alpha;
        }
        __syncwarp();
        if (lane == 0) {
          sm->need[pb][hgp] = (uint8_t)(any != 0);
          mbar_arrive(&bar.m_full[pb]);
        }
        const float eu = E == -INFINITY ? 0.f : E;
        f32x2 sum2 = 0;
        const uint32_t at = smem_addr(p_s + pb * kPBytes + hl * 128) + ((hl & 7) << 4) + 2 * m;
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          const f32x2 x = add_2(y[jj], pair(-eu, -eu));
          const float p0 = ex2(lo_of(x)), p1 = ex2(hi_of(x));
          const float2 is = *reinterpret_cast<const float2*>(&sm->isc[ri][8 * jj + 2 * m]);
          sum2 = fma_2(pair(p0, p1), pair(is.x, is.y), sum2);
          const uint32_t h = f16x2(p0, p1);
          const uint16_t hi = e4m3_of_f16x2(h);
          const uint16_t lo = e4m3_of_f16x2(sub_f16x2(h, f16x2_of_e4m3(hi)));
          asm volatile("st.shared.b16 [%0], %1;\n" ::"r"((at ^ ((jj >> 1) << 4)) + (jj & 1) * 8), "h"(hi) : "memory");
          asm volatile("st.shared.b16 [%0], %1;\n" ::"r"((at ^ ((4 + (jj >> 1)) << 4)) + (jj & 1) * 8), "h"(lo) : "memory");
        }
        const float sum = lo_of(sum2) + hi_of(sum2);
        const float f = E == -INFINITY ? 0.f : ex2(E - E0);
        if constexpr (kDense) {
          // of up to 2^25 blocks: with what the last sum lost (Kahan 1965), or 4 million equal weights are off by 2^-8
          const float term = fmaf(sum, f, -lost * alpha), last = l * alpha;
          l = last + term;
          lost = (l - last) - term;
        } else {
          l = fmaf(sum, f, l * alpha);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.p_full[pb]);
          mbar_arrive(&bar.ix_empty[ri]);
        }
      }
      if (!ok) break;
      if constexpr (kLong) {
        if (told & kGoesOn) kept_E0 = E0, kept_l = l, kept_lost = lost, kept_valid = any_valid;
      }
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (!any_valid) l = 0.f;
      if (!(ok = wait(&bar.l_empty[oc & 1], ((oc >> 1) & 1) ^ 1))) break;
      if constexpr (kLong) {
        if (m == 0) {
          sm->carry[oc & 1][hl] = ex2(E_added - E0);
          if (told & kGoesOn) sm->lsum[oc & 1][hl] = l == 0.f ? 0.f : 1.f;
        }
        E_added = E0;
      }
      if (m == 0 && !(kLong && (told & kGoesOn))) {
        sm->lsum[oc & 1][hl] = l == 0.f ? 0.f : 1.f / l;
        const Item I = item_of<kForm>(p, item);
        const float v = l == 0.f ? -INFINITY : (E0 + log2f(l)) * kLn2;
        const int slot = kDense ? sm->share.slot(item) : -1;
        if (kParts) sm->part_lse[hl] = v;
        else if (slot >= 0) p.parts[(int64_t)slot * kPartFloats + kHg * kLatentDim + hl] = v;
        else if (p.lse && hl < I.heads) p.lse[(int64_t)I.row * p.H + I.h0 + hl] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.l_full[oc & 1]);
      ++oc;
    }
    finish(false);
  } else {
    if constexpr (Regs<kFour>::kEpi < Regs<kFour>::kLaunch) reg_dec<Regs<kFour>::kEpi>();
    if (warp < kQWarp0) {
      // ================= O^T: block scales, half of the epilogue =================
      const int t = threadIdx.x - kOWarp0 * 32;
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      tmem_st_x2(tmem + lane_base + kColSfA, 0x7f7f7f7fu, 0x7f7f7f7fu);  // V as it stands
      tmem_st_x2(tmem + lane_base + kColSfA + 2, 0x7f7f7f7fu, 0x7f7f7f7fu);
      tmem_wait_stores();
      tc_fence_before();
      int it = 0, oc = 0;
      uint32_t g = 0;
      bool ok = true;
      for (int item = first, told = 0; ok && item < items; item += step(told), ++it) {
        if (!(ok = wait(&bar.info_full[it & 1], (it >> 1) & 1))) break;
        told = sm->nb[it & 1];
        const int nb = blocks_told(told);
        // (FP8 rows) Keys of the item from `hidden` on, up to `hidden_end`, are not seen by every token of the tile.
        int hidden = INT_MAX, hidden_end = 0;
        if constexpr (kForm > kAll && !kFour) {
          if (p.causal && p.tile_t > 1) {
            const Item I = item_of<kForm>(p, item);
            hidden_end = sm->sees[it & 1] - sm->j0[it & 1] * kNB;
            hidden = max(0, hidden_end - (I.last - I.t));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.info_empty[it & 1]);
        if (nb == 0) {  // nothing selected: O = 0, LSE = -inf
          const Item I = item_of<kForm>(p, item);
          uint16_t* og = p.out + ((int64_t)I.row * p.H + I.h0) * kLatentDim;
          if (kParts) {  // (no part is read whose weight is 0)
            if (t < kHg) sm->part_lse[t] = -INFINITY;
          } else {
            for (int i = t; i < I.heads * kLatentDim / 8; i += 128) reinterpret_cast<uint4*>(og)[i] = make_uint4(0, 0, 0, 0);
            if (p.lse && t < I.heads) p.lse[(int64_t)I.row * p.H + I.h0 + t] = -INFINITY;
          }
          continue;
        }
        for (int j = 0; j < nb; ++j, ++g) {
          // told at every block, when its scales are known and its weights are not yet formed
          if (!(ok = wait(&bar.m_full[g & 1], (g >> 1) & 1))) break;
          const bool need = j > 0 && __any_sync(0xffffffffu, *reinterpret_cast<const volatile uint64_t*>(sm->need[g & 1]) != 0);
          if (need) {
            // O^T complete up to the block before: rescale the heads whose E0 moved
            if (!(ok = wait(&bar.p_empty[(g - 1) & 1], ((g - 1) >> 1) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int w = 0; w < 8; ++w) {
              if (!sm->need[g & 1][w]) continue;
              const float4 a0 = *reinterpret_cast<const float4*>(&sm->alpha[g & 1][8 * w]);
              const float4 a1 = *reinterpret_cast<const float4*>(&sm->alpha[g & 1][8 * w + 4]);
              const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
              uint32_t v[4][8];
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_ld_x8(tmem + lane_base + kColO + c * kHg + 8 * w, v[c]);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] = __float_as_uint(__uint_as_float(v[c][i]) * a[i]);
                tmem_st_x8(tmem + lane_base + kColO + c * kHg + 8 * w, v[c]);
              }
            }
          }
          if (kForm > kAll && !kFour && j * kNB + kNB - 1 >= hidden) {
            // Weights of rows that a token does not see are zero, which times a NaN code would still reach its values.  The
            // scores have been taken of those codes, so that tokens which see them have NaN weights: zeros in their place.
            if (!(ok = wait(&bar.kv_full[g % kStages], (g / kStages) & 1))) break;
#pragma unroll 1
            for (int r = max(0, hidden - j * kNB) + (warp & 3); r < min(kNB, hidden_end - j * kNB); r += 4)
              drop_nan_codes(smem_addr(kv_s) + g % kStages * kStage + (lane >> 3) * kAtom + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            async_fence();
          }
          // the block's scales (the products that read this buffer's last ones are done: the softmax
          // waited for them before it wrote these)
          tmem_st_x2(tmem + lane_base + kColSfB + 4 * (g & 1), sm->sf[g & 1][lane], sm->sf[g & 1][32 + lane]);
          tmem_wait_stores();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sf_full[g & 1]);
        }
        if (!ok || !(ok = epilogue(item, oc, told))) break;
        ++oc;
      }
      meet_last(ok);
    } else {
      // ================= queries: hi and lo rows; half of the epilogue =================
      const int qw = warp - kQWarp0;
      int it = 0, oc = 0;
      int last = -1, last_told = 0;  // the item whose O is still to be stored
      bool ok = true;
      for (int item = first, told = 0; item < items || last >= 0; item += step(told), ++it) {
        int nb = told = 0;
        if (item < items) {
          if (it > 0) convert(item, qw, 4);
          ok = wait(&bar.info_full[it & 1], (it >> 1) & 1);
          told = ok ? sm->nb[it & 1] : 0;
          nb = blocks_told(told);
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bar.info_empty[it & 1]);
          if (kForm == kRows && qw == 0 && nb <= kFetchBlocks && item + G < items && p.H > kFetchHeads) fetch(item + G);
          if (ok && nb) ok = wait(&bar.q_empty, (oc & 1) ^ 1);
          if (named_sync_or(2, 128, !ok)) {  // all rows are there; the four warps go on or leave together
            ok = false;
            break;
          }
          if (nb) {
            if (lane < 16) sm->qs[oc & 1][16 * qw + lane] = sm->qnext[16 * qw + lane];
            if (it > 0) {
              tc_fence_after();
              copy_q(0, 5);
            }
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bar.qs_full[oc & 1]);
              mbar_arrive(&bar.q_full);
            }
          }
          named_sync(2, 128);  // the room has been read
        }
        // the O warps wait in the last item's epilogue: join them before any wait on a later item
        // than this one, whose publication they hold up
        if (last >= 0 && !(ok = epilogue(last, oc - 1, last_told))) break;
        if (nb) ++oc;
        last = nb ? item : -1;
        last_told = told;
      }
      meet_last(ok);
      asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    }
    finish(true);
  }

  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.flags, DSA_FLAG_TIMEOUT);
}
static_assert(kColQR == kColQ + 128, "the converted query row is stored in one run of columns");

// A launch whose CTAs work in clusters of n on a row each.
template <bool kFour>
cudaLaunchConfig_t launch_config(int ctas, int n, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)ctas);
  c.blockDim = dim3(kThreads<kFour>);
  c.dynamicSmemBytes = kSmem;
  c.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)n;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  c.attrs = attr;
  c.numAttrs = n > 1;
  return c;
}

// Shared memory for a kernel, and that a block is launched with the registers that its warpgroups' moves count on.
template <bool kFour>
cudaError_t prepare_kernel(void (*kern)(LatentAttnLaunch)) {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != Regs<kFour>::kLaunch) return cudaErrorInvalidKernelImage;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
}

// What the launcher knows of a device, found out once: the clusters of n CTAs that fit on it at a time.
struct ClusterRoom {
  int clusters[kMaxLatentSplits + 1];
};

template <bool kFour>
auto kernel_of(bool poll, bool parts) {
  return poll ? (parts ? k_latent_attn<true, kRowParts, kFour> : k_latent_attn<true, kRows, kFour>)
              : (parts ? k_latent_attn<false, kRowParts, kFour> : k_latent_attn<false, kRows, kFour>);
}

// Whether index rows of kk entries are worth n parts: about 128 keys a part (one block at least), and the
// keys of six blocks less for a CTA to walk, which is what leaving and joining the parts takes.  Unsplit
// against split as by the first condition alone, us (64 heads; the inputs in L2):
//   kk           129          192          257          384          448          512          768
//   1 row        11.5 / 16.7  11.5 / 16.7  13.6 / 16.2  14.6 / 16.3  15.5 / 15.8  16.5 / 15.8  20.7 / 16.0
//   16 rows      11.7 / 17.3  11.6 / 17.3  13.7 / 16.5  14.6 / 16.5  15.7 / 16.1  16.6 / 16.0  20.9 / 16.7
//   70 (2 parts) 12.1 / 18.5  12.2 / 18.3  14.3 / 19.5  15.3 / 19.6  16.4 / 20.6  17.3 / 20.6  21.8 / 23.0
// and 70 rows of 1,024 25.5 / 25.2, of 2,048 43.7 / 35.4.
inline bool splits_pay(int kk, int n) {
  const int blocks = (kk + kNB - 1) / kNB;
  return n <= (kk + 127) / 128 && kk - (blocks + n - 1) / n * kNB >= 6 * kNB;
}

// Once per device: the kernels, and the clusters.
template <bool kFour>
cudaError_t prepare_kernels(ClusterRoom& room) {
  static ClusterRoom rooms[64];
  static std::atomic<int> state[64];  // 0: unknown, 1: being written, 2: known
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && state[dev].load(std::memory_order_acquire) == 2) {
    room = rooms[dev];
    return cudaSuccess;
  }
  for (int k = 0; k < 4; ++k)
    if ((e = prepare_kernel<kFour>(kernel_of<kFour>(k & 1, k & 2))) != cudaSuccess) return e;
  for (int n = 2; n <= kMaxLatentSplits; ++n) {
    cudaLaunchAttribute attr{};
    const cudaLaunchConfig_t c = launch_config<kFour>(n, n, nullptr, &attr);
    if ((e = cudaOccupancyMaxActiveClusters(&room.clusters[n], kernel_of<kFour>(false, true), &c)) != cudaSuccess) return e;
  }
  int unknown = 0;
  if (kept && state[dev].compare_exchange_strong(unknown, 1)) {
    rooms[dev] = room;
    state[dev].store(2, std::memory_order_release);
  }
  return cudaSuccess;
}

// Attention over index rows.
template <bool kFour>
cudaError_t launch_rows(LatentAttnLaunch p, cudaStream_t st) {
  TraceScope trace(kTraceAttention, st);
  p.groups = (p.H + kHg - 1) / kHg;
  p.wait = wait_limit();
  const bool poll = p.wait < kDefaultWaitCycles;
  ClusterRoom room{};
  cudaError_t e = prepare_kernels<kFour>(room);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.B * p.T * p.groups;
  p.splits = 1;
  for (int n = 2; n <= kMaxLatentSplits; ++n)
    if (rows <= room.clusters[n] && splits_pay(p.kk, n)) p.splits = n;
  const int sms = device_sm_count();
  // Tokens that share an index row, their queries side by side: one token of all their heads, so that rows of few heads fill
  // tiles together (k 2,048, 1,024 tokens of 1 / 16 / 40 heads: 297 -> 47, 297 -> 91, 303 -> 212 us; FP8 259 -> 42, 263 -> 82,
  // 267 -> 191).  Not where there is an SM for every row as it is.  A head's results do not depend on what shares its tile.
  if (rows > sms && p.idx_st == 0 && p.q_st == (int64_t)p.H * kD && (int64_t)p.T * p.H <= INT_MAX - kHg) {
    p.H *= p.T;
    p.T = 1;
    p.groups = (p.H + kHg - 1) / kHg;
  }
  const int64_t items = (int64_t)p.B * p.T * p.groups * p.splits;
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t cfg = launch_config<kFour>((int)(p.splits > 1 || items < sms ? items : sms), p.splits, st, &attr);
  if ((e = cudaLaunchKernelEx(&cfg, kernel_of<kFour>(poll, p.splits > 1), p)) != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dsa
