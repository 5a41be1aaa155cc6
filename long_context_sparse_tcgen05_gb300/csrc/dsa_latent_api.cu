// Entry points of the serving operators around the sparse attention path: per-head norm and
// rotation, the paged FP8 latent cache, and attention over it.  Host validation and launches only.
#include <atomic>
#include <climits>
#include <cstdarg>
#include <cstdio>

#include "dsa_internal.cuh"

namespace {

dsa_status fail(dsa_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
dsa_status fail(dsa_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return dsa::record_error(s, buf);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

dsa_status check_ws(const void* ws, size_t ws_bytes) {
  if (!ws) return fail(DSA_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 16)) return fail(DSA_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  if (ws_bytes < DSA_WS_MIN) return fail(DSA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, DSA_WS_MIN);
  return DSA_OK;
}

uint32_t* ws_flags(void* ws) { return reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + dsa::kWsFlags); }

dsa_status done(cudaError_t e, const char* what) {
  return e == cudaSuccess ? DSA_OK : fail(DSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Kernels count a call's rows in 32 bits.
dsa_status check_count(int64_t rows, int64_t per) {
  if (rows > INT_MAX / per) return fail(DSA_ERR_UNSUPPORTED, "%lld tokens are too many for one call", (long long)rows);
  return DSA_OK;
}

// Positions that the host knows: rows [pos0, pos0 + n) of `limit`.
dsa_status check_range(int64_t pos0, int64_t n, int64_t limit, const char* what) {
  if (pos0 < 0 || (limit > 0 && pos0 > limit - n))
    return fail(DSA_ERR_INVALID_ARG, "positions [%lld, %lld) fall outside the %lld rows of %s", (long long)pos0,
                (long long)pos0 + n, (long long)limit, what);
  return DSA_OK;
}

// The checks both norm entry points share; fills the launch but for its output.
dsa_status norm_rope_launch(const dsa_norm_rope_args* a, dsa::NormRopeLaunch& P) {
  if (!a) return fail(DSA_ERR_INVALID_ARG, "norm args are NULL");
  if (a->B < 1 || a->n < 0 || a->H < 1) return fail(DSA_ERR_INVALID_ARG, "B >= 1, n >= 0 and H >= 1 are required");
  if (!a->x) return fail(DSA_ERR_INVALID_ARG, "x is NULL");
  if (a->d < 8 || a->d > 1024 || a->d % 8)
    return fail(DSA_ERR_UNSUPPORTED, "d = %d; a multiple of 8 in [8, 1024] is required", a->d);
  if (a->norm != DSA_NORM_NONE && a->norm != DSA_NORM_RMS && a->norm != DSA_NORM_LAYER)
    return fail(DSA_ERR_INVALID_ARG, "unknown norm %d", (int)a->norm);
  if (a->norm != DSA_NORM_NONE && !(a->eps >= 0.f)) return fail(DSA_ERR_INVALID_ARG, "eps must be >= 0");
  if (a->norm == DSA_NORM_NONE && (a->weight || a->bias))
    return fail(DSA_ERR_INVALID_ARG, "weight and bias need a norm");
  if (a->bias && a->norm != DSA_NORM_LAYER) return fail(DSA_ERR_INVALID_ARG, "bias needs the layer norm");
  if (a->x_stride_b < 0 || a->x_stride_t < 0 || a->x_stride_h < 0)
    return fail(DSA_ERR_INVALID_ARG, "strides must be >= 0 (0: dense)");
  if (a->x_stride_h && a->x_stride_h < a->d) return fail(DSA_ERR_INVALID_ARG, "x_stride_h is smaller than d");
  if (a->rope_dim < 0 || a->rope_off < 0 || (int64_t)a->rope_off + a->rope_dim > a->d)
    return fail(DSA_ERR_INVALID_ARG, "rotated values [%d, %d + %d) fall outside the head's %d", a->rope_off, a->rope_off,
                a->rope_dim, a->d);
  if (a->rope_dim > 0) {
    const int unit = a->interleaved ? 8 : 16;
    if (a->rope_dim % unit || a->rope_off % 8)
      return fail(DSA_ERR_UNSUPPORTED, "rope_off must be a multiple of 8 and rope_dim of %d", unit);
    if (!a->cos || !a->sin) return fail(DSA_ERR_INVALID_ARG, "a rotation needs cos and sin");
    if (a->max_pos < 1) return fail(DSA_ERR_INVALID_ARG, "max_pos must be >= 1");
    if (!aligned(a->cos, 16) || !aligned(a->sin, 16)) return fail(DSA_ERR_MISALIGNED, "cos and sin must be 16-byte aligned");
  }
  if (!aligned(a->x, 16) || a->x_stride_b % 8 || a->x_stride_t % 8 || a->x_stride_h % 8)
    return fail(DSA_ERR_MISALIGNED, "x must be 16-byte aligned, its strides multiples of 8 elements");
  if (!aligned(a->weight, 16) || !aligned(a->bias, 16))
    return fail(DSA_ERR_MISALIGNED, "weight and bias must be 16-byte aligned");
  if (!aligned(a->positions, 8)) return fail(DSA_ERR_MISALIGNED, "positions must be 8-byte aligned");
  // (a warp of the kernel takes at least four heads of a token, of wide heads one)
  dsa_status s = check_count((int64_t)a->B * a->n, a->d <= 256 ? a->H / 4 + 1 : a->H);
  if (s != DSA_OK || (!a->positions && (s = check_range(a->pos0, a->n, 0, "the tokens")) != DSA_OK)) return s;
  P.B = a->B; P.n = a->n; P.H = a->H; P.d = a->d;
  P.x = static_cast<const uint16_t*>(a->x);
  P.x_sh = a->x_stride_h ? a->x_stride_h : a->d;
  P.x_st = a->x_stride_t ? a->x_stride_t : a->H * P.x_sh;
  P.x_sb = a->x_stride_b ? a->x_stride_b : a->n * P.x_st;
  P.norm = a->norm; P.eps = a->eps; P.weight = a->weight; P.bias = a->bias;
  P.cos = a->cos; P.sin = a->sin;
  P.rope_off = a->rope_off; P.rope_dim = a->rope_dim; P.interleaved = a->interleaved != 0;
  P.limit = a->rope_dim > 0 ? a->max_pos : 0;
  P.positions = a->positions; P.pos0 = a->pos0;
  return DSA_OK;
}

// The checks every call on a cache of B sequences makes; fills the device view.
dsa_status cache_view(const dsa_latent_cache* c, int B, dsa::LatentCacheView& v) {
  if (!c) return fail(DSA_ERR_INVALID_ARG, "the cache is NULL");
  if (!c->codes || !c->scales || !c->rope) return fail(DSA_ERR_INVALID_ARG, "cache codes, scales and rope must be non-NULL");
  if (c->n_pages < 1 || c->page_size < 1) return fail(DSA_ERR_INVALID_ARG, "n_pages and page_size must be >= 1");
  if (c->block_table ? c->table_ld < 1 : c->n_pages < B)
    return fail(DSA_ERR_INVALID_ARG, c->block_table ? "table_ld must be >= 1" : "without a block table n_pages must cover the sequences");
  if (!aligned(c->codes, 16) || !aligned(c->rope, 16) || !aligned(c->scales, 4) || !aligned(c->block_table, 4))
    return fail(DSA_ERR_MISALIGNED, "cache codes and rope need 16-byte alignment, scales and block_table 4-byte");
  v.codes = c->codes; v.groups = nullptr; v.scales = c->scales; v.rope = static_cast<uint16_t*>(c->rope);
  v.table = c->block_table; v.table_ld = c->table_ld; v.page_size = c->page_size; v.n_pages = c->n_pages;
  v.cap = c->block_table ? (int64_t)c->table_ld * c->page_size : c->page_size;
  if (v.cap > INT_MAX) v.cap = INT_MAX;
  return DSA_OK;
}

// The 4-bit cache's view, by the same checks.
dsa_status cache_view(const dsa_latent4_cache* c, int B, dsa::LatentCacheView& v) {
  if (!c) return fail(DSA_ERR_INVALID_ARG, "the cache is NULL");
  const dsa_latent_cache as{c->n_pages, c->page_size, c->table_ld, c->codes, c->scales, c->rope, c->block_table};
  const dsa_status s = cache_view(&as, B, v);
  if (s != DSA_OK) return s;
  if (!c->groups) return fail(DSA_ERR_INVALID_ARG, "cache groups must be non-NULL");
  v.groups = c->groups;
  return DSA_OK;
}

// Attention args of either cache; k: entries of an index row, 0 without index rows.
template <class Args>
dsa_status latent_attn_launch(const Args* a, int32_t k, bool dense, dsa::LatentAttnLaunch& L) {
  if (!a) return fail(DSA_ERR_INVALID_ARG, "attention args are NULL");
  if (a->B < 1 || a->T < 1 || a->S < 1) return fail(DSA_ERR_INVALID_ARG, "B, T and S must be positive");
  if (a->H < 1 || a->H > 128) return fail(DSA_ERR_UNSUPPORTED, "H = %d outside [1, 128]", a->H);
  if (!dense && (k < 1 || k > 65536)) return fail(DSA_ERR_UNSUPPORTED, "k = %d outside [1, 65536]", k);
  if ((int64_t)a->B * a->T > (1 << 24)) return fail(DSA_ERR_UNSUPPORTED, "B * T = %lld queries; at most 2^24", (long long)a->B * a->T);
  if (!dense && a->idx_T != 1 && a->idx_T != a->T) return fail(DSA_ERR_INVALID_ARG, "idx_T = %d is neither 1 nor T = %d", a->idx_T, a->T);
  if (!(a->scale > 0.f) || a->scale > 3.4e38f) return fail(DSA_ERR_INVALID_ARG, "scale must be positive and finite");
  if (!a->q) return fail(DSA_ERR_INVALID_ARG, "q is NULL");
  if (a->q_stride_b < 0 || a->q_stride_t < 0) return fail(DSA_ERR_INVALID_ARG, "strides must be >= 0 (0: dense)");
  if (a->q_stride_t && a->q_stride_t < (int64_t)a->H * 576) return fail(DSA_ERR_INVALID_ARG, "q_stride_t is smaller than H * 576");
  if (!aligned(a->q, 16) || a->q_stride_b % 8 || a->q_stride_t % 8)
    return fail(DSA_ERR_MISALIGNED, "q must be 16-byte aligned, its strides multiples of 8 elements");
  dsa_status s = cache_view(&a->cache, a->B, L.cache);
  if (s != DSA_OK) return s;
  if (a->S > L.cache.cap)
    return fail(DSA_ERR_INVALID_ARG, "S = %d exceeds the %lld rows a sequence of the cache holds", a->S, (long long)L.cache.cap);
  L.B = a->B; L.T = a->T; L.S = a->S; L.H = a->H; L.scale = a->scale;
  L.q = static_cast<const uint16_t*>(a->q);
  L.q_st = a->q_stride_t ? a->q_stride_t : (int64_t)a->H * 576;
  L.q_sb = a->q_stride_b ? a->q_stride_b : a->T * L.q_st;
  L.kk = k;
  L.idx_st = a->idx_T == 1 ? 0 : k;
  L.idx_sb = (int64_t)a->idx_T * k;
  return DSA_OK;
}

template <class Cache>
dsa_status append_rows(const dsa_latent_append_args* a, const Cache* cache, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return fail(DSA_ERR_INVALID_ARG, "append args are NULL");
  if (a->B < 1 || a->n < 0) return fail(DSA_ERR_INVALID_ARG, "B >= 1 and n >= 0 are required");
  if (dsa_status c = check_count((int64_t)a->B * a->n, 1)) return c;
  if (!a->x) return fail(DSA_ERR_INVALID_ARG, "x is NULL");
  if (!a->cos != !a->sin) return fail(DSA_ERR_INVALID_ARG, "cos and sin go together");
  if (a->cos && a->max_pos < 1) return fail(DSA_ERR_INVALID_ARG, "max_pos must be >= 1");
  if (a->weight && !(a->eps >= 0.f)) return fail(DSA_ERR_INVALID_ARG, "eps must be >= 0");
  if (a->x_stride_b < 0 || a->x_stride_t < 0) return fail(DSA_ERR_INVALID_ARG, "strides must be >= 0 (0: dense)");
  if (a->x_stride_t && a->x_stride_t < 576) return fail(DSA_ERR_INVALID_ARG, "x_stride_t is smaller than 576");
  if (!aligned(a->x, 16) || a->x_stride_b % 8 || a->x_stride_t % 8)
    return fail(DSA_ERR_MISALIGNED, "x must be 16-byte aligned, its strides multiples of 8 elements");
  if (!aligned(a->weight, 16) || !aligned(a->cos, 8) || !aligned(a->sin, 8) || !aligned(a->positions, 8))
    return fail(DSA_ERR_MISALIGNED, "weight needs 16-byte alignment, cos, sin and positions 8-byte");
  dsa::LatentAppendLaunch P{};
  dsa_status s = cache_view(cache, a->B, P.cache);
  if (s != DSA_OK) return s;
  const int64_t rows = a->cos && a->max_pos < P.cache.cap ? a->max_pos : P.cache.cap;
  if (!a->positions && (s = check_range(a->pos0, a->n, rows, "the table or the cache")) != DSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes)) != DSA_OK) return s;
  P.B = a->B; P.n = a->n;
  P.x = static_cast<const uint16_t*>(a->x);
  P.x_st = a->x_stride_t ? a->x_stride_t : 576;
  P.x_sb = a->x_stride_b ? a->x_stride_b : a->n * P.x_st;
  P.weight = a->weight; P.eps = a->eps; P.cos = a->cos; P.sin = a->sin;
  P.interleaved = a->interleaved != 0; P.max_pos = a->max_pos;
  P.positions = a->positions; P.pos0 = a->pos0;
  P.flags = ws_flags(ws);
  return done(dsa::launch_latent_append(P, static_cast<cudaStream_t>(stream)), "append launch");
}

// Reads rows to P's outputs; their addresses once more, to be checked: two on 16 bytes, one on 4.
template <class Cache>
dsa_status read_rows(const Cache* cache, int32_t B, int32_t n, const int32_t* idx, int64_t pos0, dsa::LatentReadLaunch P,
                const void* wide, const void* wide2, const void* scales, void* ws, size_t ws_bytes, void* stream) {
  if (B < 1 || n < 0) return fail(DSA_ERR_INVALID_ARG, "B >= 1 and n >= 0 are required");
  dsa_status s = check_count((int64_t)B * n, 1);
  if (s != DSA_OK || (s = cache_view(cache, B, P.cache)) != DSA_OK) return s;
  if (!wide || !wide2 || !scales) return fail(DSA_ERR_INVALID_ARG, "outputs must be non-NULL");
  if (!aligned(wide, 16) || !aligned(wide2, 16) || !aligned(scales, 4) || !aligned(idx, 4))
    return fail(DSA_ERR_MISALIGNED, "rows out must be 16-byte aligned, scales and idx 4-byte");
  if (!idx && (s = check_range(pos0, n, P.cache.cap, "the cache")) != DSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes)) != DSA_OK) return s;
  P.B = B; P.n = n; P.idx = idx; P.pos0 = pos0;
  P.flags = ws_flags(ws);
  return done(dsa::launch_latent_read(P, static_cast<cudaStream_t>(stream)), "read launch");
}

// The status of an attention launch over this cache.
dsa_status attended(cudaError_t e, const dsa::LatentCacheView& cache) {
  if (e == cudaErrorInvalidKernelImage)  // (returned by the launcher's own look at the kernels, too)
    return fail(DSA_ERR_CUDA, "attention launch: the kernel is not built for this device, or not with the %d registers a "
                "thread that its warpgroups share out (build it with the package's own build step)", cache.groups ? dsa::kLatent4AttnRegs : dsa::kLatentAttnRegs);
  return done(e, "attention launch");
}

template <class Args>
dsa_status attend(const Args* a, const int32_t* idx, int32_t k, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  dsa::LatentAttnLaunch L{};
  dsa_status s = latent_attn_launch(a, k, false, L);
  if (s != DSA_OK) return s;
  if (!idx || !out) return fail(DSA_ERR_INVALID_ARG, "idx and out must be non-NULL");
  if (!aligned(out, 16) || !aligned(idx, 4) || !aligned(lse, 4) || !aligned(a->flags, 4))
    return fail(DSA_ERR_MISALIGNED, "out must be 16-byte aligned, idx, lse and flags 4-byte");
  if ((s = check_ws(ws, ws_bytes)) != DSA_OK) return s;
  L.idx = idx; L.out = static_cast<uint16_t*>(out); L.lse = lse;
  L.flags = a->flags ? a->flags : ws_flags(ws);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return attended(L.cache.groups ? dsa::launch_latent4_attn(L, st) : dsa::launch_latent_attn(L, st), L.cache);
}

template <class Args>
dsa_status attend_dense(const Args* a, const int32_t* lens, int32_t causal, void* out, float* lse, void* ws, size_t ws_bytes,
                        void* stream) {
  dsa::LatentAttnLaunch L{};
  dsa_status s = latent_attn_launch(a, 0, true, L);
  if (s != DSA_OK) return s;
  if (!lens || !out) return fail(DSA_ERR_INVALID_ARG, "lens and out must be non-NULL");
  if (!aligned(out, 16) || !aligned(lens, 4) || !aligned(lse, 4) || !aligned(a->flags, 4))
    return fail(DSA_ERR_MISALIGNED, "out must be 16-byte aligned, lens, lse and flags 4-byte");
  if ((s = check_ws(ws, ws_bytes)) != DSA_OK) return s;
  const size_t need = dsa::kWsScratch + dsa::latent_dense_scratch(L);
  if (ws_bytes < need) return fail(DSA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  L.lens = lens; L.causal = causal != 0;
  L.out = static_cast<uint16_t*>(out); L.lse = lse;
  L.flags = a->flags ? a->flags : ws_flags(ws);
  return attended(dsa::launch_latent_dense(L, static_cast<uint8_t*>(ws) + dsa::kWsScratch, static_cast<cudaStream_t>(stream)), L.cache);
}

}  // namespace

namespace dsa {
int device_sm_count() {
  static std::atomic<int> count[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < 64 && (n = count[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 1;
  if (dev >= 0 && dev < 64) count[dev].store(n, std::memory_order_relaxed);
  return n;
}
}  // namespace dsa

extern "C" {

dsa_status dsa_norm_rope(const dsa_norm_rope_args* a, void* out, int64_t out_stride_b, int64_t out_stride_t,
                         int64_t out_stride_h, void* ws, size_t ws_bytes, void* stream) {
  dsa::NormRopeLaunch P{};
  dsa_status s = norm_rope_launch(a, P);
  if (s != DSA_OK) return s;
  if (!out) return fail(DSA_ERR_INVALID_ARG, "out is NULL");
  if (out_stride_b < 0 || out_stride_t < 0 || out_stride_h < 0 || (out_stride_h && out_stride_h < a->d))
    return fail(DSA_ERR_INVALID_ARG, "out strides must be >= 0 (0: dense) and out_stride_h at least d");
  if (!aligned(out, 16) || out_stride_b % 8 || out_stride_t % 8 || out_stride_h % 8)
    return fail(DSA_ERR_MISALIGNED, "out must be 16-byte aligned, its strides multiples of 8 elements");
  if (!a->positions && P.limit > 0 && (s = check_range(a->pos0, a->n, P.limit, "cos and sin")) != DSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes)) != DSA_OK) return s;
  P.out = static_cast<uint16_t*>(out);
  P.o_sh = out_stride_h ? out_stride_h : a->d;
  P.o_st = out_stride_t ? out_stride_t : a->H * P.o_sh;
  P.o_sb = out_stride_b ? out_stride_b : a->n * P.o_st;
  P.flags = ws_flags(ws);
  return done(dsa::launch_norm_rope(P, static_cast<cudaStream_t>(stream)), "norm launch");
}

dsa_status dsa_norm_rope_e4m3(const dsa_norm_rope_args* a, uint8_t* codes, float* scales, int32_t S_cap,
                              int32_t at_position, void* ws, size_t ws_bytes, void* stream) {
  dsa::NormRopeLaunch P{};
  dsa_status s = norm_rope_launch(a, P);
  if (s != DSA_OK) return s;
  if (!codes || !scales) return fail(DSA_ERR_INVALID_ARG, "codes and scales must be non-NULL");
  if (S_cap < 1 || (!at_position && S_cap < a->n)) return fail(DSA_ERR_INVALID_ARG, "S_cap = %d rows cannot hold the tokens", S_cap);
  if ((int64_t)a->H * dsa::norm_rope_units(a->d) > 2048)
    return fail(DSA_ERR_UNSUPPORTED, "H = %d heads of d = %d are too wide for one token's scale", a->H, a->d);
  if (!aligned(codes, 8) || !aligned(scales, 4)) return fail(DSA_ERR_MISALIGNED, "codes need 8-byte alignment, scales 4-byte");
  if (at_position) P.limit = P.limit > 0 && P.limit < S_cap ? P.limit : S_cap;
  if (!a->positions && P.limit > 0 && (s = check_range(a->pos0, a->n, P.limit, "the table or the cache")) != DSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes)) != DSA_OK) return s;
  P.codes = codes; P.scales = scales; P.S_cap = S_cap; P.at_position = at_position != 0;
  P.flags = ws_flags(ws);
  return done(dsa::launch_norm_rope(P, static_cast<cudaStream_t>(stream)), "norm launch");
}

dsa_status dsa_latent_append(const dsa_latent_append_args* a, const dsa_latent_cache* cache, void* ws, size_t ws_bytes,
                             void* stream) {
  return append_rows(a, cache, ws, ws_bytes, stream);
}
dsa_status dsa_latent4_append(const dsa_latent_append_args* a, const dsa_latent4_cache* cache, void* ws, size_t ws_bytes,
                              void* stream) {
  return append_rows(a, cache, ws, ws_bytes, stream);
}

dsa_status dsa_latent_read(const dsa_latent_cache* cache, int32_t B, int32_t n, const int32_t* idx, int64_t pos0, void* out,
                           void* ws, size_t ws_bytes, void* stream) {
  dsa::LatentReadLaunch P{};
  P.out = static_cast<uint16_t*>(out);
  return read_rows(cache, B, n, idx, pos0, P, out, out, out, ws, ws_bytes, stream);
}
dsa_status dsa_latent4_read(const dsa_latent4_cache* cache, int32_t B, int32_t n, const int32_t* idx, int64_t pos0, void* out,
                            void* ws, size_t ws_bytes, void* stream) {
  dsa::LatentReadLaunch P{};
  P.out = static_cast<uint16_t*>(out);
  return read_rows(cache, B, n, idx, pos0, P, out, out, out, ws, ws_bytes, stream);
}
dsa_status dsa_latent4_unpack(const dsa_latent4_cache* cache, int32_t B, int32_t n, const int32_t* idx, int64_t pos0,
                              uint8_t* codes, float* scales, void* rope, void* ws, size_t ws_bytes, void* stream) {
  dsa::LatentReadLaunch P{};
  P.out_codes = codes;
  P.out_scales = scales;
  P.out_rope = static_cast<uint16_t*>(rope);
  return read_rows(cache, B, n, idx, pos0, P, codes, rope, scales, ws, ws_bytes, stream);
}

size_t dsa_latent_attn_workspace_size(const dsa_latent_attn_args*, int32_t) { return DSA_WS_MIN; }
size_t dsa_latent_attn_dense_workspace_size(int32_t B, int32_t T, int32_t S, int32_t H) {
  if (B < 1 || T < 1 || S < 1 || H < 1 || H > 128) return DSA_WS_MIN;  // (the call refuses these)
  dsa::LatentAttnLaunch L{};
  L.B = B; L.T = T; L.S = S; L.H = H;
  return dsa::kWsScratch + dsa::latent_dense_scratch(L);
}

dsa_status dsa_latent_attn(const dsa_latent_attn_args* a, const int32_t* idx, int32_t k, void* out, float* lse, void* ws,
                           size_t ws_bytes, void* stream) {
  return attend(a, idx, k, out, lse, ws, ws_bytes, stream);
}
dsa_status dsa_latent4_attn(const dsa_latent4_attn_args* a, const int32_t* idx, int32_t k, void* out, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  return attend(a, idx, k, out, lse, ws, ws_bytes, stream);
}
dsa_status dsa_latent_attn_dense(const dsa_latent_attn_args* a, const int32_t* lens, int32_t causal, void* out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
  return attend_dense(a, lens, causal, out, lse, ws, ws_bytes, stream);
}
dsa_status dsa_latent4_attn_dense(const dsa_latent4_attn_args* a, const int32_t* lens, int32_t causal, void* out, float* lse,
                                  void* ws, size_t ws_bytes, void* stream) {
  return attend_dense(a, lens, causal, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
