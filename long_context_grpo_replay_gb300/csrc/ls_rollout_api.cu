// Host side of the rollout and scoring entry points: the quantised cache,
// cached attention and vocabulary log-probabilities.  Validation, planning
// and dispatch; the kernels are in ls_cache.cu, ls_cached_attn.cu,
// ls_cached_tc.cu, ls_vocab.cu and ls_vocab_tc.cu.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "ls_internal.h"

namespace ls {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool known_dtype(int32_t t) { return t == LS_DTYPE_F32 || t == LS_DTYPE_BF16; }

#define LS_CHECK(expr)               \
  do {                               \
    const ls_status _st = (expr);    \
    if (_st != LS_OK) return _st;    \
  } while (0)

#define LS_CUDA(expr, what)                                                       \
  do {                                                                            \
    const cudaError_t _e = (expr);                                                \
    if (_e != cudaSuccess)                                                        \
      return fail(LS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(_e));           \
  } while (0)

ls_status check_cache(const ls_kv_cache* c) {
  if (!c) return fail(LS_ERR_INVALID_ARGUMENT, "cache is NULL");
  if (c->format != LS_CACHE_F32 && c->format != LS_CACHE_BF16 && c->format != LS_CACHE_E4M3)
    return fail(LS_ERR_INVALID_ARGUMENT, "cache format %d is not an ls_cache_format", c->format);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(LS_ERR_UNSUPPORTED, "head_dim=%d: supported are 64, 128, 256", c->head_dim);
  if (c->hkv < 1 || c->page_size < 1 || c->pool_pages < 1)
    return fail(LS_ERR_INVALID_ARGUMENT, "cache hkv, page_size and pool_pages must be >= 1");
  if (c->hkv > 65535) return fail(LS_ERR_UNSUPPORTED, "hkv %d > 65535", c->hkv);
  if (!c->k || !c->v) return fail(LS_ERR_INVALID_ARGUMENT, "cache pools must be non-NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(LS_ERR_INVALID_ARGUMENT, "cache pools must be 16-byte aligned");
  if (c->format == LS_CACHE_E4M3 && (!c->k_exp || !c->v_exp))
    return fail(LS_ERR_INVALID_ARGUMENT, "an E4M3 cache needs k_exp and v_exp");
  // rows are numbered in 32 bits by the kernels (their byte offsets in 64)
  if (c->pool_pages > INT32_MAX / c->hkv / c->page_size)
    return fail(LS_ERR_UNSUPPORTED, "a pool of more than 2^31-1 rows");
  return LS_OK;
}

ls_status status_word(void* ws, size_t ws_bytes, uint32_t** status) {
  *status = nullptr;
  if (!ws) return LS_OK;
  LS_CHECK(check_ws(ws, ws_bytes, kWsHeader));
  *status = static_cast<uint32_t*>(ws);
  return LS_OK;
}

// ------------------------------------------------------------ cached attention
enum Route { kRouteSimt, kRouteMma, kRouteTc };

struct CachedPlan {
  Route route;
  int32_t ns;
  int64_t span;
  size_t o_bytes, ws_bytes;
};

ls_status check_cached(const ls_cached_attn_desc* d, const ls_kv_cache* c) {
  if (!d) return fail(LS_ERR_INVALID_ARGUMENT, "desc is NULL");
  LS_CHECK(check_cache(c));
  if (!known_dtype(d->q_dtype))
    return fail(LS_ERR_INVALID_ARGUMENT, "q_dtype %d is not an ls_dtype", d->q_dtype);
  if (d->o_dtype != d->q_dtype && d->o_dtype != LS_DTYPE_F32)
    return fail(LS_ERR_INVALID_ARGUMENT, "o_dtype must be q_dtype or LS_DTYPE_F32");
  if (d->hq < 1 || d->hq % c->hkv != 0)
    return fail(LS_ERR_INVALID_ARGUMENT, "hq=%d hkv=%d: need hq %% hkv == 0", d->hq, c->hkv);
  if (d->batch < 0 || d->total_q < 0 || d->max_q < 0 || d->max_kv < 0)
    return fail(LS_ERR_INVALID_ARGUMENT, "batch, total_q, max_q and max_kv must be >= 0");
  if (d->batch > 65535) return fail(LS_ERR_UNSUPPORTED, "batch %d > 65535", d->batch);
  if (d->max_q > d->total_q || (int64_t)d->batch * d->max_q < d->total_q)
    return fail(LS_ERR_INVALID_ARGUMENT, "need max_q <= total_q <= batch * max_q");
  if (d->total_q * d->hq > INT32_MAX || d->total_q > INT32_MAX || (int64_t)d->max_q * d->hq > INT32_MAX / 2)
    return fail(LS_ERR_UNSUPPORTED, "total_q or max_q * hq too large");
  if (d->max_kv > INT32_MAX - 65536) return fail(LS_ERR_UNSUPPORTED, "max_kv too large");
  if (d->q_stride < (int64_t)d->hq * c->head_dim || d->q_stride % 8 != 0)
    return fail(LS_ERR_INVALID_ARGUMENT, "q_stride must be a multiple of 8, at least hq * head_dim");
  if (!(d->softmax_scale > 0.f) || !std::isfinite(d->softmax_scale))
    return fail(LS_ERR_INVALID_ARGUMENT, "softmax_scale must be finite and > 0");
  return LS_OK;
}

// Multiplier and shift of j / d for 0 <= j < 2^31 (d >= 1): with 2^(s-1) < d <=
// 2^s, m = ceil(2^(31+s) / d) is below 2^32 and off by e < d <= 2^s, so j m /
// 2^(31+s) exceeds j / d by j e / (d 2^(31+s)) < 1 / d.  umulhi takes 2^32 of
// the divisor; d = 1 has no such pair, and a multiplier of 0 stands for it.
void page_divisor(uint32_t d, uint32_t* mul, uint32_t* shift) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  if (s == 0) {
    *mul = 0, *shift = 0;
    return;
  }
  *mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  *shift = s - 1;
}

CachedPlan plan_cached(const ls_cached_attn_desc& d, const ls_kv_cache& c) {
  CachedPlan pl{};
  const int gq = d.hq / c.hkv, sms = device_sms();
  const int64_t rows = (int64_t)d.max_q * gq;
  const double key_bytes = 2.0 * c.head_dim * (c.format == LS_CACHE_F32 ? 4 : c.format == LS_CACHE_BF16 ? 2 : 1);
  // A CTA's tile of rows, the keys that parts are counted in, and about how
  // long a CTA takes for them and for its start and end (microseconds).
  int64_t tile, quantum, ctas = sms;
  double per_quantum, fixed;
  if (d.q_dtype != LS_DTYPE_BF16 || c.format == LS_CACHE_F32 || force_simt()) {
    pl.route = kRouteSimt;
    tile = 16, quantum = 32, ctas = 4 * sms;
    per_quantum = 6.0, fixed = 6.0;
  } else if (rows <= cached_mma_rows(c.head_dim, c.format)) {
    pl.route = kRouteMma;
    tile = rows < 8 ? 8 : rows;
    quantum = 128, ctas = 2 * sms;
    per_quantum = quantum * key_bytes / 22e3, fixed = 10.0;
  } else {
    pl.route = kRouteTc;
    const bool pair = cached_tc_pairs(rows, c.head_dim);
    tile = pair ? 256 : 128, quantum = 128, ctas = pair ? sms / 2 : sms;
    per_quantum = (pair ? 1.6 : 2.6) + 0.4 * c.head_dim / 256.0, fixed = pair ? 24.0 : 8.0;
  }
  const int64_t units = (int64_t)d.batch * c.hkv * ((rows + tile - 1) / tile);
  const int64_t quanta = d.max_kv > 0 ? (d.max_kv + quantum - 1) / quantum : 1;
  const size_t out_rows = (size_t)d.total_q * d.hq;
  // Rounds of CTAs against the parts' float32 results, written and read once.
  // Where everything runs at once the longest part counts.  Beyond that,
  // sequences that end at different lengths, taken for half the longest on
  // average, fill rounds unevenly.
  int64_t best = 1;
  double best_cost = 1e300;
  for (int64_t ns = 1; ns <= kCachedMaxParts && ns <= quanta && units > 0; ++ns) {
    const int64_t span = (quanta + ns - 1) / ns;
    if ((quanta + span - 1) / span != ns) continue;
    const double x = (double)(units * ns) / ctas;
    const double rounds = x <= 1.0 ? 1.0 : d.batch > 1 ? 0.5 * x + 0.7 : std::ceil(x);
    const double cost = rounds * (span * per_quantum + fixed) +
                        (ns > 1 ? 3.0 + ns * (double)out_rows * c.head_dim * 8.0 / 6.0e6 : 0.0);
    if (cost < best_cost * 0.99) best_cost = cost, best = ns;
  }
  pl.span = (quanta + best - 1) / best * quantum;
  pl.ns = (int32_t)((quanta * quantum + pl.span - 1) / pl.span);
  pl.o_bytes = pl.ns > 1 ? round_up((size_t)pl.ns * out_rows * c.head_dim * sizeof(float), 256) : 0;
  pl.ws_bytes = kWsHeader + pl.o_bytes +
                (pl.ns > 1 ? round_up((size_t)pl.ns * out_rows * sizeof(float), 256) : 0);
  return pl;
}

// ------------------------------------------------------------ vocabulary
ls_status check_vocab(const ls_vocab_desc* d) {
  if (!d) return fail(LS_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (!known_dtype(d->dtype))
    return fail(LS_ERR_INVALID_ARGUMENT, "dtype %d is not LS_DTYPE_F32 or LS_DTYPE_BF16", d->dtype);
  if (d->hidden < 1 || d->vocab < 1 || d->n_rows < 0)
    return fail(LS_ERR_INVALID_ARGUMENT, "need hidden, vocab >= 1 and n_rows >= 0");
  if (d->n_rows > INT32_MAX / 2 || d->vocab > INT32_MAX / 2 || d->hidden > INT32_MAX / 2)
    return fail(LS_ERR_UNSUPPORTED, "n_rows, vocab and hidden must stay below 2^30");
  if (d->h_stride < d->hidden || d->w_stride < d->hidden)
    return fail(LS_ERR_INVALID_ARGUMENT, "row strides must be at least hidden");
  if (d->piece < 0) return fail(LS_ERR_INVALID_ARGUMENT, "piece < 0");
  if (d->ignore_index >= 0 && d->ignore_index < d->vocab)
    return fail(LS_ERR_INVALID_ARGUMENT, "ignore_index %lld is a token of the vocabulary",
                (long long)d->ignore_index);
  if (!std::isfinite(d->logit_scale))
    return fail(LS_ERR_INVALID_ARGUMENT, "logit_scale must be finite");
  return LS_OK;
}

// The tensor-core route by the desc alone, so that the workspace's size does
// not depend on addresses; a call whose addresses do not suit it takes the
// CUDA-core route in the same workspace.
bool vocab_tc_shape(const ls_vocab_desc& d) {
  return d.dtype == LS_DTYPE_BF16 && d.hidden % 8 == 0 && d.h_stride % 8 == 0 &&
         d.w_stride % 8 == 0 && !force_simt() && device_is_sm100_family();
}

size_t vocab_need(const ls_vocab_desc& d, bool with_grad) {
  size_t need = vocab_simt_scratch(d, with_grad);
  if (vocab_tc_shape(d)) {
    const size_t t = vocab_tc_scratch(d, with_grad);
    need = t > need ? t : need;
  }
  return kWsHeader + need;
}

}  // namespace
}  // namespace ls

using namespace ls;

extern "C" {

ls_status ls_cache_write(const ls_kv_cache* cache, int32_t src_dtype, const void* k, const void* v,
                         int64_t k_stride, int64_t v_stride, const int64_t* slots, int64_t n_tok,
                         void* ws, size_t ws_bytes, void* stream) {
  LS_CHECK(check_cache(cache));
  if (!known_dtype(src_dtype))
    return fail(LS_ERR_INVALID_ARGUMENT, "src_dtype %d is not an ls_dtype", src_dtype);
  if (n_tok < 0) return fail(LS_ERR_INVALID_ARGUMENT, "n_tok < 0");
  if (n_tok == 0) return LS_OK;
  const int64_t row = (int64_t)cache->hkv * cache->head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return fail(LS_ERR_INVALID_ARGUMENT,
                "k_stride and v_stride must be multiples of 8, at least hkv * head_dim");
  if (!k || !v || !slots) return fail(LS_ERR_INVALID_ARGUMENT, "k, v and slots must be non-NULL");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return fail(LS_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned, slots 8-byte");
  if (n_tok > INT32_MAX / cache->hkv) return fail(LS_ERR_UNSUPPORTED, "n_tok * hkv too large");
  uint32_t* status;
  LS_CHECK(status_word(ws, ws_bytes, &status));
  LS_CUDA(launch_cache_write(*cache, src_dtype, k, v, k_stride, v_stride, slots, n_tok, status,
                             static_cast<cudaStream_t>(stream)),
          "cache write launch");
  return LS_OK;
}

ls_status ls_cache_read(const ls_kv_cache* cache, const int64_t* slots, int64_t n_tok,
                        int32_t dst_dtype, void* k, void* v, void* ws, size_t ws_bytes,
                        void* stream) {
  LS_CHECK(check_cache(cache));
  if (!known_dtype(dst_dtype))
    return fail(LS_ERR_INVALID_ARGUMENT, "dst_dtype %d is not an ls_dtype", dst_dtype);
  if (n_tok < 0) return fail(LS_ERR_INVALID_ARGUMENT, "n_tok < 0");
  if (n_tok == 0) return LS_OK;
  if (!k || !v || !slots) return fail(LS_ERR_INVALID_ARGUMENT, "k, v and slots must be non-NULL");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return fail(LS_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned, slots 8-byte");
  if (n_tok > INT32_MAX / cache->hkv) return fail(LS_ERR_UNSUPPORTED, "n_tok * hkv too large");
  uint32_t* status;
  LS_CHECK(status_word(ws, ws_bytes, &status));
  LS_CUDA(launch_cache_read(*cache, slots, n_tok, dst_dtype, k, v, status,
                            static_cast<cudaStream_t>(stream)),
          "cache read launch");
  return LS_OK;
}

ls_status ls_cached_attn_workspace_size(const ls_cached_attn_desc* desc, const ls_kv_cache* cache,
                                        size_t* bytes) {
  LS_CHECK(check_cached(desc, cache));
  if (!bytes) return fail(LS_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = plan_cached(*desc, *cache).ws_bytes;
  return LS_OK;
}

ls_status ls_cached_attn(const ls_cached_attn_desc* desc, const ls_kv_cache* cache, const void* q,
                         const int32_t* q_start, const int64_t* kv_len, const int32_t* page_table,
                         int64_t pages_per_seq, void* o, float* lse, void* ws, size_t ws_bytes,
                         void* stream) {
  LS_CHECK(check_cached(desc, cache));
  if (desc->batch == 0 || desc->total_q == 0) return LS_OK;
  if (!q || !q_start || !kv_len || !o || !lse)
    return fail(LS_ERR_INVALID_ARGUMENT, "q, q_start, kv_len, o and lse must be non-NULL");
  if (pages_per_seq < 0 || (pages_per_seq > 0 && !page_table))
    return fail(LS_ERR_INVALID_ARGUMENT, "pages_per_seq < 0, or page_table is NULL");
  if (pages_per_seq > INT32_MAX || pages_per_seq * cache->page_size > INT32_MAX - 65536)
    return fail(LS_ERR_UNSUPPORTED, "pages_per_seq * page_size too large");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(q_start, 4) ||
      !aligned(kv_len, 8) || !aligned(page_table, 4))
    return fail(LS_ERR_INVALID_ARGUMENT, "q and o must be 16-byte aligned, the others by element");
  const CachedPlan pl = plan_cached(*desc, *cache);
  LS_CHECK(check_ws(ws, ws_bytes, pl.ws_bytes));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CachedParams p{};
  p.c = *cache;
  p.hq = desc->hq;
  p.gq = desc->hq / cache->hkv;
  p.batch = desc->batch;
  p.max_q = desc->max_q;
  p.causal = desc->causal != 0;
  p.q_dtype = desc->q_dtype;
  p.o_dtype = desc->o_dtype;
  p.total_q = desc->total_q;
  p.q_stride = desc->q_stride;
  p.pages_per_seq = pages_per_seq;
  page_divisor(cache->page_size, &p.page_mul, &p.page_shift);
  p.scale = desc->softmax_scale;
  p.scale_log2 = desc->softmax_scale * 1.4426950408889634f;
  p.ns = pl.ns;
  p.span = pl.span;
  p.q = q;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.page_table = page_table;
  p.o = o;
  p.lse = lse;
  p.o_parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  p.lse_parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader + pl.o_bytes);
  p.status = static_cast<uint32_t*>(ws);
  if (pl.route == kRouteSimt)
    LS_CUDA(launch_cached_simt(p, s), "cached attention launch");
  else if (pl.route == kRouteMma)
    LS_CUDA(launch_cached_mma(p, s), "cached attention launch");
  else
    LS_CUDA(launch_cached_tc(p, s), "cached attention launch");
  if (pl.ns > 1)
    LS_CUDA(launch_cached_join(p, s), "part join launch");
  return LS_OK;
}

ls_status ls_vocab_logprob_workspace_size(const ls_vocab_desc* desc, int32_t with_grad,
                                          size_t* bytes) {
  LS_CHECK(check_vocab(desc));
  if (!bytes) return fail(LS_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = vocab_need(*desc, with_grad != 0);
  return LS_OK;
}

ls_status ls_vocab_logprob_fwd(const ls_vocab_desc* desc, const void* h, const void* w,
                               const int64_t* targets, float* logp, float* lse, void* ws,
                               size_t ws_bytes, void* stream) {
  LS_CHECK(check_vocab(desc));
  if (desc->n_rows == 0) return LS_OK;
  if (!h || !w || !targets || !logp || !lse)
    return fail(LS_ERR_INVALID_ARGUMENT, "h, w, targets, logp and lse must be non-NULL");
  const size_t esz = desc->dtype == LS_DTYPE_F32 ? 4 : 2;
  if (!aligned(h, esz) || !aligned(w, esz) || !aligned(targets, 8) || !aligned(logp, 4) ||
      !aligned(lse, 4))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  LS_CHECK(check_ws(ws, ws_bytes, vocab_need(*desc, false)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tc = vocab_tc_shape(*desc) && aligned(h, 16) && aligned(w, 16);
  for (int64_t r0 = 0; r0 < desc->n_rows; r0 += kVocabRows) {
    VocabParams p{};
    p.d = *desc;
    p.d.n_rows = desc->n_rows - r0 < kVocabRows ? desc->n_rows - r0 : kVocabRows;
    p.h = static_cast<const char*>(h) + r0 * desc->h_stride * (int64_t)esz;
    p.w = w;
    p.targets = targets + r0;
    p.logp = logp + r0;
    p.lse = lse + r0;
    p.scratch = static_cast<char*>(ws) + kWsHeader;
    p.status = static_cast<uint32_t*>(ws);
    if (tc)
      LS_CUDA(launch_vocab_tc_fwd(p, s), "vocabulary forward launch");
    else
      LS_CUDA(launch_vocab_simt_fwd(p, s), "vocabulary forward launch");
  }
  return LS_OK;
}

ls_status ls_vocab_logprob_bwd(const ls_vocab_desc* desc, const void* h, const void* w,
                               const int64_t* targets, const float* lse, const float* d_logp,
                               void* dh, void* dw, void* ws, size_t ws_bytes, void* stream) {
  LS_CHECK(check_vocab(desc));
  if (!dh && !dw) return LS_OK;
  const size_t esz = desc->dtype == LS_DTYPE_F32 ? 4 : 2;
  if (!aligned(dh, 16) || !aligned(dw, 16))
    return fail(LS_ERR_INVALID_ARGUMENT, "dh and dw must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (desc->n_rows == 0) {  // no row: nothing reaches the weight
    if (dw) LS_CUDA(cudaMemsetAsync(dw, 0, (size_t)desc->vocab * desc->hidden * esz, s), "dw clear");
    return LS_OK;
  }
  if (!h || !w || !targets || !lse || !d_logp)
    return fail(LS_ERR_INVALID_ARGUMENT, "h, w, targets, lse and d_logp must be non-NULL");
  if (!aligned(h, esz) || !aligned(w, esz) || !aligned(targets, 8) || !aligned(lse, 4) ||
      !aligned(d_logp, 4))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  LS_CHECK(check_ws(ws, ws_bytes, vocab_need(*desc, true)));
  VocabParams p{};
  p.d = *desc;
  p.h = h;
  p.w = w;
  p.targets = targets;
  p.lse_in = lse;
  p.d_logp = d_logp;
  p.dh = dh;
  p.dw = dw;
  p.scratch = static_cast<char*>(ws) + kWsHeader;
  p.status = static_cast<uint32_t*>(ws);
  if (vocab_tc_shape(*desc) && aligned(h, 16) && aligned(w, 16))
    LS_CUDA(launch_vocab_tc_bwd(p, s), "vocabulary backward launch");
  else
    LS_CUDA(launch_vocab_simt_bwd(p, s), "vocabulary backward launch");
  return LS_OK;
}

}  // extern "C"
