// Host side of the entry points of a rollout with drafted tokens: pages of a
// cache, verification of drafts and the recurrent step of the gated-DeltaNet
// state.  Validation and dispatch; the kernels are in ls_pages.cu, ls_verify.cu
// and ls_gdn_decode.cu.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "ls_internal.h"

namespace ls {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// A run of bytes (none of them, or NULL: nothing).
struct Run {
  const void* at;
  uint64_t bytes;
};
bool overlap(const Run& a, const Run& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// What a block writes, none of what others still read.
bool apart(std::initializer_list<Run> written, std::initializer_list<Run> read) {
  for (const Run& a : written)
    for (const Run& b : read)
      if (overlap(a, b)) return false;
  return true;
}
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

ls_status status_word(void* ws, size_t ws_bytes, uint32_t** status) {
  *status = nullptr;
  if (!ws) return LS_OK;
  LS_CHECK(check_ws(ws, ws_bytes, kWsHeader));
  *status = static_cast<uint32_t*>(ws);
  return LS_OK;
}

// The tokens of a step: batch, total_q and max_q of a desc.
ls_status check_tokens(int64_t batch, int64_t total_q, int64_t max_q) {
  if (batch < 0 || total_q < 0 || max_q < 0)
    return fail(LS_ERR_INVALID_ARGUMENT, "batch, total_q and max_q must be >= 0");
  if (batch > 65535) return fail(LS_ERR_UNSUPPORTED, "batch %lld > 65535", (long long)batch);
  if (total_q > INT32_MAX) return fail(LS_ERR_UNSUPPORTED, "total_q %lld > 2^31-1", (long long)total_q);
  if (max_q > total_q || batch * max_q < total_q)
    return fail(LS_ERR_INVALID_ARGUMENT, "need max_q <= total_q <= batch * max_q");
  return LS_OK;
}

ls_status check_gdn_decode(const ls_gdn_decode_desc* d) {
  if (!d) return fail(LS_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (!known_dtype(d->dtype))
    return fail(LS_ERR_INVALID_ARGUMENT, "dtype %d is not LS_DTYPE_F32 or LS_DTYPE_BF16", d->dtype);
  if (d->heads < 1 || d->key_heads < 1 || d->heads % d->key_heads != 0)
    return fail(LS_ERR_INVALID_ARGUMENT, "heads=%d key_heads=%d: need heads %% key_heads == 0", d->heads, d->key_heads);
  if (d->heads > 65535) return fail(LS_ERR_UNSUPPORTED, "heads %d > 65535", d->heads);
  if (d->dk != 128 || d->dv != 128)
    return fail(LS_ERR_UNSUPPORTED, "dk=%d dv=%d: supported is 128", d->dk, d->dv);
  LS_CHECK(check_tokens(d->batch, d->total_q, d->max_q));
  if ((int64_t)d->batch * d->heads > INT32_MAX / 2) return fail(LS_ERR_UNSUPPORTED, "batch * heads too large");
  if (d->n_states < 1 || d->n_states > INT32_MAX)
    return fail(LS_ERR_INVALID_ARGUMENT, "n_states must be 1 .. 2^31-1");
  const int64_t key = (int64_t)d->key_heads * d->dk, val = (int64_t)d->heads * d->dv;
  if (d->q_stride < key || d->k_stride < key || d->v_stride < val || d->q_stride % 8 || d->k_stride % 8 ||
      d->v_stride % 8)
    return fail(LS_ERR_INVALID_ARGUMENT, "q_stride, k_stride and v_stride must be multiples of 8, at least a token's heads");
  return LS_OK;
}

ls_status check_book(const ls_page_book* b) {
  if (!b) return fail(LS_ERR_INVALID_ARGUMENT, "book is NULL");
  if (b->page_size < 1 || b->n_seqs < 1 || b->pages_per_seq < 1 || b->pool_pages < 1)
    return fail(LS_ERR_INVALID_ARGUMENT, "page_size, n_seqs, pages_per_seq and pool_pages must be >= 1");
  if ((int64_t)b->pages_per_seq * b->page_size > INT32_MAX - 65536)
    return fail(LS_ERR_UNSUPPORTED, "pages_per_seq * page_size too large");
  if (b->pool_pages > (1 << 29) || b->n_seqs > (1 << 26))
    return fail(LS_ERR_UNSUPPORTED, "pool_pages must be at most 2^29, n_seqs 2^26");
  if (!b->refs || !b->page_table || !b->kv_len)
    return fail(LS_ERR_INVALID_ARGUMENT, "refs, page_table and kv_len must be non-NULL");
  if (!aligned(b->refs, 4) || !aligned(b->page_table, 4) || !aligned(b->kv_len, 8))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  return LS_OK;
}

ls_status pages_params(const ls_page_book* b, int64_t n, void* ws, size_t ws_bytes, PagesParams* p) {
  if (n < 0 || n > b->n_seqs)
    return fail(LS_ERR_INVALID_ARGUMENT, "n=%lld: a call names each of the %d sequences at most once", (long long)n, b->n_seqs);
  LS_CHECK(check_ws(ws, ws_bytes, kWsHeader + pages_scratch(*b)));
  p->b = *b;
  p->n = (int32_t)n;
  page_divisor(b->page_size, &p->page_mul, &p->page_shift);
  p->status = static_cast<uint32_t*>(ws);
  int32_t* w = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kWsHeader);
  p->list = w, w += b->pool_pages;
  p->high = w, w += b->pool_pages;
  p->rank = w, w += b->pool_pages;
  p->owner = w, w += 8 * (int64_t)b->n_seqs;
  p->lists = w;
  return LS_OK;
}

Run refs_of(const ls_page_book& b) { return {b.refs, 4 * (uint64_t)b.pool_pages}; }
Run table_of(const ls_page_book& b) { return {b.page_table, 4 * (uint64_t)b.n_seqs * b.pages_per_seq}; }
Run lengths_of(const ls_page_book& b) { return {b.kv_len, 8 * (uint64_t)b.n_seqs}; }
// Lists that a kernel of pages reads in every block before, and beside, the first writes (of lengths as int64,
// kv_len itself may be one: it is written when all have been read).
ls_status check_lists(const ls_page_book& b, const Run& seqs, const Run& more, const Run& lengths, const Run& slots, const Run& copies) {
  const Run len = lengths.at == b.kv_len ? Run{nullptr, 0} : lengths;
  if (!apart({slots, copies, refs_of(b), table_of(b), lengths_of(b)}, {seqs, more, len}) ||
      !apart({refs_of(b), table_of(b), slots, copies}, {lengths}) || !apart({slots, copies}, {refs_of(b), table_of(b), lengths_of(b)}) ||
      overlap(slots, copies))
    return fail(LS_ERR_INVALID_ARGUMENT, "slots, copies and the book must not overlap each other or the lists");
  return LS_OK;
}

ls_status check_verify(const ls_verify_desc* d) {
  if (!d) return fail(LS_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (!known_dtype(d->dtype))
    return fail(LS_ERR_INVALID_ARGUMENT, "dtype %d is not LS_DTYPE_F32 or LS_DTYPE_BF16", d->dtype);
  if (d->vocab < 1) return fail(LS_ERR_INVALID_ARGUMENT, "vocab < 1");
  // a random number in float32 has 2^24 values, and the sums that accept drafts lose a bit with each doubling
  if (d->vocab > (1 << 24)) return fail(LS_ERR_UNSUPPORTED, "vocab %d > 2^24", d->vocab);
  LS_CHECK(check_tokens(d->batch, d->total_q, d->max_q));
  if (d->logits_stride < d->vocab) return fail(LS_ERR_INVALID_ARGUMENT, "logits_stride must be at least vocab");
  if (!(d->logit_scale > 0.f) || !std::isfinite(d->logit_scale))
    return fail(LS_ERR_INVALID_ARGUMENT, "logit_scale must be finite and > 0");
  // beyond these a masked token's product is not far enough below the others', or overflows
  if (d->logit_scale < 0x1p-100f || d->logit_scale > 0x1p100f)
    return fail(LS_ERR_UNSUPPORTED, "logit_scale %g is not within 2^-100 .. 2^100", (double)d->logit_scale);
  if (d->total_q * verify_chunks(*d) > INT32_MAX) return fail(LS_ERR_UNSUPPORTED, "total_q * vocab too large");
  return LS_OK;
}

size_t verify_need(const ls_verify_desc& d) {
  return kWsHeader + verify_scratch(d);
}

}  // namespace
}  // namespace ls

using namespace ls;

extern "C" {

ls_status ls_pages_workspace_size(const ls_page_book* book, size_t* bytes) {
  LS_CHECK(check_book(book));
  if (!bytes) return fail(LS_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = kWsHeader + pages_scratch(*book);
  return LS_OK;
}

ls_status ls_pages_advance(const ls_page_book* book, int32_t n, const int32_t* seqs,
                           const int64_t* keep, const int32_t* q_start, int64_t total_q,
                           int64_t* slots, int32_t* copies, void* ws, size_t ws_bytes,
                           void* stream) {
  LS_CHECK(check_book(book));
  if (total_q < 0) return fail(LS_ERR_INVALID_ARGUMENT, "total_q < 0");
  if (total_q > (1 << 29)) return fail(LS_ERR_UNSUPPORTED, "total_q > 2^29");  // so that counts of pages fit 30 bits
  if (total_q > 0 && (!q_start || !slots || n == 0))
    return fail(LS_ERR_INVALID_ARGUMENT, "new tokens need q_start, slots and sequences");
  if (q_start && !copies && n > 0) return fail(LS_ERR_INVALID_ARGUMENT, "growing sequences need copies");
  if (!aligned(seqs, 4) || !aligned(keep, 8) || !aligned(q_start, 4) || !aligned(slots, 8) || !aligned(copies, 4))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  PagesParams p{};
  LS_CHECK(pages_params(book, n, ws, ws_bytes, &p));
  if (n == 0) return LS_OK;
  LS_CHECK(check_lists(*book, {seqs, 4 * (uint64_t)n}, {q_start, 4 * ((uint64_t)n + 1)}, {keep, 8 * (uint64_t)n},
                       {slots, 8 * (uint64_t)total_q}, {copies, 12 * (uint64_t)n}));
  p.seqs = seqs;
  p.keep = keep;
  p.q_start = q_start;
  p.total_q = total_q;
  p.slots = slots;
  p.copies = copies;
  LS_CUDA(launch_pages_advance(p, static_cast<cudaStream_t>(stream)), "pages launch");
  return LS_OK;
}

ls_status ls_pages_release(const ls_page_book* book, int32_t n, const int32_t* seqs, void* ws,
                           size_t ws_bytes, void* stream) {
  LS_CHECK(check_book(book));
  if (!aligned(seqs, 4)) return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  PagesParams p{};
  LS_CHECK(pages_params(book, seqs ? n : book->n_seqs, ws, ws_bytes, &p));
  if (p.n == 0) return LS_OK;
  LS_CHECK(check_lists(*book, {seqs, 4 * (uint64_t)p.n}, {}, {}, {}, {}));
  p.seqs = seqs;
  p.drop_all = true;
  LS_CUDA(launch_pages_advance(p, static_cast<cudaStream_t>(stream)), "pages launch");
  return LS_OK;
}

ls_status ls_pages_fork(const ls_page_book* book, int32_t n, const int32_t* src, const int32_t* dst,
                        const int64_t* lens, void* ws, size_t ws_bytes, void* stream) {
  LS_CHECK(check_book(book));
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(lens, 8))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  PagesParams p{};
  LS_CHECK(pages_params(book, n, ws, ws_bytes, &p));
  if (n == 0) return LS_OK;
  if (!src || !dst) return fail(LS_ERR_INVALID_ARGUMENT, "src and dst must be non-NULL");
  LS_CHECK(check_lists(*book, {src, 4 * (uint64_t)n}, {dst, 4 * (uint64_t)n}, {lens, 8 * (uint64_t)n}, {}, {}));
  p.src = src;
  p.seqs = dst;
  p.keep = lens;
  LS_CUDA(launch_pages_fork(p, static_cast<cudaStream_t>(stream)), "pages launch");
  return LS_OK;
}

ls_status ls_pages_compact(const ls_page_book* book, int32_t* table_out, int32_t* refs_out,
                           int32_t* copies, void* ws, size_t ws_bytes, void* stream) {
  LS_CHECK(check_book(book));
  if (!table_out || !refs_out || (book->pool_pages > 1 && !copies))
    return fail(LS_ERR_INVALID_ARGUMENT, "table_out, refs_out and copies must be non-NULL");
  if (!aligned(table_out, 4) || !aligned(refs_out, 4) || !aligned(copies, 4))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  PagesParams p{};
  LS_CHECK(pages_params(book, 0, ws, ws_bytes, &p));
  const Run refs = refs_of(*book), table = table_of(*book), out_refs{refs_out, refs.bytes}, out_table{table_out, table.bytes},
            moves{copies, 12 * (uint64_t)(book->pool_pages / 2)};
  if (!apart({out_refs, moves}, {table, lengths_of(*book), out_table}) || !apart({out_table, moves}, {refs, lengths_of(*book), out_refs}) ||
      (refs_out != book->refs && overlap(out_refs, refs)) || (table_out != book->page_table && overlap(out_table, table)))
    return fail(LS_ERR_INVALID_ARGUMENT, "table_out, refs_out and copies must not overlap each other or the book (but the first two may be its own)");
  p.copies = copies;
  p.table_out = table_out;
  p.refs_out = refs_out;
  LS_CUDA(launch_pages_compact(p, static_cast<cudaStream_t>(stream)), "pages launch");
  return LS_OK;
}

ls_status ls_cache_copy_pages(const ls_kv_cache* cache, const int32_t* copies, int64_t n, void* ws,
                              size_t ws_bytes, void* stream) {
  LS_CHECK(check_cache(cache));
  if (n < 0) return fail(LS_ERR_INVALID_ARGUMENT, "n < 0");
  if (n > INT32_MAX) return fail(LS_ERR_UNSUPPORTED, "n > 2^31-1");
  if (n == 0) return LS_OK;
  if (!copies || !aligned(copies, 4)) return fail(LS_ERR_INVALID_ARGUMENT, "copies must be non-NULL and 4-byte aligned");
  uint32_t* status;
  LS_CHECK(status_word(ws, ws_bytes, &status));
  LS_CUDA(launch_page_copy(*cache, copies, n, status, static_cast<cudaStream_t>(stream)), "page copy launch");
  return LS_OK;
}

ls_status ls_draft_verify_workspace_size(const ls_verify_desc* desc, size_t* bytes) {
  LS_CHECK(check_verify(desc));
  if (!bytes) return fail(LS_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = verify_need(*desc);
  return LS_OK;
}

ls_status ls_draft_verify(const ls_verify_desc* desc, const void* logits, const float* draft_probs,
                          const int64_t* tokens, const int32_t* q_start, const float* u,
                          const float* u_next, const int64_t* kv_len, int32_t* n_emitted,
                          int64_t* emitted, float* logp, int64_t* keep, void* ws, size_t ws_bytes,
                          void* stream) {
  LS_CHECK(check_verify(desc));
  if (desc->batch == 0) return LS_OK;
  if (!q_start || !n_emitted || !u_next) return fail(LS_ERR_INVALID_ARGUMENT, "q_start, u_next and n_emitted must be non-NULL");
  if (desc->total_q > 0 && (!logits || !tokens || !u || !emitted))
    return fail(LS_ERR_INVALID_ARGUMENT, "logits, tokens, u and emitted must be non-NULL");
  if (keep && !kv_len) return fail(LS_ERR_INVALID_ARGUMENT, "keep needs kv_len");
  if (draft_probs && desc->draft_stride < desc->vocab)
    return fail(LS_ERR_INVALID_ARGUMENT, "draft_stride must be at least vocab");
  if (!aligned(logits, desc->dtype == LS_DTYPE_F32 ? 4 : 2) || !aligned(draft_probs, 4) || !aligned(tokens, 8) ||
      !aligned(q_start, 4) || !aligned(u, 4) || !aligned(u_next, 4) || !aligned(kv_len, 8) || !aligned(n_emitted, 4) ||
      !aligned(emitted, 8) || !aligned(logp, 4) || !aligned(keep, 8))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  // one block of a sequence writes while others, and those of other sequences, read on
  const uint64_t n = desc->total_q, b = desc->batch;
  if (!apart({{n_emitted, 4 * b}, {emitted, 8 * n}, {logp, 4 * n}, {keep, 8 * b}},
             {{tokens, 8 * n}, {q_start, 4 * (b + 1)}, {u, 4 * n}, {u_next, 4 * b}}) ||
      (keep && !apart({{n_emitted, 4 * b}, {emitted, 8 * n}, {logp, 4 * n}, {keep == kv_len ? nullptr : keep, 8 * b}}, {{kv_len, 8 * b}})))
    return fail(LS_ERR_INVALID_ARGUMENT, "the results must not overlap the inputs (but keep may be kv_len)");
  LS_CHECK(check_ws(ws, ws_bytes, verify_need(*desc)));
  VerifyParams p{};
  p.d = *desc;
  const double c = (double)desc->logit_scale * 1.4426950408889634074;
  p.c = (float)c;
  p.c_low = (float)(c - (double)p.c);
  p.logits = logits;
  p.probs = draft_probs;
  p.tokens = tokens;
  p.q_start = q_start;
  p.u = u;
  p.u_next = u_next;
  p.kv_len = kv_len;
  p.n_emitted = n_emitted;
  p.emitted = emitted;
  p.logp = logp;
  p.keep = keep;
  p.chunks = verify_chunks(*desc);
  p.status = static_cast<uint32_t*>(ws);
  p.parts = reinterpret_cast<float2*>(static_cast<char*>(ws) + kWsHeader);
  LS_CUDA(launch_draft_verify(p, static_cast<cudaStream_t>(stream)), "draft verification launch");
  return LS_OK;
}

ls_status ls_gdn_decode(const ls_gdn_decode_desc* desc, float* states, const void* q, const void* k,
                        const void* v, const float* g, const float* beta, const int32_t* q_start,
                        const int32_t* n_use, const int32_t* state_in, const int32_t* state_out,
                        void* o, void* ws, size_t ws_bytes, void* stream) {
  LS_CHECK(check_gdn_decode(desc));
  if (desc->batch == 0 || (!o && !state_out)) return LS_OK;
  if (!states || !q_start || !state_in)
    return fail(LS_ERR_INVALID_ARGUMENT, "states, q_start and state_in must be non-NULL");
  if (desc->total_q > 0 && (!q || !k || !v || !g || !beta))
    return fail(LS_ERR_INVALID_ARGUMENT, "q, k, v, g and beta must be non-NULL");
  if (!aligned(states, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return fail(LS_ERR_INVALID_ARGUMENT, "states, q, k, v and o must be 16-byte aligned");
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(q_start, 4) || !aligned(n_use, 4) || !aligned(state_in, 4) ||
      !aligned(state_out, 4))
    return fail(LS_ERR_INVALID_ARGUMENT, "buffers must be aligned to their elements");
  // a block writes its rows of o and of the states while others read on
  const uint64_t size = desc->dtype == LS_DTYPE_F32 ? 4 : 2, n = desc->total_q, b = desc->batch, h = desc->heads,
                 key = (uint64_t)desc->key_heads * desc->dk, val = h * desc->dv, last = n > 0 ? n - 1 : 0;
  const Run results[] = {{o, size * n * val}, {states, 4 * desc->n_states * val * desc->dk}};
  if (overlap(results[0], results[1]) ||
      !apart({results[0], results[1]}, {{q, n ? size * (last * desc->q_stride + key) : 0},
                                        {k, n ? size * (last * desc->k_stride + key) : 0},
                                        {v, n ? size * (last * desc->v_stride + val) : 0},
                                        {g, 4 * n * h},
                                        {beta, 4 * n * h},
                                        {q_start, 4 * (b + 1)},
                                        {n_use, 4 * b},
                                        {state_in, 4 * b},
                                        {state_out, 4 * b}}))
    return fail(LS_ERR_INVALID_ARGUMENT, "o and states must not overlap each other or what the call reads");
  GdnDecodeParams p{};
  LS_CHECK(status_word(ws, ws_bytes, &p.status));
  p.d = *desc;
  p.states = states;
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.q_start = q_start;
  p.n_use = n_use;
  p.state_in = state_in;
  p.state_out = state_out;
  p.o = o;
  LS_CUDA(launch_gdn_decode(p, static_cast<cudaStream_t>(stream)), "recurrent step launch");
  return LS_OK;
}

}  // extern "C"
