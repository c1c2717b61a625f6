/*
 * ls.h -- C ABI of the response-replay attention library (libls).
 *
 * The operator: exact response-replay attention for GRPO post-training with a
 * shared, detached long prompt.  The prompt is run once without gradients and
 * its full-attention K/V are kept as compact pages (the capture step of the
 * LongStraw DeepRead summary, section Method).  Each group member's short
 * response is then replayed on its own: its queries attend over every prompt
 * key through the page table and causally over the response's own keys,
 * partial results are recombined exactly by log-sum-exp (the Qwen path's
 * global merge in the same section; the LongStraw abstract on exact attention
 * composition), and the backward treats the prompt K/V as constants (the
 * stored prompt state is stop-gradient, DeepRead summary, Method, last
 * paragraph; the review's mind map, node on equations 1-3: the
 * d(loss)/d(z_P) d(z_P)/d(theta) term is omitted).
 *
 * Conventions shared by every call
 * --------------------------------
 *  Shapes: Hq query heads, Hkv KV heads (Hq % Hkv == 0), head dim d, page
 *  size S_p; query head h reads KV head h / (Hq/Hkv).  R = response length,
 *  P = prompt length.  Response row i sees all P prompt keys and response keys
 *  j <= i.  The softmax scale is a parameter (normally 1/sqrt(d)).
 *  Layouts (all row-major, contiguous, device memory unless stated):
 *    prompt pools   k_pool, v_pool : [pool_pages][Hkv][S_p][d]   element dtype
 *    page table                    : int32 [num_pages], logical page -> slot
 *    q, d_o, o, dq                 : [R][Hq][d]                  element dtype
 *    k_resp, v_resp, dk, dv        : [R][Hkv][d]                 element dtype
 *    lse, delta                    : float32 [R][Hq]; lse is the natural log
 *                                    of the softmax denominator, scale included
 *  Element dtype is uniform per call (LS_DTYPE_F32 or LS_DTYPE_BF16);
 *  accumulation is always float32.
 *
 *  Ownership: the caller allocates every buffer and keeps each one alive
 *  until the work that reads it has finished on its stream; the structs
 *  (ls_prompt_kv, ls_member) only hold pointers.  The library never allocates
 *  or frees device memory.  It keeps a small host-side cache (tensor-map
 *  descriptors) and per-process trace counters, nothing else.  The prompt
 *  pools are read-only for every replay call.
 *
 *  Workspace: one caller-owned device buffer of ls_replay_workspace_size()
 *  bytes, sized for the longest response, reused by every member (the
 *  workspace does not grow with the group size).  Its first 256 bytes hold a
 *  device status word that kernels set on device-side errors.
 *
 *  Errors: every call validates its arguments on the host before any launch
 *  and returns a status; nothing aborts.  Device-side problems set bits in
 *  the workspace status word: a page-table entry outside the pool (that page
 *  is then treated as holding no keys: nothing is read from it and it adds
 *  nothing to the softmax), or a bounded wait that ran out (the affected work
 *  is skipped).  The call itself has already returned LS_OK by then, so read
 *  them with ls_read_device_status().
 *  ls_last_error() gives a one-line reason for the last failing call on the
 *  calling thread.
 *
 *  Streams: every compute call is asynchronous on the given stream
 *  (a cudaStream_t passed as void*; NULL = legacy default stream).  Calls are
 *  thread-safe when they use distinct workspaces.
 */
#ifndef LS_H_
#define LS_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LS_API __attribute__((visibility("default")))
#else
#define LS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LS_OK = 0,
  LS_ERR_INVALID_ARGUMENT = 1,   /* null pointer, bad size, misaligned buffer */
  LS_ERR_UNSUPPORTED = 2,        /* valid but unsupported shape or dtype */
  LS_ERR_WORKSPACE_TOO_SMALL = 3,
  LS_ERR_CUDA = 4,               /* a CUDA runtime/driver call failed */
  LS_ERR_DEVICE_BOUNDS = 5,      /* device saw a page id, slot, length or target out of range */
  LS_ERR_DEVICE_TIMEOUT = 6,     /* a device-side bounded wait ran out */
  LS_ERR_OUT_OF_PAGES = 7        /* sequences could not grow: no free page, or their table's row ended */
} ls_status;

typedef enum { LS_DTYPE_F32 = 0, LS_DTYPE_BF16 = 1 } ls_dtype;

/* Shape and numerics of one attention layer.
 * dtype: ls_dtype of every element buffer.  head_dim in {64, 128, 256};
 * page_size >= 1.  softmax_scale > 0 and finite. */
typedef struct {
  int32_t dtype;
  int32_t hq;
  int32_t hkv;
  int32_t head_dim;
  int32_t page_size;
  float softmax_scale;
} ls_attn_desc;

/* The captured prompt of one layer: pools plus page table (device pointers).
 * Logical prompt position t lives in slot page_table[t / page_size] at row
 * t % page_size.  Requires num_pages * page_size >= prompt_len; rows of the
 * last page beyond prompt_len are never read as keys (they may hold anything,
 * NaN included). */
typedef struct {
  const void* k_pool;
  const void* v_pool;
  int64_t pool_pages;
  const int32_t* page_table;
  int64_t num_pages;
  int64_t prompt_len;
} ls_prompt_kv;

/* One group member for ls_replay_group.  Inputs q, k, v, d_o; outputs o, lse,
 * delta (rowsum(dO*O), written as a by-product), dq, dk, dv. */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  const void* d_o;
  int32_t resp_len;
  int32_t reserved;
  void* o;
  float* lse;
  float* delta;
  void* dq;
  void* dk;
  void* dv;
} ls_member;

/* A1. Capture-side page write (DeepRead summary, Method, the capture step;
 * review section 二.2: the full-attention layers keep their K/V in pages).
 * Scatters token t of k, v ([n_tok][Hkv][d]) to
 *   pool[page_table[(start_pos+t)/S_p]][kv][(start_pos+t)%S_p][:].
 * page_table holds num_pages entries; requires start_pos + n_tok <=
 * num_pages * S_p.  Entries outside [0, pool_pages) are skipped on the device
 * and, if ws is non-NULL, reported through its status word.  Bit-exact copy.
 * ws may be NULL (then ws_bytes is ignored). */
LS_API ls_status ls_kv_page_write(const ls_attn_desc* desc, void* k_pool, void* v_pool,
                           int64_t pool_pages, const int32_t* page_table,
                           int64_t num_pages, int64_t start_pos, int64_t n_tok,
                           const void* k, const void* v, void* ws, size_t ws_bytes,
                           void* stream);

/* Workspace bytes needed by ls_replay_fwd / ls_replay_bwd / ls_replay_group
 * for responses of up to max_resp_len tokens against this prompt on the
 * current device.  Host-only; does not touch the device. */
LS_API ls_status ls_replay_workspace_size(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                                   int32_t max_resp_len, size_t* bytes);

/* A2+A3+A4. Replay forward: O [R][Hq][d] (element dtype) and LSE [R][Hq]
 * (float32, natural log, scale included) of softmax attention over all prompt
 * keys plus the causal response keys.  The prompt part runs split over page
 * ranges into float32 partials held in ws, the response part adds one more
 * partial, and an exact LSE merge writes o and lse (DeepRead summary,
 * Method, Qwen path).  resp_len == 0 is a no-op. */
LS_API ls_status ls_replay_fwd(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                        const void* q, const void* k_resp, const void* v_resp,
                        int32_t resp_len, void* o, float* lse, void* ws, size_t ws_bytes,
                        void* stream);

/* A4. Exact log-sum-exp merge of partial attention results (the global
 * LSE and output merge of the DeepRead summary, Method):
 *   L[n] = log sum_s exp(Lp[s][n]);  O[n] = sum_s exp(Lp[s][n] - L[n]) Op[s][n].
 * o_parts float32 [n_parts][n_rows][head_dim], lse_parts float32
 * [n_parts][n_rows], natural log; a part with Lp = -inf contributes nothing;
 * a row whose parts are all -inf gets O = 0, L = -inf.  o is written in
 * out_dtype, lse as float32 (lse may be NULL).  head_dim % 4 == 0. */
LS_API ls_status ls_lse_merge(int32_t n_parts, int64_t n_rows, int32_t head_dim,
                       const float* o_parts, const float* lse_parts, int32_t out_dtype,
                       void* o, float* lse, void* stream);

/* A5. Backward preprocess: delta[r][h] = sum_c dO[r][h][c] * O[r][h][c]
 * (float32 accumulation of the element-dtype inputs). */
LS_API ls_status ls_replay_bwd_preprocess(const ls_attn_desc* desc, const void* o, const void* d_o,
                                   int32_t resp_len, float* delta, void* stream);

/* A6+A7. Replay backward with the prompt state detached (DeepRead summary,
 * Method: stored prompt state is stop-gradient; review section 二, last
 * paragraph: on the Qwen path only the query gradient crosses ranks).
 * Recomputes P = exp(s - LSE) from the stored lse (no score matrix is kept),
 * dS = P * (dO.v - delta), and returns
 *   dq      [R][Hq][d]  = scale * sum over prompt and visible response keys of dS k
 *   dk_resp [R][Hkv][d] = scale * sum over the group's heads, rows i >= j of dS q
 *   dv_resp [R][Hkv][d] = sum over the group's heads, rows i >= j of P dO
 * No gradient is produced for prompt K/V.  lse and delta come from
 * ls_replay_fwd and ls_replay_bwd_preprocess. */
LS_API ls_status ls_replay_bwd(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                        const void* q, const void* k_resp, const void* v_resp,
                        const void* d_o, const float* lse, const float* delta,
                        int32_t resp_len, void* dq, void* dk_resp, void* dv_resp,
                        void* ws, size_t ws_bytes, void* stream);

/* A8. Serial replay of a group's response suffixes (DeepRead summary, Method;
 * abstract: one response at a time is rebuilt under autograd and
 * backpropagated, back to the prompt boundary).  For each member in order:
 * forward, preprocess, backward, all on one stream and into the one workspace,
 * so only one member's intermediates are live and the workspace does not grow
 * with n_members.  Each member's results equal a standalone replay of it. */
LS_API ls_status ls_replay_group(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                          int32_t n_members, const ls_member* members, void* ws,
                          size_t ws_bytes, void* stream);

/* Context parallelism, one rank's share (DeepRead summary, Method, Qwen path:
 * the prompt pages are sharded over ranks and the partial results are merged
 * globally by LSE; review section 二: the query gradient is what crosses
 * ranks).  `prompt` holds the pages this rank owns, in any order: attention
 * over a set of keys does not depend on their order.  Every rank holds the
 * whole response (q, k_resp, v_resp, d_o).  Exactly one rank passes
 * with_response != 0 and adds the causal response keys.
 *
 * ls_replay_fwd_part writes the rank's exact partial in float32: o_part
 * [R][Hq][d], normalised over the rank's keys, and lse_part [R][Hq].  A rank
 * with no visible key gets O = 0 and LSE = -inf.  The global O, LSE is
 * ls_lse_merge over all ranks' partials (an all-gather, then the merge).
 *
 * ls_replay_bwd_part writes dq_part float32 [R][Hq][d], the rank's share of
 * dQ with the scale applied.  The global dQ is the sum over ranks (an
 * all-reduce).  lse and delta must be the global ones (from the merged
 * forward).  dk_resp and dv_resp are written only with_response, and may be
 * NULL otherwise.  Workspace: ls_replay_workspace_size for the rank's prompt.
 * The interface is this library's; the pages describe the split, not a call. */
LS_API ls_status ls_replay_fwd_part(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                                    const void* q, const void* k_resp, const void* v_resp,
                                    int32_t resp_len, int32_t with_response, float* o_part,
                                    float* lse_part, void* ws, size_t ws_bytes, void* stream);
LS_API ls_status ls_replay_bwd_part(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                                    const void* q, const void* k_resp, const void* v_resp,
                                    const void* d_o, const float* lse, const float* delta,
                                    int32_t resp_len, int32_t with_response, float* dq_part,
                                    void* dk_resp, void* dv_resp, void* ws, size_t ws_bytes,
                                    void* stream);

/* Sum of float32 partials: out[i] = sum_s parts[s][i] (float32
 * accumulation, in part order), written in out_dtype.  parts float32
 * [n_parts][n_elems], 16-byte aligned; n_elems % 4 == 0; n_parts == 0 writes
 * zeros.  The dQ reduction of A6 as a call of its own, for callers that hold
 * several dQ shares (context-parallel ranks without a collective, or prompt
 * pages streamed from host memory in chunks). */
LS_API ls_status ls_sum_parts(int32_t n_parts, int64_t n_elems, const float* parts,
                              int32_t out_dtype, void* out, void* stream);

/* Staging of prompt pages kept outside HBM (the GLM path of the DeepRead
 * summary, Method, keeps its prompt state in CPU memory and stages it per
 * layer; on GB300 the Grace memory sits behind the coherent CPU-GPU link).
 * Copies logical pages first_page .. first_page + n_pages - 1 of a prompt,
 * K and V, from source pools [src_pages][Hkv][S_p][d] into staging pools
 * [n_pages][Hkv][S_p][d], in logical order:
 *   k_dst[i] = k_src[page_table[first_page + i]], likewise v.
 * The GPU reads the sources directly (one kernel, no copy-engine calls), so
 * they must be device memory or pinned host memory (pageable host memory is
 * refused with LS_ERR_INVALID_ARGUMENT).  page_table is device memory and
 * holds at least first_page + n_pages entries; the staging pools hold
 * n_pages pages.  An entry outside [0, src_pages) zeroes its staging page and
 * is reported through the status word of ws (ws may be NULL).  Pages are
 * copied bit for bit.  0 <= n_pages <= 65535.  The interface is this
 * library's. */
LS_API ls_status ls_stage_pages(const ls_attn_desc* desc, const void* k_src, const void* v_src,
                                int64_t src_pages, const int32_t* page_table, int64_t first_page,
                                int32_t n_pages, void* k_dst, void* v_dst, void* ws,
                                size_t ws_bytes, void* stream);

/* Gated-DeltaNet state replay (the Qwen model's recurrent layers keep a
 * fixed-size state for the prompt and replay each response from it with that
 * state detached: DeepRead summary, Method, Qwen path; review sections 二,
 * 三).  The pages name the layer but not its recurrence.  This library takes
 * the published gated delta rule, per member and head, with S [dv][dk] and
 * S_0 the captured state:
 *   a_t = exp(g_t);  S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T;
 *   o_t = S_t q_t.
 * A call replays `batch` members of one group, all of resp_len tokens, from
 * one shared S_0.  float32 throughout, row-major, device memory:
 *   s0 [H][dv][dk] (shared);  s_final [B][H][dv][dk];
 *   q, k [B][R][H][dk];  v, o [B][R][H][dv];  g, beta [B][R][H].
 * Supported: dk = dv = 128.  s0 and the token buffers are read only.
 * ls_gdn_replay_fwd writes o and, if s_final is non-NULL, the state after the
 * last token.  ls_gdn_replay_bwd returns the gradient of sum(d_o * o) for q,
 * k, v, g and beta (same shapes); none is formed for s0 (the detached prompt
 * state).  The backward, and the forward with LS_GDN_TENSOR_CORE, need
 * ls_gdn_workspace_size() bytes of workspace (256-byte aligned, owned by the
 * caller; the forward with LS_GDN_EXACT takes ws = NULL, ws_bytes = 0, and
 * ignores a workspace it is given).  The workspace starts with the same
 * 256-byte device status word as the attention workspace: a bounded device
 * wait that ran out in the tensor-core path sets it, and
 * ls_read_device_status(ws) reports it (the outputs of that call are then
 * not to be used).  resp_len == 0 or batch == 0 is a no-op (the forward still
 * copies s0 to s_final when R = 0).
 *
 * precision selects the kernels (a zeroed desc selects the exact path):
 *   LS_GDN_EXACT        float32 recurrence, one token at a time; about 1e-7
 *                       relative error, held to 1e-5 against the float64
 *                       oracle.
 *   LS_GDN_TENSOR_CORE  the chunk-parallel forward and backward (chunks of
 *                       128 tokens) on tcgen05 tensor cores with bf16
 *                       operands and float32 accumulation; about 5e-3
 *                       relative error, held to 2e-2 (the bf16 bar).  s0, q,
 *                       k, v, d_o and the outputs must be 16-byte aligned
 *                       (else LS_ERR_CUDA).
 * Float32 callers that need the 1e-5 result keep LS_GDN_EXACT.
 * Errors: LS_ERR_UNSUPPORTED for other dk/dv, LS_ERR_INVALID_ARGUMENT for
 * NULL buffers, negative sizes, an unknown precision or unknown flags,
 * LS_ERR_WORKSPACE_TOO_SMALL; all before any launch. */
typedef enum { LS_GDN_EXACT = 0, LS_GDN_TENSOR_CORE = 1 } ls_gdn_precision;

/* flags (0 by default):
 *   LS_GDN_BWD_REUSES_FORWARD  with LS_GDN_TENSOR_CORE, the backward takes the
 *       forward's per-chunk terms and states from ws instead of forming them
 *       again: the caller promises that ws was last written by
 *       ls_gdn_replay_fwd with the same desc precision, buffers and resp_len
 *       (the inputs unchanged since).  The results are then the ones the
 *       backward forms without the flag, bit for bit; if the promise is
 *       broken they are wrong (every access still stays inside ws).  Ignored
 *       by LS_GDN_EXACT. */
enum { LS_GDN_BWD_REUSES_FORWARD = 1 };

typedef struct {
  int32_t batch;
  int32_t heads;
  int32_t dk;
  int32_t dv;
  int32_t precision; /* ls_gdn_precision */
  int32_t flags;     /* LS_GDN_BWD_REUSES_FORWARD or 0 */
} ls_gdn_desc;

LS_API ls_status ls_gdn_workspace_size(const ls_gdn_desc* desc, int32_t resp_len, size_t* bytes);
LS_API ls_status ls_gdn_replay_fwd(const ls_gdn_desc* desc, const float* s0, const float* q,
                                   const float* k, const float* v, const float* g,
                                   const float* beta, int32_t resp_len, float* o, float* s_final,
                                   void* ws, size_t ws_bytes, void* stream);
LS_API ls_status ls_gdn_replay_bwd(const ls_gdn_desc* desc, const float* s0, const float* q,
                                   const float* k, const float* v, const float* g,
                                   const float* beta, const float* d_o, int32_t resp_len,
                                   float* dq, float* dk, float* dv, float* dg, float* dbeta,
                                   void* ws, size_t ws_bytes, void* stream);

/* Prompt prefill with capture (the capture step of the DeepRead summary,
 * Method: the shared prompt is run once without gradients and its
 * full-attention K/V are kept as pages; the summary's Key Results put most
 * of the wall time in this no-gradient prefill).  Two steps on one stream:
 *   1. page write, as ls_kv_page_write with start_pos 0: token t of k, v
 *      ([n_tok][Hkv][d]) goes to pool[page_table[t/S_p]][kv][t%S_p][:];
 *   2. causal self-attention of the prompt: o [n_tok][Hq][d] (element dtype)
 *      and lse float32 [n_tok][Hq] (natural log, scale included), row t over
 *      keys 0..t of k, v (read from the contiguous k, v, not the pages).
 * Step 2 is the replay forward with an empty prompt and the prompt in the
 * response's place, so it runs on the same kernels.  ws must hold
 * ls_prompt_prefill_workspace_size() bytes (float32 partials of n_tok rows);
 * a page-table entry outside the pool is skipped and reported through the
 * workspace status word.  n_tok == 0 is a no-op.  No counterpart in the pages
 * beyond the step itself: the interface is this library's. */
LS_API ls_status ls_prompt_prefill(const ls_attn_desc* desc, const void* q, const void* k,
                                   const void* v, int32_t n_tok, void* o, float* lse,
                                   void* k_pool, void* v_pool, int64_t pool_pages,
                                   const int32_t* page_table, int64_t num_pages, void* ws,
                                   size_t ws_bytes, void* stream);

/* Workspace bytes ls_prompt_prefill needs for n_tok tokens.  Host-only. */
LS_API ls_status ls_prompt_prefill_workspace_size(const ls_attn_desc* desc, int32_t n_tok,
                                                  size_t* bytes);

/* Replay forward (same arguments and results as ls_replay_fwd) for callers
 * that cannot allocate device memory: no workspace argument; the library's
 * own fixed 64 MiB device scratch (held by every GPU that loads the library
 * until exit) takes the workspace's place.  The pages have no counterpart to
 * this call; it exists for embedders that own every allocation.
 * The first call on each device looks up the scratch's device address with
 * that device current; make it before any stream capture.  All calls share
 * the one scratch, so calls that overlap on the GPU race.  A call that would
 * need more scratch than 64 MiB returns LS_ERR_WORKSPACE_TOO_SMALL.  Device
 * status bits set by this call are not reported (the status word lives in
 * the scratch). */
LS_API ls_status ls_replay_fwd_noalloc(const ls_attn_desc* desc, const ls_prompt_kv* prompt,
                                       const void* q, const void* k_resp, const void* v_resp,
                                       int32_t resp_len, void* o, float* lse, void* stream);

/* Bytes of the fixed scratch ls_replay_fwd_noalloc uses (64 MiB). */
LS_API size_t ls_replay_fwd_noalloc_scratch_bytes(void);

/* ---------------------------------------------------------------------------
 * Rollout and scoring: the quantised K/V cache, attention of new tokens over
 * it, and log-probabilities over the vocabulary.  A GRPO step decodes the
 * group's responses over the captured prompt, scores the sampled tokens and
 * starts the backward pass from their log-probabilities; the pages name these
 * stages (the five-stage transaction of the review's mind map, capture to
 * policy replay) and give no interface, so the interfaces are this library's.
 * ------------------------------------------------------------------------- */

/* How a cache holds a row (one token's K or V of one KV head).
 *   LS_CACHE_F32, LS_CACHE_BF16: the values.
 *   LS_CACHE_E4M3: 8-bit codes (4 exponent bits, 3 of mantissa, no infinity)
 *     and one exponent e per row, value = code * 2^e.  ls_cache_write takes
 *     the least e with max|row| <= 448 * 2^e (not below -126; 0 for a row of
 *     zeros) and rounds to nearest even, so a value keeps a relative error of
 *     2^-4 down to max|row| / 2^15.  e = -128 marks a row that held an
 *     infinity or a NaN: all of it reads as NaN. */
typedef enum { LS_CACHE_F32 = 0, LS_CACHE_BF16 = 1, LS_CACHE_E4M3 = 2 } ls_cache_format;

/* A paged cache of one layer (device pointers).  k, v: [pool_pages][Hkv][S_p][d]
 * in the format's elements; k_exp, v_exp: int8 [pool_pages][Hkv][S_p], E4M3
 * only (NULL otherwise).  head_dim in {64, 128, 256}.  A pool in bf16 or
 * float32 is laid out as ls_prompt_kv's, so a captured prompt is a cache as
 * it stands.  A slot is a row's place: page * S_p + row in the page. */
typedef struct {
  int32_t format;
  int32_t hkv;
  int32_t head_dim;
  int32_t page_size;
  int64_t pool_pages;
  void* k;
  void* v;
  int8_t* k_exp;
  int8_t* v_exp;
} ls_kv_cache;

/* Writes token t's rows of k, v (src_dtype; heads contiguous, token t at
 * element t * k_stride / t * v_stride, both multiples of 8) into slot
 * slots[t].  A negative slot skips the token; one past the pool is skipped and
 * reported through ws's status word (ws may be NULL).  Two tokens of one call
 * must not share a slot.  n_tok == 0 is a no-op. */
LS_API ls_status ls_cache_write(const ls_kv_cache* cache, int32_t src_dtype, const void* k,
                                const void* v, int64_t k_stride, int64_t v_stride,
                                const int64_t* slots, int64_t n_tok, void* ws, size_t ws_bytes,
                                void* stream);

/* Reads slots[t] into token t of k, v ([n_tok][Hkv][d], dst_dtype).  E4M3
 * values are exact in both dtypes (bf16 values below 2^-133 aside).  A negative slot
 * gives zeros, one past the pool zeros and the status word. */
LS_API ls_status ls_cache_read(const ls_kv_cache* cache, const int64_t* slots, int64_t n_tok,
                               int32_t dst_dtype, void* k, void* v, void* ws, size_t ws_bytes,
                               void* stream);

/* Attention of each sequence's new tokens over its pages, in which the new
 * tokens' own K/V already are.  Sequence b has query tokens q_start[b] ..
 * q_start[b+1]-1 of q and keys 0 .. kv_len[b]-1 (key j in page
 * page_table[b][j / S_p], row j % S_p).  With causal, its token i of n sees
 * keys up to kv_len[b] - n + i, else all; o is the softmax's mean of V, lse
 * its natural log-sum-exp (scale included).  A token that sees no key
 * gives o = 0, lse = -infinity.  Rows of the pages past kv_len may hold
 * anything; a NaN in a key that a token sees makes that token's rows NaN (a NaN
 * or an infinity in a bf16 or float32 value row, which weights of 0 multiply too,
 * perhaps also those of the sequence's earlier tokens in the call).  An E4M3 value
 * row more than 2^80 times smaller than the sequence's largest may count as 2^-80
 * of that.  Without causal, several members' tokens over a prompt that they
 * share are one sequence; a float32 o and lse are then parts for ls_lse_merge.
 *   q_dtype / o_dtype: o_dtype is q_dtype or LS_DTYPE_F32.
 *   max_q, max_kv: upper bounds of the lengths (max_q <= total_q <= batch *
 *     max_q), for planning and the workspace; a longer sequence of queries is
 *     refused on the device (its keys are not read, its o and lse hold nothing of
 *     use, the status word says so), a longer kv_len is computed, more slowly.
 *     kv_len is at most pages_per_seq * S_p (more is cut there and reported).
 *   q_stride: elements from one token of q to the next (a multiple of 8, at
 *     least Hq * d); o is contiguous. */
typedef struct {
  int32_t q_dtype;
  int32_t o_dtype;
  int32_t hq;
  int32_t batch;
  int64_t total_q;
  int32_t max_q;
  int32_t causal;
  int64_t max_kv;
  int64_t q_stride;
  float softmax_scale;
} ls_cached_attn_desc;

LS_API ls_status ls_cached_attn_workspace_size(const ls_cached_attn_desc* desc,
                                               const ls_kv_cache* cache, size_t* bytes);

/* q [total_q][Hq][d]; q_start int32 [batch+1] from 0 to total_q; kv_len int64
 * [batch]; page_table int32 [batch][pages_per_seq]; o [total_q][Hq][d]; lse
 * float32 [total_q][Hq].  All on the device.  A page id outside the pool that
 * a length reaches holds no keys and is reported. */
LS_API ls_status ls_cached_attn(const ls_cached_attn_desc* desc, const ls_kv_cache* cache,
                                const void* q, const int32_t* q_start, const int64_t* kv_len,
                                const int32_t* page_table, int64_t pages_per_seq, void* o,
                                float* lse, void* ws, size_t ws_bytes, void* stream);

/* Log-probabilities of target tokens over a large vocabulary and their
 * gradients, without the logits in memory: with x_v = logit_scale * (h_n . w_v),
 *   lse_n = log sum_v exp(x_v),  logp_n = x_target - lse_n  (minus the softmax
 *   cross entropy),  d logp_n / d x_v = [v = target] - exp(x_v - lse_n).
 * h [n_rows][hidden], w [vocab][hidden] in dtype, row strides in elements.
 * A row whose target is ignore_index has logp 0 and no gradient (its lse is
 * still written); any other target outside [0, vocab) is treated the same and
 * reported through the status word.  An ignored row's h and d_logp reach no
 * other row's results, but dw multiplies its h by 0: it has to be finite there.
 * Sums are float32; dh and dw are rounded to dtype once.  bf16 with hidden,
 * strides and addresses in multiples of 16 bytes runs on the tensor cores,
 * where the backward also rounds the logits' gradient to bf16, once, as the
 * operand of its two products; float32 and other layouts run on the CUDA
 * cores.
 *   piece: vocabulary columns whose gradient is held at a time in the backward
 *     (0: chosen from n_rows); the workspace grows with it. */
typedef struct {
  int32_t dtype;
  int32_t hidden;
  int32_t vocab;
  int32_t piece;
  int64_t n_rows;
  int64_t h_stride;
  int64_t w_stride;
  int64_t ignore_index;
  float logit_scale;
} ls_vocab_desc;

/* with_grad != 0: enough for the backward too (one buffer serves both). */
LS_API ls_status ls_vocab_logprob_workspace_size(const ls_vocab_desc* desc, int32_t with_grad,
                                                 size_t* bytes);

/* targets int64 [n_rows]; logp, lse float32 [n_rows]. */
LS_API ls_status ls_vocab_logprob_fwd(const ls_vocab_desc* desc, const void* h, const void* w,
                                      const int64_t* targets, float* logp, float* lse, void* ws,
                                      size_t ws_bytes, void* stream);

/* lse: what the forward wrote for the same inputs; d_logp float32 [n_rows]:
 * the loss's gradient for logp.  dh [n_rows][hidden], dw [vocab][hidden]
 * (contiguous, dtype) are overwritten; either may be NULL. */
LS_API ls_status ls_vocab_logprob_bwd(const ls_vocab_desc* desc, const void* h, const void* w,
                                      const int64_t* targets, const float* lse,
                                      const float* d_logp, void* dh, void* dw, void* ws,
                                      size_t ws_bytes, void* stream);

/* Pages of a paged cache, kept on the device: which pages a sequence has, and
 * who else has them.  One book serves the caches of all layers whose pages are
 * numbered alike.
 *   refs int32 [pool_pages]: how many table entries name the page, 0 if free;
 *   page_table int32 [n_seqs][pages_per_seq], kv_len int64 [n_seqs]: as
 *   ls_cached_attn takes them (a run of rows of a table is a table).  A sequence
 *   of n tokens has its first ceil(n / S_p) entries; the others mean nothing.
 * A new book is all zeros.  Page ids outside the pool in a table are left out
 * and reported.  A call whose lists are not valid (a sequence out of range or
 * named twice, a length out of range, q_start not rising from 0 to total_q)
 * changes nothing but the results for the caller (slots and copies all -1), and
 * is reported.  The book's tensors, the lists and the results must not overlap (but
 * kv_len may be the list of lengths that are kept).  ws: ls_pages_workspace_size()
 * bytes, for one call at a time. */
typedef struct {
  int32_t page_size;
  int32_t n_seqs;
  int32_t pages_per_seq;
  int32_t pool_pages;
  int32_t* refs;
  int32_t* page_table;
  int64_t* kv_len;
} ls_page_book;

LS_API ls_status ls_pages_workspace_size(const ls_page_book* book, size_t* bytes);

/* Sequences drop tokens from their ends and take slots for new ones (a step of
 * a rollout: the rejected drafts go, the next ones come).  For each i < n,
 * sequence seqs[i] (i where seqs is NULL) keeps its first keep[i] tokens (all
 * where keep is NULL) and grows by q_start[i+1] - q_start[i] (nothing where
 * q_start is NULL); slots[t], t in q_start's order, gets the slot of each new
 * token, as ls_cache_write takes it.  First all pages that are dropped lose a
 * reference; then pages are taken in order of i, each time the free page of the
 * lowest number.  A sequence that grows inside a page that others name too gets
 * a page of its own for it: copies[i] = (from, to, rows), which the caller hands
 * to ls_cache_copy_pages for every layer's cache before it writes; -1s where
 * nothing is to be copied.  Where the free pages do not reach, or the table's
 * row ends, the sequence does not grow (slots -1, which ls_cache_write leaves
 * out), and the status word says so (LS_ERR_OUT_OF_PAGES); later ones still do
 * if they need no page.
 *   keep int64 [n]; q_start int32 [n+1]; slots int64 [total_q] (total_q at most 2^29);
 *   copies int32 [n][3]. */
LS_API ls_status ls_pages_advance(const ls_page_book* book, int32_t n, const int32_t* seqs,
                                  const int64_t* keep, const int32_t* q_start, int64_t total_q,
                                  int64_t* slots, int32_t* copies, void* ws, size_t ws_bytes,
                                  void* stream);

/* Frees the pages of sequences seqs[i] (all n_seqs where seqs is NULL): length 0. */
LS_API ls_status ls_pages_release(const ls_page_book* book, int32_t n, const int32_t* seqs,
                                  void* ws, size_t ws_bytes, void* stream);

/* Sequence dst[i] becomes the first lens[i] tokens (lens NULL: all) of sequence
 * src[i], without a copy: its own pages are freed, src's gain a reference.  (The
 * page that both end in is copied when one of them grows.)  The same src may be
 * named many times; a dst must be named once and be no src. */
LS_API ls_status ls_pages_fork(const ls_page_book* book, int32_t n, const int32_t* src,
                               const int32_t* dst, const int64_t* lens, void* ws, size_t ws_bytes,
                               void* stream);

/* Moves the pages in use to the front of the pool: with A of them, the k-th one
 * numbered A or more goes to the k-th free one below A.  table_out and refs_out
 * get the book's table and references after the moves (they may be the book's
 * own); copies int32 [pool_pages / 2][3] gets the moves for ls_cache_copy_pages,
 * -1s after the last. */
LS_API ls_status ls_pages_compact(const ls_page_book* book, int32_t* table_out, int32_t* refs_out,
                                  int32_t* copies, void* ws, size_t ws_bytes, void* stream);

/* Copies rows of pages within a cache, K and V: for each i < n, the first
 * copies[i][2] rows of page copies[i][0] to page copies[i][1], for every head.
 * A negative page leaves the entry out; one past the pool, or more rows than a
 * page has, is left out and reported (ws: the status word, or NULL).  A page
 * must not be written by two entries, nor be read by one and written by another. */
LS_API ls_status ls_cache_copy_pages(const ls_kv_cache* cache, const int32_t* copies, int64_t n,
                                     void* ws, size_t ws_bytes, void* stream);

/* Verification of drafted tokens against the target's logits, and the draw of
 * the token after them, from given random numbers: the tokens that come out are
 * distributed as if each had been drawn from the target.  Rows lie as the query
 * tokens of ls_cached_attn: sequence b has rows r = q_start[b] .. q_start[b+1]-1,
 * tokens[r] its last token and then its drafts, and logits row r is for the
 * token after tokens[r], so that it judges the draft tokens[r+1].  With
 *   p_r(v) = exp(logit_scale * logits[r][v] - lse_r)   (1 / temperature in logit_scale)
 * and q_r = draft_probs[r] what that draft was drawn from (draft_probs NULL: q_r is 1
 * at the draft), the drafts are accepted while u[r] * q_r(x) < p_r(x).  At the row
 * where that ends the next token is the least v with
 *   sum_{j <= v} w_j > u_next[b] * sum_j w_j,
 * w = max(p - q, 0) after a rejection (p where its sum is at most 2^-30) and p after the
 * last draft.  So a sequence of n rows has 1 to n tokens come out: emitted[r] =
 * accepted drafts, then the new token, then -1s; logp[r] = log p_r(emitted[r]), 0
 * where there is none; n_emitted[b] their number; keep[b] = kv_len[b] - n +
 * n_emitted[b], the tokens whose keys stay valid (what ls_pages_advance keeps and, as
 * n_use, n_emitted makes ls_gdn_decode keep; but see the row without a distribution).
 * A sequence without rows has none:
 * n_emitted 0, keep its kv_len.  Rows that judge no draft may hold anything in
 * draft_probs and u; elsewhere what is not above 0 in draft_probs counts as 0.
 *   logits may be -infinity or the type's lowest value (a masked token); a draft's
 *     probability below 2^-149 of the row's largest is 0.  A row
 *     that has no distribution (all -infinity, or a NaN or +infinity in it) accepts
 *     nothing; where it had to give the next token, emitted is -1 there, n_emitted
 *     counts the drafts before it, keep their keys and the last token's, and the
 *     status word says so.  There n_emitted is one less than the tokens that are kept:
 *     a caller that goes on gives ls_gdn_decode n_use = keep - kv_len + n, which is
 *     n_emitted for all other sequences that were not left out.  A draft outside [0, vocab) is rejected and reported.
 *   An acceptance within 2^-16 of its border (relative; twice that for each
 *     doubling of vocab beyond 2^17; about 2^-20 in practice) may fall either way.
 *     The weights of the draw are good to 2^-30 each (those below 2^-23 of the row to
 *     2^-47 of it) and their sums to about 2^-31 of the row, so that in a vocabulary
 *     of 10^5 one draw in some thousands gives a neighbour of the definition's token.
 *     A token below 2^-60 of the row is never drawn.
 *   vocab: at most 2^24.
 *   dtype: of logits; draft_probs is float32.  Strides in elements, any.
 *   logit_scale: 2^-100 to 2^100. */
typedef struct {
  int32_t dtype;
  int32_t vocab;
  int32_t batch;
  int32_t max_q;
  int64_t total_q;
  int64_t logits_stride;
  int64_t draft_stride;
  float logit_scale;
} ls_verify_desc;

LS_API ls_status ls_draft_verify_workspace_size(const ls_verify_desc* desc, size_t* bytes);

/* logits [total_q][vocab], draft_probs [total_q][vocab] or NULL, tokens int64
 * [total_q], q_start int32 [batch+1] from 0 to total_q, u float32 [total_q] and u_next
 * float32 [batch] in [0, 1); n_emitted int32 [batch], emitted int64 [total_q], logp
 * float32 [total_q] or NULL; kv_len and keep int64 [batch], or keep NULL.  max_q is an
 * upper bound of a sequence's rows (max_q <= total_q <= batch * max_q); a sequence with
 * more, or with rows outside [0, total_q), is left out (n_emitted 0, its rows of emitted
 * and logp as they were, keep its kv_len) and reported.  The results must not overlap
 * the inputs; but keep may be kv_len (not a book's: ls_pages_advance has to see the
 * length before as well, or the pages between stay taken). */
LS_API ls_status ls_draft_verify(const ls_verify_desc* desc, const void* logits,
                                 const float* draft_probs, const int64_t* tokens,
                                 const int32_t* q_start, const float* u, const float* u_next,
                                 const int64_t* kv_len, int32_t* n_emitted, int64_t* emitted,
                                 float* logp, int64_t* keep, void* ws, size_t ws_bytes,
                                 void* stream);

/* Recurrent step of the gated-DeltaNet state (the layer of ls_gdn_replay_fwd),
 * for one or a few new tokens of each sequence: the decoding of the layers that
 * keep a fixed-size state.  Each sequence has a slot in a pool of states; its
 * tokens t = q_start[b] .. q_start[b+1]-1 move the state on in order,
 *   S <- exp(g_t) S;  S <- S + b_t (v_t - S k_t) k_t^T;  o_t = S q_t,
 * from the state in slot state_in[b] (-1: a state of zeros) to slot
 * state_out[b] (-1, or state_out NULL: not kept; the same slot: in place).  So a
 * group forks the captured prompt's state by reading one slot and writing
 * several, drafted tokens run ahead of a state that stays, and the accepted ones
 * move it on by a second call with n_use.  A sequence without tokens copies its
 * state.  A slot that is written must not be read or written by another
 * sequence of the call.  All sums are float32.
 *   dtype: of q, k, v and o; states, g and beta are float32.
 *   key_heads divides heads: value head h takes q and k of head
 *     h / (heads / key_heads).  q, k [total_q][key_heads][dk], v [total_q][heads][dv],
 *     token strides in elements, multiples of 8 (rows of one projection as they
 *     lie); g, beta [total_q][heads] and o [total_q][heads][dv] contiguous.  o and
 *     the states must not overlap each other or anything that the call reads.
 *   states [n_states][heads][dv][dk].  dk = dv = 128.
 *   max_q: upper bound of a sequence's tokens (max_q <= total_q <= batch * max_q). */
typedef struct {
  int32_t dtype;
  int32_t heads;
  int32_t key_heads;
  int32_t dk;
  int32_t dv;
  int32_t batch;
  int32_t max_q;
  int32_t reserved;
  int64_t total_q;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  int64_t n_states;
} ls_gdn_decode_desc;

/* q_start int32 [batch+1], from 0 to total_q; n_use int32 [batch] or NULL: only
 * the first n_use[b] tokens of sequence b count (the others' rows of o stay as
 * they were); state_in int32 [batch]; state_out int32 [batch] or NULL; o or NULL.
 * ws: 256 bytes, the status word, or NULL.  A sequence whose state_in, token
 * range or n_use is out of range is left out and reported; a state_out past the
 * pool is not written and reported. */
LS_API ls_status ls_gdn_decode(const ls_gdn_decode_desc* desc, float* states, const void* q,
                               const void* k, const void* v, const float* g, const float* beta,
                               const int32_t* q_start, const int32_t* n_use,
                               const int32_t* state_in, const int32_t* state_out, void* o, void* ws,
                               size_t ws_bytes, void* stream);

/* Synchronises the stream, then reports the device status word of ws
 * (LS_OK, LS_ERR_DEVICE_BOUNDS or LS_ERR_DEVICE_TIMEOUT) and clears it. */
LS_API ls_status ls_read_device_status(void* ws, size_t ws_bytes, void* stream);

/* Zeroes the workspace status word (asynchronous on the stream). */
LS_API ls_status ls_clear_device_status(void* ws, size_t ws_bytes, void* stream);

LS_API const char* ls_status_string(ls_status status);
/* One-line reason for the last non-OK status returned on this thread. */
LS_API const char* ls_last_error(void);

/* Tracing.  When enabled, every kernel launch is bracketed by CUDA events on
 * its own stream and accumulated per kernel id; ls_trace_read synchronises
 * those events and reports launches and total milliseconds since the last
 * reset.  ls_launch_count counts every kernel this library launched in this
 * process (traced or not). */
LS_API ls_status ls_trace_enable(int32_t on);
LS_API ls_status ls_trace_reset(void);
LS_API ls_status ls_trace_read(int32_t kernel_id, int64_t* launches, double* total_ms);
LS_API int32_t ls_num_kernel_ids(void);
LS_API const char* ls_kernel_name(int32_t kernel_id);
LS_API int64_t ls_launch_count(void);

/* Which prompt-attention implementation the current device and desc select:
 * 1 = tcgen05/TMEM tensor-core kernels, 0 = CUDA-core kernels. */
LS_API int32_t ls_uses_tensor_cores(const ls_attn_desc* desc);

#ifdef __cplusplus
}
#endif

#endif /* LS_H_ */
