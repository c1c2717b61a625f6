// Internal declarations shared by the libls translation units (not installed).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ls.h"

namespace ls {

// Bits of the device status word (first 4 bytes of the workspace).  The
// next word records the first bounded wait that gave up: kernel id << 16 | line.
enum : uint32_t {
  kStatusBadPage = 1u,   // a page-table entry pointed outside the pool
  kStatusTimeout = 2u,   // a bounded device wait gave up
  kStatusBadIndex = 4u,  // a slot, length or target was out of range
  kStatusNoPages = 8u,   // a sequence could not grow
};

// Bytes at the head of the workspace reserved for the status word.
constexpr size_t kWsHeader = 256;

// Runs every host-side check ls_replay_fwd makes (descriptor, prompt,
// pointers, alignment) without launching anything, and gives the workspace
// bytes the call needs on the current device.
ls_status replay_fwd_validate(const ls_attn_desc* desc, const ls_prompt_kv* prompt, const void* q,
                              const void* k_resp, const void* v_resp, int32_t resp_len,
                              const void* o, const float* lse, size_t* ws_need);

// Kernel ids used by tracing (ls_trace_read / ls_kernel_name).
enum KernelId : int32_t {
  kKPageWrite = 0,
  kKSimtFwd,
  kKTcFwd,
  kKLseMerge,
  kKBwdPre,
  kKSimtBwdDq,
  kKTcBwdDq,
  kKSimtDkDv,
  kKTcDkDv,
  kKDqReduce,
  kKGdnFwd,
  kKGdnBwd,
  kKStagePages,
  kKCacheWrite,
  kKCacheRead,
  kKCachedSimt,
  kKCachedMma,
  kKCachedTc,
  kKCachedJoin,
  kKVocabSimt,
  kKVocabTc,
  kKVocabReduce,
  kKGdnDecode,
  kKPages,
  kKPageCopy,
  kKVerifyRows,
  kKVerifyDraw,
  kNumKernelIds
};

// Launch bookkeeping (ls_api.cu): count every launch, optionally bracket it
// with events on its stream.
struct LaunchScope {
  LaunchScope(int32_t kid, cudaStream_t s);
  ~LaunchScope();
  // A scope counts as one kernel launch; a launcher that runs n kernels
  // under one scope (one trace entry) adds the other n - 1 here.
  void more_kernels(int n);
  int32_t kid;
  cudaStream_t stream;
  void* ev0;
  void* ev1;
};

// Rows of one KV group are numbered t = hh * R + r (hh = head within group).
// Output row index is n = r * Hq + h with h = g * Gq + hh.

// Common geometry of the attention kernels.
struct AttnGeom {
  int32_t hq, hkv, gq, d, page_size;
  int32_t R;             // response length
  int64_t P;             // prompt length
  int64_t pool_pages;
  float scale;           // softmax scale
  float scale_log2;      // scale * log2(e)
  int32_t ns;            // prompt splits (part ns is the response part)
  int64_t split_span;    // prompt keys per split (a multiple of every key tile)
  bool resp_part;        // compute part ns; false on a context-parallel rank
                         // that does not hold the response (parts 0..ns-1 only)
};

// Parts a forward/backward launch covers: the ns prompt splits plus the
// causal response part when it is wanted.
inline int launch_parts(const AttnGeom& g) { return g.ns + (g.resp_part ? 1 : 0); }

struct FwdParams {
  AttnGeom g;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* page_table;
  const void* k_resp;
  const void* v_resp;
  float* o_parts;    // [n_parts][R*Hq][d]
  float* lse_parts;  // [n_parts][R*Hq]
  uint32_t* status;
};

struct BwdParams {
  AttnGeom g;
  const void* q;
  const void* d_o;
  const float* lse;    // [R][Hq]
  const float* delta;  // [R][Hq]
  const void* k_pool;
  const void* v_pool;
  const int32_t* page_table;
  const void* k_resp;
  const void* v_resp;
  float* dq_parts;     // [n_parts][R*Hq][d], unscaled
  void* dk;            // [R][Hkv][d] element dtype
  void* dv;
  uint32_t* status;
};

// CUDA-core kernels (ls_simt.cu)
cudaError_t launch_page_write(int dtype, int hkv, int d, int page_size, void* k_pool,
                              void* v_pool, int64_t pool_pages, const int32_t* pt,
                              int64_t start_pos, int64_t n_tok, const void* k,
                              const void* v, uint32_t* status, cudaStream_t s);
cudaError_t launch_simt_fwd(int dtype, const FwdParams& p, cudaStream_t s);
cudaError_t launch_simt_fwd_resp(int dtype, const FwdParams& p, cudaStream_t s);
// Whole pages of a device-readable source pool into a staging pool (ls_stage_pages).
cudaError_t launch_stage_pages(int64_t page_bytes, const void* k_src, const void* v_src,
                               int64_t src_pages, const int32_t* pt, int64_t first, int n_pages,
                               void* k_dst, void* v_dst, uint32_t* status, cudaStream_t s);
cudaError_t launch_lse_merge(int n_parts, int64_t n_rows, int d, const float* o_parts,
                             const float* lse_parts, int out_dtype, void* o, float* lse,
                             cudaStream_t s);
cudaError_t launch_bwd_preprocess(int dtype, int64_t n_rows, int d, const void* o,
                                  const void* d_o, float* delta, cudaStream_t s);
cudaError_t launch_simt_bwd_dq(int dtype, const BwdParams& p, cudaStream_t s);
cudaError_t launch_simt_bwd_dq_resp(int dtype, const BwdParams& p, cudaStream_t s);
cudaError_t launch_simt_dkdv(int dtype, const BwdParams& p, cudaStream_t s);
cudaError_t launch_dq_reduce(int n_parts, int64_t n_rows, int d, float scale,
                             const float* parts, int out_dtype, void* dq, cudaStream_t s);

// Tensor-core kernels (ls_tc_fwd.cu, ls_tc_bwd.cu): bf16, d = 256,
// page_size % 128 == 0, sm_100-family device.  Query tiles are 128 rows;
// split spans are multiples of kTcSpanQuantum keys.
constexpr int kTcRows = 128;
constexpr int kTcSpanQuantum = 128;
cudaError_t launch_tc_fwd(const FwdParams& p, cudaStream_t s);
cudaError_t launch_tc_bwd_dq(const BwdParams& p, cudaStream_t s);

// 2-D TMA map over a bf16 matrix [rows][256] with [box_rows x 64] boxes and
// the 128-byte swizzle (ls_api.cu; cuTensorMapEncodeTiled resolved once
// through the runtime, no -lcuda).
// Sets the message ls_last_error() returns on this thread.
void set_last_error(const char* msg);

ls_status fail(ls_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ls_status check_ws(const void* ws, size_t ws_bytes, size_t need);
ls_status check_cache(const ls_kv_cache* c);
// j / d = umulhi(j, mul) >> shift for 0 <= j < 2^31 (mul 0: d is 1).
void page_divisor(uint32_t d, uint32_t* mul, uint32_t* shift);
int device_sms();
bool device_is_sm100_family();
bool force_simt();  // LS_FORCE_SIMT is set

bool encode_pool_map(CUtensorMap* m, const void* base, int64_t rows, int box_rows);
// 3-D TMA map over a bf16 tensor [rows][heads][256] with [box_rows x 1 x 64]
// boxes and the 128-byte swizzle (response K/V, Q, dO); rows past the end
// read as zeros.
bool encode_rows_map(CUtensorMap* m, const void* base, int heads, int64_t rows, int box_rows);
// One-instruction [box_rows x 64*box_blocks] tiles landing as box_blocks
// swizzled [box_rows x 64] column boxes (pool rows; token-major rows).
bool encode_pool_tile_map(CUtensorMap* m, const void* base, int64_t rows, int box_rows,
                          int box_blocks = 4);
// A bf16 matrix [rows][cols] of any row stride (16-byte multiple): blocks == 1
// gives a 2-D map with boxes of 64 columns x box_rows (any cols, zeros past the
// end), blocks > 1 a 3-D one (64, rows, cols / 64) whose box lands `blocks`
// column boxes one after the other (cols a multiple of 64).
bool encode_matrix_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t stride,
                       int box_rows, int blocks);
bool encode_rows_tile_map(CUtensorMap* m, const void* base, int heads, int64_t rows, int box_rows,
                          int box_blocks = 4);
cudaError_t launch_tc_dkdv(const BwdParams& p, cudaStream_t s);
// Gated-DeltaNet replay (ls_gdn.cu): dk = dv = 128, one CTA per (head, member).
bool gdn_supported(int dk, int dv);
size_t gdn_workspace_bytes(int B, int H, int R);
cudaError_t launch_gdn_fwd(int B, int H, int R, const float* s0, const float* q, const float* k,
                           const float* v, const float* g, const float* beta, float* o,
                           float* s_final, cudaStream_t st);
// Chunk-parallel tensor-core forward and backward (ls_gdn_cp.cu), precision
// LS_GDN_TENSOR_CORE; both use gdn_cp_workspace_bytes of scratch.
size_t gdn_cp_workspace_bytes(int B, int H, int R);
// status: the workspace status word a wait that gives up sets.
cudaError_t launch_gdn_cp_fwd(int B, int H, int R, const float* s0, const float* q, const float* k,
                              const float* v, const float* g, const float* beta, float* o,
                              float* s_final, float* ws, uint32_t* status, cudaStream_t st);
// reuse_forward: ws holds the scratch of launch_gdn_cp_fwd on the same inputs.
cudaError_t launch_gdn_cp_bwd(int B, int H, int R, const float* s0, const float* q, const float* k,
                              const float* v, const float* g, const float* beta, const float* d_o,
                              float* dq, float* dk, float* dv, float* dg, float* dbeta, float* ws,
                              bool reuse_forward, uint32_t* status, cudaStream_t st);
cudaError_t launch_gdn_bwd(int B, int H, int R, const float* s0, const float* q, const float* k,
                           const float* v, const float* g, const float* beta, const float* d_o,
                           float* dq, float* dk, float* dv, float* dg, float* dbeta, float* ws,
                           cudaStream_t st);

// Quantised cache (ls_cache.cu).
cudaError_t launch_cache_write(const ls_kv_cache& c, int src_dtype, const void* k, const void* v,
                               int64_t k_stride, int64_t v_stride, const int64_t* slots,
                               int64_t n_tok, uint32_t* status, cudaStream_t s);
cudaError_t launch_cache_read(const ls_kv_cache& c, const int64_t* slots, int64_t n_tok,
                              int dst_dtype, void* k, void* v, uint32_t* status, cudaStream_t s);

// Cached attention.  The keys of a sequence are cut into parts of `span`
// keys; part ns-1 takes whatever lies beyond.  Row t of a (sequence, KV head)
// is token t / gq, head t % gq of the group, so that a tile's rows are
// neighbours in time.
struct CachedParams {
  ls_kv_cache c;
  int32_t hq, gq, batch, max_q, causal;
  int32_t q_dtype, o_dtype;
  int64_t total_q, q_stride, pages_per_seq;
  // j / page_size = umulhi(j, page_mul) >> page_shift for 0 <= j < 2^31 (page_mul 0: page_size 1)
  uint32_t page_mul, page_shift;
  float scale, scale_log2;
  int32_t ns;
  int64_t span;
  const void* q;
  const int32_t* q_start;
  const int64_t* kv_len;
  const int32_t* page_table;
  void* o;           // [total_q][hq][d], o_dtype (ns == 1)
  float* lse;
  float* o_parts;    // [ns][total_q * hq][d] (ns > 1)
  float* lse_parts;  // [ns][total_q * hq]
  uint32_t* status;
};
cudaError_t launch_cached_simt(const CachedParams& p, cudaStream_t s);
cudaError_t launch_cached_mma(const CachedParams& p, cudaStream_t s);
// Tiles of 128 rows, or of 256 for a pair of CTAs where there are that many.
cudaError_t launch_cached_tc(const CachedParams& p, cudaStream_t s);
bool cached_tc_pairs(int64_t rows, int d);
// Joins the ns parts (at most kCachedMaxParts) of every row.
constexpr int kCachedMaxParts = 128;
cudaError_t launch_cached_join(const CachedParams& p, cudaStream_t s);
int cached_mma_rows(int d, int format);  // rows that launch_cached_mma takes, at most

// Vocabulary log-probabilities (ls_vocab.cu, ls_vocab_tc.cu).
struct VocabParams {
  ls_vocab_desc d;
  const void* h;
  const void* w;
  const int64_t* targets;
  const float* lse_in;
  const float* d_logp;
  float* logp;
  float* lse;
  void* dh;
  void* dw;
  void* scratch;  // after the status header
  uint32_t* status;
};
// Rows that the forward takes at a time, so that its tiles' statistics stay
// within 8 bytes x 65,536 rows per 256 (or 64) columns.
constexpr int64_t kVocabRows = 65536;
size_t vocab_simt_scratch(const ls_vocab_desc& d, bool with_grad);
// lse and logp from n_tiles (maximum, sum) pairs per row, [tile][row], in base 2.
cudaError_t launch_vocab_join(int n_tiles, const VocabParams& p, const float2* parts, const float* hit,
                              cudaStream_t s);
cudaError_t launch_vocab_simt_fwd(const VocabParams& p, cudaStream_t s);
cudaError_t launch_vocab_simt_bwd(const VocabParams& p, cudaStream_t s);
// bf16; hidden, the row strides and the addresses multiples of 16 bytes.
size_t vocab_tc_scratch(const ls_vocab_desc& d, bool with_grad);
cudaError_t launch_vocab_tc_fwd(const VocabParams& p, cudaStream_t s);
cudaError_t launch_vocab_tc_bwd(const VocabParams& p, cudaStream_t s);

// Recurrent step of the gated-DeltaNet state (ls_gdn_decode.cu).
struct GdnDecodeParams {
  ls_gdn_decode_desc d;
  float* states;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const int32_t* q_start;
  const int32_t* n_use;
  const int32_t* state_in;
  const int32_t* state_out;
  void* o;
  uint32_t* status;
};
cudaError_t launch_gdn_decode(const GdnDecodeParams& p, cudaStream_t s);

// Verification of drafted tokens (ls_verify.cu).
struct VerifyParams {
  ls_verify_desc d;
  float c, c_low;  // logit_scale * log2(e), and what its rounding to float32 left
  const void* logits;
  const float* probs;
  const int64_t* tokens;
  const int32_t* q_start;
  const float* u;
  const float* u_next;
  const int64_t* kv_len;
  int32_t* n_emitted;
  int64_t* emitted;
  float* logp;
  int64_t* keep;
  float2* parts;  // [total_q][chunks] (maximum, sum of the others' exponentials relative to it), or what replaces them
  int32_t chunks;
  uint32_t* status;
};
int verify_chunks(const ls_verify_desc& d);
size_t verify_scratch(const ls_verify_desc& d);
cudaError_t launch_draft_verify(const VerifyParams& p, cudaStream_t s);

// Pages of a cache (ls_pages.cu).  The work arrays lie after the status header.
struct PagesParams {
  ls_page_book b;
  int32_t n;
  const int32_t* seqs;   // advance; fork: the destinations
  const int32_t* src;    // fork
  const int64_t* keep;   // advance; fork: lengths
  const int32_t* q_start;
  int64_t total_q;
  int64_t* slots;
  int32_t* copies;
  int32_t* table_out;
  int32_t* refs_out;
  bool drop_all;         // advance: keep nothing
  uint32_t page_mul, page_shift;  // of a division by page_size (page_divisor)
  int32_t share_shift;   // 2^this threads share a sequence
  int32_t* list;         // [pool_pages] free pages in order
  int32_t* high;         // [pool_pages] compact: pages that move, in order
  int32_t* rank;         // [pool_pages] compact: their places in `high`
  int32_t* owner;        // [8][n_seqs] a block's: who names the sequence
  int32_t* lists;        // [8][7][n_seqs] a block's, where shared memory does not hold them
  uint32_t* status;
};
size_t pages_scratch(const ls_page_book& b);
cudaError_t launch_pages_advance(const PagesParams& p, cudaStream_t s);
cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t s);
cudaError_t launch_pages_compact(const PagesParams& p, cudaStream_t s);
cudaError_t launch_page_copy(const ls_kv_cache& c, const int32_t* copies, int64_t n, uint32_t* status,
                             cudaStream_t s);

}  // namespace ls
