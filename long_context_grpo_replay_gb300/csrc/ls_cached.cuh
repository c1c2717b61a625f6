// What the cached-attention kernels share: the extent of a sequence and of
// one part of its keys, and where rows are written.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "ls_internal.h"

namespace ls {

// The queries and keys of one sequence, clamped to what the call allows;
// anything out of range sets the status word.
struct Seq {
  int q0, n;  // first token and number of tokens
  int kv;     // keys
};
__device__ __forceinline__ Seq load_seq(const CachedParams& p, int b, bool report) {
  Seq s;
  s.q0 = __ldg(p.q_start + b);
  s.n = __ldg(p.q_start + b + 1) - s.q0;
  const int64_t kv = __ldg(p.kv_len + b);
  const int64_t most = p.pages_per_seq * p.c.page_size;
  bool bad = kv < 0 || kv > most;
  s.kv = (int)(kv < 0 ? 0 : kv > most ? most : kv);
  if (s.q0 < 0 || s.n < 0 || s.n > p.max_q || s.q0 > p.total_q - s.n) {
    bad = true;
    s.n = 0;
  }
  if (bad && report) atomicOr(p.status, kStatusBadIndex);
  return s;
}

// Keys [kb, ke) of part `part` that a tile whose last token is `last` sees.
__device__ __forceinline__ void part_range(const CachedParams& p, const Seq& s, int part, int last,
                                           int& kb, int& ke) {
  kb = (int)(part * p.span);
  ke = part == p.ns - 1 || kb + p.span > s.kv ? s.kv : (int)(kb + p.span);
  if (p.causal) {
    const int lim = s.kv - s.n + last + 1;
    ke = ke < lim ? ke : lim;
  }
}

// One past the last key that token i sees.
__device__ __forceinline__ int row_limit(const CachedParams& p, const Seq& s, int i) {
  return p.causal ? s.kv - s.n + i + 1 : s.kv;
}

// The pool row of key j of sequence b, or -1 where the page id lies outside
// the pool (such a page holds no keys).
__device__ __forceinline__ int pool_row(const CachedParams& p, int b, int kvh, int j) {
  // j / page_size
  const int page = p.page_mul ? (int)(__umulhi((unsigned)j, p.page_mul) >> p.page_shift) : j;
  const int slot = __ldg(p.page_table + (int64_t)b * p.pages_per_seq + page);
  if (slot < 0 || slot >= p.c.pool_pages) {
    atomicOr(p.status, kStatusBadPage);
    return -1;
  }
  return (slot * p.c.hkv + kvh) * p.c.page_size + (j - page * p.c.page_size);
}

__device__ __forceinline__ float exp_scale(int e) {  // 2^e of a row; NaN for a NaN row
  return e == -128 ? __int_as_float(0x7fffffff) : __int_as_float((e + 127) << 23);
}

}  // namespace ls
