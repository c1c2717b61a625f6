// Pages of a paged cache: which sequence has which (advance, fork, compact), and
// the copying of their rows.
//
// The book of a pool is small (4 bytes a page, 4 an entry of a table), and each
// step of it depends on the whole of the one before: references fall before free
// pages are counted, and counted before they are given out.  So one cluster of
// blocks does a call in phases with cluster barriers between them, every thread
// striding over sequences, entries or pages; only what other threads wrote is
// read past the first-level cache.  Free pages are handed out by number: each
// warp counts those of its own stretch of the pool, the counts' prefix gives each
// free page its rank, and the rank its taker, so the result does not depend on
// which thread came first.
#include "ls_cluster.cuh"
#include "ls_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int32_t kShared = 1 << 30;   // need[]: its last page is others' too
constexpr int32_t kNoRoom = INT32_MIN; // need[]: the table's row ends, or its last page is no page

__device__ __forceinline__ int32_t per(int32_t n, int32_t page) { return n > 0 ? (n - 1) / page + 1 : 0; }
__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }

template <int C>
struct Team {
  uint32_t rank, warp, lane;
  int tid;        // in the cluster
  int gw;         // warp in the cluster
  static constexpr int threads = C * kThreads, warps = C * kWarps;
  __device__ Team() {
    rank = Cluster<C>::rank();
    warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    tid = (int)rank * kThreads + threadIdx.x;
    gw = (int)rank * kWarps + (int)warp;
  }
  __device__ void sync() const { Cluster<C>::sync(); }
  // Whether `flag`, a word of each block's shared memory, is set in any block.
  __device__ bool any(const int* flag) const {
    int x = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) x |= Cluster<C>::at(flag, c);
    return x != 0;
  }
  // Of each warp's count (count[kWarps] in each block): the sum before this warp, and of all.
  __device__ int2 prefix(const int* count) const {
    int before = 0, all = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int x = Cluster<C>::at(count + lane, c);
      all += x;
      if (c * kWarps + (int)lane < gw) before += x;
    }
    return make_int2(warp_sum(before), warp_sum(all));
  }
};

// Calls f(page, in) for the pages of this warp's stretch, 32 at a time (all lanes; `in`: page is in the stretch).
template <int C, typename F>
__device__ __forceinline__ void for_pages(const Team<C>& t, int32_t pages, F f) {
  const int32_t each = (per(pages, t.warps) + 31) / 32 * 32;
  const int64_t lo = (int64_t)t.gw * each, hi = lo + each < pages ? lo + each : pages;
#pragma unroll 4
  for (int64_t p = lo; p < hi; p += 32) f((int32_t)(p + t.lane), p + t.lane < hi);
}

// ---------------------------------------------------------------- advance
template <int C>
__global__ void __launch_bounds__(kThreads, 1) pages_advance_kernel(const PagesParams p) {
  __shared__ int bad, total, count[kWarps], scan[kWarps];
  const Team<C> t;
  const int32_t S = p.b.page_size, cap = p.b.pages_per_seq * S;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  auto seq = [&](int i) { return p.seqs ? p.seqs[i] : i; };
  auto grows = [&](int i) { return p.q_start ? p.q_start[i + 1] - p.q_start[i] : 0; };
  // the lists, before anything is changed
  for (int i = t.tid; i < p.n; i += t.threads) {
    const int s = seq(i);
    bool ok = s >= 0 && s < p.b.n_seqs;
    if (ok) {
      const int64_t old = p.b.kv_len[s], keep = p.drop_all ? 0 : p.keep ? p.keep[i] : old;
      ok = old >= 0 && old <= cap && keep >= 0 && keep <= old;
      if (p.q_start) {
        const int a = p.q_start[i], e = p.q_start[i + 1];
        ok = ok && a >= 0 && a <= e && e <= p.total_q && (i != 0 || a == 0) && (i != p.n - 1 || e == p.total_q);
      }
      if (p.seqs) __stcg(p.owner + s, i);
    }
    if (!ok) bad = 1;
  }
  if (p.seqs) {
    t.sync();
    for (int i = t.tid; i < p.n; i += t.threads) {
      const int s = seq(i);
      if (s >= 0 && s < p.b.n_seqs && __ldcg(p.owner + s) != i) bad = 1;
    }
  }
  t.sync();
  if (t.any(&bad)) {
    for (int64_t x = t.tid; x < p.total_q; x += t.threads) p.slots[x] = -1;
    if (p.copies)
      for (int64_t x = t.tid; x < 3 * (int64_t)p.n; x += t.threads) p.copies[x] = -1;
    if (t.tid == 0) atomicOr(p.status, kStatusBadIndex);
    t.sync();  // the others may still read this block's flag
    return;
  }
  const int ways = t.warps > p.n ? t.warps / p.n : 1, sub = t.gw % ways;
  // pages that are dropped
  for (int i = t.gw / ways; i < p.n; i += t.warps / ways) {
    const int s = seq(i);
    const int32_t old = (int32_t)p.b.kv_len[s], keep = p.drop_all ? 0 : p.keep ? (int32_t)p.keep[i] : old;
    const int32_t* row = p.b.page_table + (int64_t)s * p.b.pages_per_seq;
    for (int32_t j = per(keep, S) + sub * 32 + t.lane; j < per(old, S); j += ways * 32) {
      const int32_t page = row[j];
      bool ok = page >= 0 && page < p.b.pool_pages;
      if (ok && atomicSub(p.b.refs + page, 1) <= 0) atomicAdd(p.b.refs + page, 1), ok = false;
      if (!ok) atomicOr(p.status, kStatusBadPage);
    }
  }
  t.sync();
  // free pages, and what each sequence takes
  {
    int free = 0;
    for_pages(t, p.b.pool_pages, [&](int32_t page, bool in) { free += in && __ldcg(p.b.refs + page) == 0; });
    free = warp_sum(free);
    if (t.lane == 0) count[t.warp] = free;
  }
  if (t.rank == 0) {
    int carry = 0;
    for (int i0 = 0; i0 < p.n; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      int need = 0;
      bool shared = false, full = false;
      if (i < p.n) {
        const int s = seq(i);
        const int32_t keep = p.drop_all ? 0 : p.keep ? (int32_t)p.keep[i] : (int32_t)p.b.kv_len[s];
        const int64_t want = (int64_t)keep + grows(i);
        full = want > cap;
        if (!full && want > keep) {
          need = per((int32_t)want, S) - per(keep, S);
          if (keep % S != 0) {
            const int32_t page = p.b.page_table[(int64_t)s * p.b.pages_per_seq + keep / S];
            if (page < 0 || page >= p.b.pool_pages)
              full = true, need = 0, atomicOr(p.status, kStatusBadPage);
            else
              shared = __ldcg(p.b.refs + page) > 1, need += shared;
          }
        }
        __stcg(p.kept + i, keep);
      }
      int upto = need;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)t.lane >= o) upto += x;
      }
      if (t.lane == 31) scan[t.warp] = upto;
      __syncthreads();
      const int w = scan[t.lane];
      upto += carry + warp_sum(t.lane < t.warp ? w : 0);
      carry += warp_sum(w);
      if (i < p.n) {
        __stcg(p.begin + i, upto - need);
        __stcg(p.need + i, full ? kNoRoom : need | (shared ? kShared : 0));
      }
      __syncthreads();
    }
    if (threadIdx.x == 0) total = carry;
  }
  t.sync();
  const int wanted = Cluster<C>::at(&total, 0);
  const int2 rank = t.prefix(count);
  if (wanted > 0) {
    int at = rank.x;
    for_pages(t, p.b.pool_pages, [&](int32_t page, bool in) {
      const bool free = in && __ldcg(p.b.refs + page) == 0;
      const unsigned m = __ballot_sync(0xffffffffu, free);
      const int r = at + __popc(m & ((1u << t.lane) - 1u));
      if (free && r < wanted) __stcg(p.list + r, page);
      at += __popc(m);
    });
    t.sync();
  }
  // the new lengths, entries and slots
  for (int i = t.gw / ways; i < p.n; i += t.warps / ways) {
    const int s = seq(i);
    const int32_t word = __ldcg(p.need + i), begin = __ldcg(p.begin + i), keep = __ldcg(p.kept + i);
    const bool shared = word != kNoRoom && (word & kShared);
    const int32_t need = word == kNoRoom ? 0 : word & ~kShared;
    const bool served = word != kNoRoom && (need == 0 || (int64_t)begin + need <= rank.y);
    const int32_t grow = grows(i), have = per(keep, S), first = have - (shared ? 1 : 0);
    int32_t* row = p.b.page_table + (int64_t)s * p.b.pages_per_seq;
    const int32_t last = keep % S != 0 ? row[have - 1] : -1;
    __syncwarp();  // `last` is read before this warp writes the entry
    if (sub == 0 && t.lane == 0) {
      p.b.kv_len[s] = served ? keep + grow : keep;
      const bool copy = served && shared;
      if (copy) atomicSub(p.b.refs + last, 1);
      if (p.copies) {
        p.copies[3 * (int64_t)i] = copy ? last : -1;
        p.copies[3 * (int64_t)i + 1] = copy ? __ldcg(p.list + begin) : -1;
        p.copies[3 * (int64_t)i + 2] = copy ? keep % S : -1;
      }
      if (!served) atomicOr(p.status, kStatusNoPages);
    }
    if (served)
      for (int32_t j = sub * 32 + t.lane; j < need; j += ways * 32) {
        const int32_t page = __ldcg(p.list + begin + j);
        row[first + j] = page;
        p.b.refs[page] = 1;
      }
    if (p.q_start) {
      const int32_t t0 = p.q_start[i];
      for (int32_t x = sub * 32 + t.lane; x < grow; x += ways * 32) {
        const int32_t pos = keep + x, j = pos / S;
        const int32_t page = !served ? 0 : j >= first ? (need > 0 && j - first < need ? __ldcg(p.list + begin + j - first) : last) : last;
        p.slots[t0 + x] = served ? (int64_t)page * S + pos % S : -1;
      }
    }
  }
  t.sync();  // `count` and `total` are read by other blocks
}

// ---------------------------------------------------------------- fork
template <int C>
__global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(const PagesParams p) {
  __shared__ int bad;
  const Team<C> t;
  const int32_t S = p.b.page_size, cap = p.b.pages_per_seq * S;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  auto in = [&](int s) { return s >= 0 && s < p.b.n_seqs; };
  for (int i = t.tid; i < p.n; i += t.threads) {
    const int s = p.src[i], d = p.seqs[i];
    bool ok = in(s) && in(d);
    if (ok) {
      const int64_t len = p.b.kv_len[s], old = p.b.kv_len[d], want = p.keep ? p.keep[i] : len;
      ok = len >= 0 && len <= cap && old >= 0 && old <= cap && want >= 0 && want <= len;
      __stcg(p.owner + s, -1);
    }
    if (!ok) bad = 1;
  }
  t.sync();
  for (int i = t.tid; i < p.n; i += t.threads)
    if (in(p.seqs[i])) __stcg(p.owner + p.seqs[i], i);
  t.sync();
  for (int i = t.tid; i < p.n; i += t.threads)
    if (in(p.src[i]) && in(p.seqs[i]) && (__ldcg(p.owner + p.src[i]) != -1 || __ldcg(p.owner + p.seqs[i]) != i)) bad = 1;
  t.sync();
  const bool refused = t.any(&bad);
  const int ways = t.warps > p.n ? t.warps / p.n : 1, sub = t.gw % ways;
  if (refused) {
    if (t.tid == 0) atomicOr(p.status, kStatusBadIndex);
  } else {
    for (int i = t.gw / ways; i < p.n; i += t.warps / ways) {
      const int s = p.src[i], d = p.seqs[i];
      const int32_t had = per((int32_t)p.b.kv_len[d], S), want = per((int32_t)(p.keep ? p.keep[i] : p.b.kv_len[s]), S);
      const int32_t* from = p.b.page_table + (int64_t)s * p.b.pages_per_seq;
      int32_t* to = p.b.page_table + (int64_t)d * p.b.pages_per_seq;
      for (int32_t j = sub * 32 + t.lane; j < had || j < want; j += ways * 32) {
        bool ok = true;
        if (j < had) {
          const int32_t page = to[j];
          ok = page >= 0 && page < p.b.pool_pages;
          if (ok && atomicSub(p.b.refs + page, 1) <= 0) atomicAdd(p.b.refs + page, 1), ok = false;
        }
        if (j < want) {
          const int32_t page = from[j];
          to[j] = page;
          if (page >= 0 && page < p.b.pool_pages)
            atomicAdd(p.b.refs + page, 1);
          else
            ok = false;
        }
        if (!ok) atomicOr(p.status, kStatusBadPage);
      }
    }
  }
  t.sync();  // all lengths have been read
  if (!refused && sub == 0 && t.lane == 0)
    for (int i = t.gw / ways; i < p.n; i += t.warps / ways) p.b.kv_len[p.seqs[i]] = p.keep ? p.keep[i] : p.b.kv_len[p.src[i]];
}

// ---------------------------------------------------------------- compact
template <int C>
__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const PagesParams p) {
  __shared__ int live_of[kWarps], low_of[kWarps], high_of[kWarps];
  const Team<C> t;
  const int32_t S = p.b.page_size, pool = p.b.pool_pages;
  const bool same = p.refs_out == p.b.refs;
  auto refs = [&](int32_t page) { return __ldcg(p.b.refs + page); };
  int live = 0;
  for_pages(t, pool, [&](int32_t page, bool in) { live += in && refs(page) > 0; });
  live = warp_sum(live);
  if (t.lane == 0) live_of[t.warp] = live;
  t.sync();
  const int32_t A = t.prefix(live_of).y;  // pages in use: they end in [0, A)
  int low = 0, high = 0;
  for_pages(t, pool, [&](int32_t page, bool in) {
    const bool used = in && refs(page) > 0;
    low += in && !used && page < A;
    high += used && page >= A;
  });
  low = warp_sum(low), high = warp_sum(high);
  if (t.lane == 0) low_of[t.warp] = low, high_of[t.warp] = high;
  t.sync();
  const int2 l = t.prefix(low_of), h = t.prefix(high_of);
  const int32_t moves = h.y;
  int at_l = l.x, at_h = h.x;
  for_pages(t, pool, [&](int32_t page, bool in) {
    const bool used = in && refs(page) > 0, goes = used && page >= A, free = in && !used && page < A;
    const unsigned mh = __ballot_sync(0xffffffffu, goes), ml = __ballot_sync(0xffffffffu, free), before = (1u << t.lane) - 1u;
    if (goes) {
      const int r = at_h + __popc(mh & before);
      __stcg(p.high + r, page);
      __stcg(p.rank + page, r);
    }
    if (free) __stcg(p.list + at_l + __popc(ml & before), page);
    at_h += __popc(mh), at_l += __popc(ml);
  });
  t.sync();
  for (int64_t r = t.tid; r < pool / 2; r += t.threads) {
    const bool in = r < moves;
    const int32_t from = in ? __ldcg(p.high + r) : -1, to = in ? __ldcg(p.list + r) : -1;
    p.copies[3 * r] = from, p.copies[3 * r + 1] = to, p.copies[3 * r + 2] = in ? S : -1;
    if (in) {
      const int32_t n = refs(from);
      p.refs_out[to] = n;
      p.refs_out[from] = 0;
    }
  }
  if (!same)
    for (int32_t page = t.tid; page < pool; page += t.threads) {
      const int32_t n = refs(page);
      if (page < A ? n > 0 : n <= 0) p.refs_out[page] = page < A ? n : 0;  // the others moved, or were moved to
    }
  // the table: an entry counts where its sequence reaches it
  const int64_t pps = p.b.pages_per_seq, cells = (int64_t)p.b.n_seqs * pps;
  for (int64_t x = t.tid; x < cells; x += t.threads) {
    const int64_t s = x / pps, j = x - s * pps, n = p.b.kv_len[s];
    int32_t page = p.b.page_table[x];
    if (n > 0 && j <= (n - 1) / S) {
      if (page < 0 || page >= pool) {
        atomicOr(p.status, kStatusBadPage);
      } else if (page >= A) {
        const int32_t r = __ldcg(p.rank + page);
        if (r >= 0 && r < moves && __ldcg(p.high + r) == page)
          page = __ldcg(p.list + r);
        else
          atomicOr(p.status, kStatusBadPage);  // nothing says that the page is in use
      }
    }
    p.table_out[x] = page;
  }
  t.sync();  // the counts are read by other blocks
}

// ---------------------------------------------------------------- copies
constexpr int kCopyThreads = 256, kPiece = 16384;  // bytes of a block

// Block (x, entry): piece x % pieces of page side x / pieces (K, then V, head by head).
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const ls_kv_cache c, const int32_t* __restrict__ copies, int row_bytes,
                                                                  int pieces, int64_t n, uint32_t* status) {
  const int64_t e = (int64_t)blockIdx.z * 65535 + blockIdx.y;
  if (e >= n) return;
  const int32_t from = copies[3 * e], to = copies[3 * e + 1], rows = copies[3 * e + 2];
  if (from < 0 || to < 0) return;
  if (from >= c.pool_pages || to >= c.pool_pages || rows < 0 || rows > c.page_size) {
    if (threadIdx.x == 0 && status) atomicOr(status, kStatusBadIndex);
    return;
  }
  if (from == to) return;
  const int piece = blockIdx.x % pieces, side = blockIdx.x / pieces;
  const int head = side % c.hkv, second = side / c.hkv;
  const int64_t src = ((int64_t)from * c.hkv + head) * c.page_size, dst = ((int64_t)to * c.hkv + head) * c.page_size;  // rows
  const int64_t bytes = (int64_t)rows * row_bytes, lo = (int64_t)piece * kPiece;
  char* pool = static_cast<char*>(second ? c.v : c.k);
  const uint4* a = reinterpret_cast<const uint4*>(pool + src * row_bytes + lo);
  uint4* b = reinterpret_cast<uint4*>(pool + dst * row_bytes + lo);
  const int64_t left = (bytes - lo) / 16;  // rows are whole 16-byte pieces
  uint4 x[kPiece / 16 / kCopyThreads];
#pragma unroll
  for (int i = 0; i < kPiece / 16 / kCopyThreads; ++i)
    if (threadIdx.x + i * kCopyThreads < left) x[i] = __ldcs(a + threadIdx.x + i * kCopyThreads);
#pragma unroll
  for (int i = 0; i < kPiece / 16 / kCopyThreads; ++i)
    if (threadIdx.x + i * kCopyThreads < left) __stcs(b + threadIdx.x + i * kCopyThreads, x[i]);
  if (piece == 0 && c.format == LS_CACHE_E4M3) {
    int8_t* ex = second ? c.v_exp : c.k_exp;
    for (int i = threadIdx.x; i < rows; i += kCopyThreads) ex[dst + i] = ex[src + i];
  }
}

template <typename P>
cudaError_t launch_team(void (*one)(P), void (*eight)(P), bool wide, const P& p, cudaStream_t s) {
  LaunchScope ls(kKPages, s);
  if (!wide) {
    one<<<1, kThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(8), cfg.blockDim = dim3(kThreads), cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 8, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cfg.attrs = &at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, eight, p);
}

}  // namespace

size_t pages_scratch(const ls_page_book& b) { return 4 * (3 * (size_t)b.pool_pages + 4 * (size_t)b.n_seqs); }

cudaError_t launch_pages_advance(const PagesParams& p, cudaStream_t s) {
  return launch_team(pages_advance_kernel<1>, pages_advance_kernel<8>, p.b.pool_pages > 4096 || p.n > 64, p, s);
}
cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t s) {
  return launch_team(pages_fork_kernel<1>, pages_fork_kernel<8>, (int64_t)p.n * p.b.pages_per_seq > 4096, p, s);
}
cudaError_t launch_pages_compact(const PagesParams& p, cudaStream_t s) {
  return launch_team(pages_compact_kernel<1>, pages_compact_kernel<8>,
                     p.b.pool_pages + (int64_t)p.b.n_seqs * p.b.pages_per_seq > 4096, p, s);
}

cudaError_t launch_page_copy(const ls_kv_cache& c, const int32_t* copies, int64_t n, uint32_t* status, cudaStream_t s) {
  const int row = c.head_dim * (c.format == LS_CACHE_F32 ? 4 : c.format == LS_CACHE_BF16 ? 2 : 1);
  const int64_t pieces = ((int64_t)c.page_size * row + kPiece - 1) / kPiece, x = pieces * 2 * c.hkv;
  if (x > INT32_MAX || n > (int64_t)65535 * 65535) return cudaErrorInvalidConfiguration;
  LaunchScope ls(kKPageCopy, s);
  const dim3 grid((unsigned)x, (unsigned)(n < 65535 ? n : 65535), (unsigned)((n + 65534) / 65535));
  page_copy_kernel<<<grid, kCopyThreads, 0, s>>>(c, copies, row, (int)pieces, n, status);
  return cudaGetLastError();
}

}  // namespace ls
