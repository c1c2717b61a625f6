// Pages of a paged cache: which sequence has which (advance, fork, compact), and
// the copying of their rows.
//
// The book of a pool is small (4 bytes a page, 4 an entry of a table), and each
// step of it depends on the whole of the one before: references fall before free
// pages are counted, and counted before they are given out.  What a call takes is
// latency, so one cluster of blocks does all of it, with as few cluster barriers as
// that order needs: each block looks through the whole lists by itself (a thread a
// sequence) and keeps what it will need of them in shared memory; entries and pages
// are then dealt out to the cluster's warps.  Free pages are handed out by number:
// each warp keeps a bit for each page of its own stretch of the pool, the prefix of
// the warps' counts gives each free page its rank, and the rank its taker, so the
// result does not depend on which thread came first.  The kernels let the one after
// them start early, which waits for their end before it reads anything.
//   Measured, one call after another in a graph: a step of 8 sequences 4.3 us (6.2 as
// calls), of 384 over 131,000 pages 9.8; 16 members forked from 100,003 tokens, their
// first slots and the copies of their last page 13.0 us; 3001 pages compacted in 11 us
// before the copies.  One block alone is faster for few (8 of 10 us for the first of
// these when it was tried) and takes 97 us for the second.
#include "ls_cluster.cuh"
#include "ls_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int32_t kShared = 1 << 30;   // need[]: its last page is others' too
constexpr int32_t kNoRoom = INT32_MIN; // need[]: the table's row ends, or its last page is no page

constexpr int kListed = 1664;  // sequences of a call that are kept in shared memory
constexpr int kListArrays = 7;

__device__ __forceinline__ int32_t per(int32_t n, int32_t each) { return n > 0 ? (n - 1) / each + 1 : 0; }
// A book's page size, to divide by.
struct Pages {
  int32_t S;
  uint32_t mul, shift;
  __device__ explicit Pages(const PagesParams& p) : S(p.b.page_size), mul(p.page_mul), shift(p.page_shift) {}
  __device__ int32_t page(int32_t pos) const { return mul ? (int32_t)(__umulhi((uint32_t)pos, mul) >> shift) : pos; }
  __device__ int32_t row(int32_t pos) const { return pos - page(pos) * S; }
  __device__ int32_t of(int32_t n) const { return n > 0 ? page(n - 1) + 1 : 0; }  // that n tokens take
};
__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ void start() {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

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

// Which pages of a warp's stretch of the pool have a reference: page lo + 32 x + lane is
// bit x of the lane's word, where the stretch has at most 1024 pages; otherwise it is
// looked up again (as nothing changes the references meanwhile, with the same answer).
template <int C>
struct Stretch {
  const int32_t* refs;
  int64_t lo, hi;
  int steps;
  uint32_t used, unused;
  bool kept;
  __device__ Stretch(const Team<C>& t, const int32_t* r, int32_t pages) : refs(r), used(0), unused(0) {
    const int64_t each = ((int64_t)per(pages, t.warps) + 31) / 32 * 32;
    lo = t.gw * each + t.lane, hi = t.gw * each + each < pages ? t.gw * each + each : pages;
    steps = (int)(each / 32), kept = steps <= 32;
    if (kept)
      for (int x0 = 0; x0 < steps; x0 += 8) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x0 + x < steps && in(x0 + x)) {
            const bool is = __ldcg(refs + page(x0 + x)) > 0;
            used |= (is ? 1u : 0u) << (x0 + x), unused |= (is ? 0u : 1u) << (x0 + x);
          }
      }
  }
  __device__ int64_t page(int x) const { return lo + 32 * x; }
  __device__ bool in(int x) const { return page(x) < hi; }
  __device__ bool taken(int x) const { return kept ? used >> x & 1 : in(x) && __ldcg(refs + page(x)) > 0; }
  __device__ bool free(int x) const { return kept ? unused >> x & 1 : in(x) && __ldcg(refs + page(x)) <= 0; }
  // This lane's pages that are free, that are taken.
  __device__ int count_free() const {
    int n = __popc(unused);
    if (!kept)
      for (int x = 0; x < steps; ++x) n += free(x);
    return n;
  }
  __device__ int count_taken() const {
    int n = __popc(used);
    if (!kept)
      for (int x = 0; x < steps; ++x) n += taken(x);
    return n;
  }
};

// What a call says of its sequences, and what is worked out of it.
struct Lists {
  int32_t *seq, *keep, *old, *need, *begin, *last, *grow;
};
// In shared memory where they fit, else each block in its own part of the workspace.
__device__ __forceinline__ Lists lists(const PagesParams& p, int32_t* shared, uint32_t rank) {
  int32_t* w = p.n <= kListed ? shared : p.lists + (int64_t)rank * kListArrays * p.b.n_seqs;
  const int64_t n = p.n <= kListed ? kListed : p.b.n_seqs;
  return Lists{w, w + n, w + 2 * n, w + 3 * n, w + 4 * n, w + 5 * n, w + 6 * n};
}

// ---------------------------------------------------------------- advance
template <int C>
__global__ void __launch_bounds__(kThreads, 1) pages_advance_kernel(const PagesParams p) {
  __shared__ int count[kWarps], scan[kWarps];
  __shared__ int32_t listed[kListArrays * kListed];
  start();
  const Team<C> t;
  const Lists l = lists(p, listed, t.rank);
  const Pages pages(p);
  const int32_t S = pages.S, cap = p.b.pages_per_seq * S;
  int32_t* owner = p.owner + (int64_t)t.rank * p.b.n_seqs;
  // the lists, before anything is changed
  bool bad = false;
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int s = p.seqs ? p.seqs[i] : i;
    bool ok = s >= 0 && s < p.b.n_seqs;
    int64_t old = 0, keep = 0;
    int32_t grow = 0;
    if (p.q_start) {
      const int a = p.q_start[i], e = p.q_start[i + 1];
      grow = e - a;
      ok = ok && a >= 0 && a <= e && e <= p.total_q && (i != 0 || a == 0) && (i != p.n - 1 || e == p.total_q);
    }
    if (s >= 0 && s < p.b.n_seqs) {
      old = p.b.kv_len[s], keep = p.drop_all ? 0 : p.keep ? p.keep[i] : old;
      ok = ok && old >= 0 && old <= cap && keep >= 0 && keep <= old;
      if (p.seqs) owner[s] = i;
    }
    l.seq[i] = s, l.old[i] = (int32_t)old, l.keep[i] = (int32_t)keep, l.grow[i] = grow;
    bad |= !ok;
  }
  if (p.seqs) {
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
      const int s = l.seq[i];
      bad |= s >= 0 && s < p.b.n_seqs && owner[s] != i;
    }
  }
  if (__syncthreads_or(bad)) {  // the same in every block
    for (int64_t x = t.tid; x < p.total_q; x += t.threads) p.slots[x] = -1;
    if (p.copies)
      for (int64_t x = t.tid; x < 3 * (int64_t)p.n; x += t.threads) p.copies[x] = -1;
    if (t.tid == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  // The page that a sequence goes on in, for the first of this thread's sequences: nothing
  // waits for it before the pages that are dropped are done with.
  auto last_of = [&](int i) {
    const int32_t keep = l.keep[i], grow = l.grow[i];
    return grow > 0 && pages.row(keep) != 0 && (int64_t)keep + grow <= cap
               ? p.b.page_table[(int64_t)l.seq[i] * p.b.pages_per_seq + pages.page(keep)]
               : -1;
  };
  int32_t last = (int)threadIdx.x < p.n ? last_of(threadIdx.x) : -1;
  const int width = 1 << p.share_shift, sub = t.tid & (width - 1), groups = t.threads >> p.share_shift;
  // pages that are dropped
  for (int i = t.tid >> p.share_shift; i < p.n; i += groups) {
    const int32_t* row = p.b.page_table + (int64_t)l.seq[i] * p.b.pages_per_seq;
    for (int32_t j = pages.of(l.keep[i]) + sub, end = pages.of(l.old[i]); j < end; j += width) {
      const int32_t page = row[j];
      bool ok = page >= 0 && page < p.b.pool_pages;
      if (ok && atomicSub(p.b.refs + page, 1) <= 0) atomicAdd(p.b.refs + page, 1), ok = false;
      if (!ok) atomicOr(p.status, kStatusBadPage);
    }
  }
  t.sync();
  // free pages, and what each sequence takes
  auto others = [&](int32_t page) { return page >= 0 && page < p.b.pool_pages ? __ldcg(p.b.refs + page) : 0; };
  int32_t names = others(last);
  const Stretch<C> stretch(t, p.b.refs, p.b.pool_pages);
  int carry = 0;
  for (int i0 = 0; i0 < p.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    bool shared = false, full = false;
    if (i < p.n) {
      if (i0) last = last_of(i), names = others(last);
      const int32_t keep = l.keep[i];
      const int64_t want = (int64_t)keep + l.grow[i];
      full = want > cap;
      if (!full && want > keep) {
        need = pages.of((int32_t)want) - pages.of(keep);
        if (pages.row(keep) != 0) {
          if (last < 0 || last >= p.b.pool_pages)
            full = true, need = 0, atomicOr(p.status, kStatusBadPage);
          else
            shared = names > 1, need += shared;
        }
      }
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
      l.begin[i] = upto - need;
      l.need[i] = full ? kNoRoom : need | (shared ? kShared : 0);
      l.last[i] = last;
    }
    __syncthreads();
  }
  const int wanted = carry;
  const int free = warp_sum(stretch.count_free());
  if (t.lane == 0) count[t.warp] = free;
  t.sync();
  const int2 rank = t.prefix(count);
  if (wanted > 0) {
    int at = rank.x;
    for (int x = 0; x < stretch.steps && at < wanted; ++x) {
      const bool f = stretch.free(x);
      const unsigned m = __ballot_sync(0xffffffffu, f);
      const int r = at + __popc(m & ((1u << t.lane) - 1u));
      if (f && r < wanted) __stcg(p.list + r, (int32_t)stretch.page(x));
      at += __popc(m);
    }
  }
  t.sync();  // the list is there, and no block reads another's counts any more
  // the new lengths, entries and slots
  for (int i = t.tid >> p.share_shift; i < p.n; i += groups) {
    const int s = l.seq[i];
    const int32_t word = l.need[i], begin = l.begin[i], keep = l.keep[i], page0 = l.last[i];
    const bool shared = word != kNoRoom && (word & kShared);
    const int32_t need = word == kNoRoom ? 0 : word & ~kShared;
    const bool served = word != kNoRoom && (need == 0 || (int64_t)begin + need <= rank.y);
    const int32_t grow = l.grow[i], first = pages.of(keep) - (shared ? 1 : 0);
    int32_t* row = p.b.page_table + (int64_t)s * p.b.pages_per_seq;
    if (sub == 0) {
      p.b.kv_len[s] = served ? keep + grow : keep;
      const bool copy = served && shared;
      if (copy) atomicSub(p.b.refs + page0, 1);
      if (p.copies) {
        p.copies[3 * (int64_t)i] = copy ? page0 : -1;
        p.copies[3 * (int64_t)i + 1] = copy ? __ldcg(p.list + begin) : -1;
        p.copies[3 * (int64_t)i + 2] = copy ? pages.row(keep) : -1;
      }
      if (!served) atomicOr(p.status, kStatusNoPages);
    }
    if (served)
      for (int32_t j = sub; j < need; j += width) {
        const int32_t page = __ldcg(p.list + begin + j);
        row[first + j] = page;
        p.b.refs[page] = 1;
      }
    if (p.q_start) {
      const int32_t t0 = p.q_start[i];
      for (int32_t x = sub; x < grow; x += width) {
        const int32_t pos = keep + x, j = pages.page(pos);
        const int32_t page = !served ? 0 : j >= first ? __ldcg(p.list + begin + j - first) : page0;
        p.slots[t0 + x] = served ? (int64_t)page * S + (pos - j * S) : -1;
      }
    }
  }
}

// ---------------------------------------------------------------- fork
template <int C>
__global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(const PagesParams p) {
  __shared__ int32_t listed[kListArrays * kListed];
  start();
  const Team<C> t;
  const Lists l = lists(p, listed, t.rank);  // seq: destinations, begin: sources, keep: new lengths
  const Pages pages(p);
  const int32_t cap = p.b.pages_per_seq * pages.S;
  int32_t* owner = p.owner + (int64_t)t.rank * p.b.n_seqs;
  auto in = [&](int s) { return s >= 0 && s < p.b.n_seqs; };
  bool bad = false;
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int s = p.src[i], d = p.seqs[i];
    bool ok = in(s) && in(d);
    if (ok) {
      const int64_t len = p.b.kv_len[s], old = p.b.kv_len[d], want = p.keep ? p.keep[i] : len;
      ok = len >= 0 && len <= cap && old >= 0 && old <= cap && want >= 0 && want <= len;
      owner[s] = -1;
      l.seq[i] = d, l.begin[i] = s, l.old[i] = (int32_t)old, l.keep[i] = (int32_t)want;
    }
    bad |= !ok;
  }
  if (!__syncthreads_or(bad)) {  // the same in every block
    for (int i = threadIdx.x; i < p.n; i += kThreads) owner[l.seq[i]] = i;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kThreads) bad |= owner[l.begin[i]] != -1 || owner[l.seq[i]] != i;
  } else {
    bad = true;
  }
  if (__syncthreads_or(bad)) {
    if (t.tid == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const int width = 1 << p.share_shift, sub = t.tid & (width - 1);
  for (int i = t.tid >> p.share_shift; i < p.n; i += t.threads >> p.share_shift) {
    const int32_t had = pages.of(l.old[i]), want = pages.of(l.keep[i]);
    const int32_t* from = p.b.page_table + (int64_t)l.begin[i] * p.b.pages_per_seq;
    int32_t* to = p.b.page_table + (int64_t)l.seq[i] * p.b.pages_per_seq;
#pragma unroll 4
    for (int32_t j = sub; j < max(had, want); j += width) {
      bool ok = true;
      if (j < want) {
        const int32_t page = from[j], mine = j < had ? to[j] : -1;
        to[j] = page;
        if (page >= 0 && page < p.b.pool_pages)
          atomicAdd(p.b.refs + page, 1);
        else
          ok = false;
        if (j < had) {
          const bool real = mine >= 0 && mine < p.b.pool_pages;
          if (real && atomicSub(p.b.refs + mine, 1) <= 0) atomicAdd(p.b.refs + mine, 1), ok = false;
          ok = ok && real;
        }
      } else {
        const int32_t mine = to[j];
        ok = mine >= 0 && mine < p.b.pool_pages;
        if (ok && atomicSub(p.b.refs + mine, 1) <= 0) atomicAdd(p.b.refs + mine, 1), ok = false;
      }
      if (!ok) atomicOr(p.status, kStatusBadPage);
    }
  }
  t.sync();  // every block has read the lengths
  for (int i = t.tid; i < p.n; i += t.threads) p.b.kv_len[l.seq[i]] = l.keep[i];
}

// ---------------------------------------------------------------- compact
template <int C>
__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const PagesParams p) {
  __shared__ int live_of[kWarps], low_of[kWarps], high_of[kWarps];
  start();
  const Team<C> t;
  const int32_t S = p.b.page_size, pool = p.b.pool_pages;
  const bool same = p.refs_out == p.b.refs;
  const Stretch<C> stretch(t, p.b.refs, pool);
  const int live = warp_sum(stretch.count_taken());
  if (t.lane == 0) live_of[t.warp] = live;
  t.sync();
  const int32_t A = t.prefix(live_of).y;  // pages in use: they end in [0, A)
  auto goes = [&](int x) { return stretch.taken(x) && stretch.page(x) >= A; };
  auto gap = [&](int x) { return stretch.free(x) && stretch.page(x) < A; };
  int low = 0, high = 0;
  for (int x = 0; x < stretch.steps; ++x) low += gap(x), high += goes(x);
  low = warp_sum(low), high = warp_sum(high);
  if (t.lane == 0) low_of[t.warp] = low, high_of[t.warp] = high;
  t.sync();
  const int2 lo = t.prefix(low_of), hi = t.prefix(high_of);
  const int32_t moves = hi.y;
  int at_l = lo.x, at_h = hi.x;
  for (int x = 0; x < stretch.steps; ++x) {
    const bool g = goes(x), f = gap(x);
    const int32_t page = (int32_t)stretch.page(x);
    const unsigned mh = __ballot_sync(0xffffffffu, g), ml = __ballot_sync(0xffffffffu, f), before = (1u << t.lane) - 1u;
    if (g) {
      const int r = at_h + __popc(mh & before);
      __stcg(p.high + r, page);
      __stcg(p.rank + page, r);
    }
    if (f) __stcg(p.list + at_l + __popc(ml & before), page);
    at_h += __popc(mh), at_l += __popc(ml);
  }
  t.sync();
  for (int64_t r = t.tid; r < pool / 2; r += t.threads) {
    const bool in = r < moves;
    const int32_t from = in ? __ldcg(p.high + r) : -1, to = in ? __ldcg(p.list + r) : -1;
    p.copies[3 * r] = from, p.copies[3 * r + 1] = to, p.copies[3 * r + 2] = in ? S : -1;
    if (in) {
      const int32_t n = __ldcg(p.b.refs + from);
      p.refs_out[to] = n;
      p.refs_out[from] = 0;
    }
  }
  if (!same)
    for (int32_t page = t.tid; page < pool; page += t.threads) {
      const int32_t n = __ldcg(p.b.refs + page);
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
}

// ---------------------------------------------------------------- copies
constexpr int kCopyThreads = 256, kPiece = 16384;  // bytes of a block

// Bytes only: 588 MB read and written in 98 us (6.0 TB/s, 88 % of a copy's rate), 560
// pages of 1500 entries.  Pieces of 16 KB, dealt out in turn: piece x % pieces of side x / pieces (K's heads,
// then V's) of an entry's page.  All of a block's piece is loaded before its first
// store, eight blocks an SM.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const ls_kv_cache c, const int32_t* copies, int row_bytes,
                                                                 int pieces, int64_t n, uint32_t* status) {
  start();
  const int each = pieces * 2 * c.hkv;
  int64_t e = blockIdx.x / each;
  int x = (int)(blockIdx.x - e * each);
  const int step = (int)(gridDim.x % (unsigned)each);
  const int64_t steps = gridDim.x / (unsigned)each;
  for (; e < n; e += steps, x += step) {
    if (x >= each) x -= each, ++e;
    if (e >= n) return;
    const int32_t from = copies[3 * e], to = copies[3 * e + 1], rows = copies[3 * e + 2];
    if (from < 0 || to < 0 || from == to) continue;
    if (from >= c.pool_pages || to >= c.pool_pages || rows < 0 || rows > c.page_size) {
      if (threadIdx.x == 0 && x == 0 && status) atomicOr(status, kStatusBadIndex);
      continue;
    }
    const int side = x / pieces, piece = x - side * pieces;
    const bool second = side >= c.hkv;
    const int head = second ? side - c.hkv : side;
    const int64_t src = ((int64_t)from * c.hkv + head) * c.page_size, dst = ((int64_t)to * c.hkv + head) * c.page_size;  // rows
    const int64_t lo = (int64_t)piece * kPiece;
    char* pool = static_cast<char*>(second ? c.v : c.k);
    const uint4* a = reinterpret_cast<const uint4*>(pool + src * row_bytes + lo);
    uint4* b = reinterpret_cast<uint4*>(pool + dst * row_bytes + lo);
    const int64_t left = ((int64_t)rows * row_bytes - lo) / 16;  // rows are whole 16-byte pieces
    uint4 w[kPiece / 16 / kCopyThreads];
#pragma unroll
    for (int i = 0; i < kPiece / 16 / kCopyThreads; ++i)
      if (threadIdx.x + i * kCopyThreads < left) w[i] = __ldcs(a + threadIdx.x + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kPiece / 16 / kCopyThreads; ++i)
      if (threadIdx.x + i * kCopyThreads < left) __stcs(b + threadIdx.x + i * kCopyThreads, w[i]);
    if (piece == 0 && c.format == LS_CACHE_E4M3) {
      int8_t* ex = second ? c.v_exp : c.k_exp;
      for (int i = threadIdx.x; i < rows; i += kCopyThreads) ex[dst + i] = ex[src + i];
    }
  }
}

// Launches a kernel that begins with start(), as a cluster of `blocks` blocks, or not in clusters (0).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int blocks, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = blocks, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = blocks ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
cudaError_t launch_team(void (*one)(PagesParams), void (*eight)(PagesParams), bool wide, PagesParams p, cudaStream_t s) {
  // Threads that share one of n sequences: a power of two, eight or more.
  const int threads = (wide ? 8 : 1) * kThreads;
  p.share_shift = 3;
  while ((2 << p.share_shift) <= threads && ((int64_t)p.n << (p.share_shift + 1)) <= threads) ++p.share_shift;
  LaunchScope ls(kKPages, s);
  return wide ? launch_early(eight, dim3(8), kThreads, 8, s, p) : launch_early(one, dim3(1), kThreads, 0, s, p);
}

}  // namespace

size_t pages_scratch(const ls_page_book& b) {
  return 4 * (3 * (size_t)b.pool_pages + 8 * (size_t)b.n_seqs * (b.n_seqs > kListed ? 1 + kListArrays : 1));
}

// One block or eight, measured in a graph.  A step of three tokens a sequence (one block / eight, us): 64 sequences over
// 8192 pages 4.4 / 6.6, over 40,960 6.4 / 6.8, over 65,536 7.6 / 6.8; 384 over 8192 6.4 / 6.9, 512 7.3 / 6.7.  So a step
// that drops little goes on being faster on one block up to some 35,000 pages or 400 sequences; but a call does not say
// how many entries it drops: a release of 4096 takes 9.6 / 9.5 with the fork before it, of 8192 12.7 / 9.6.  The limits
// stand where all pages of the pool, each named once, may go.  (Entries of pages that many share and slots are not looked
// at: 64 x 4000 of the first take 197 / 35, 65,536 of the second for one sequence 22.9 / 9.4.)
cudaError_t launch_pages_advance(const PagesParams& p, cudaStream_t s) {
  return launch_team(pages_advance_kernel<1>, pages_advance_kernel<8>, p.b.pool_pages > 4096 || p.n > 64, p, s);
}
// By the entries that may be copied: 1024 take 2.8 to 3.1 us on one block and 3.1 to 3.3 on eight, 1200 to 2000 3.5 to 3.9
// and 3.1 to 3.5, 4096 4.8 to 5.1 and 3.3 to 3.6 (1 to 64 sequences).
cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t s) {
  return launch_team(pages_fork_kernel<1>, pages_fork_kernel<8>, (int64_t)p.n * p.b.pages_per_seq > 1024, p, s);
}
// By pages and entries together: 6144 take 6.4 us on one block and 8.1 on eight, 8192 7.6 and 7.8, 16,384 12.6 and 8.3.
cudaError_t launch_pages_compact(const PagesParams& p, cudaStream_t s) {
  return launch_team(pages_compact_kernel<1>, pages_compact_kernel<8>,
                     p.b.pool_pages + (int64_t)p.b.n_seqs * p.b.pages_per_seq > 8192, p, s);
}

cudaError_t launch_page_copy(const ls_kv_cache& c, const int32_t* copies, int64_t n, uint32_t* status, cudaStream_t s) {
  const int row = c.head_dim * (c.format == LS_CACHE_F32 ? 4 : c.format == LS_CACHE_BF16 ? 2 : 1);
  const int64_t pieces = ((int64_t)c.page_size * row + kPiece - 1) / kPiece, x = pieces * 2 * c.hkv;
  if (x > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  const int64_t most = 8 * device_sms();
  LaunchScope ls(kKPageCopy, s);
  return launch_early(page_copy_kernel, dim3((unsigned)(x * n < most ? x * n : most)), kCopyThreads, 0, s, c, copies, row, (int)pieces, n,
                      status);
}

}  // namespace ls
