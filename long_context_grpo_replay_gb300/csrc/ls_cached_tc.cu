// Tensor-core (tcgen05) attention of a chunk of new tokens over a paged cache,
// bf16 or e4m3, head dim 64, 128 or 256.
//
// A CTA has 128 query rows of one (sequence, KV head) -- tokens x the group's
// heads -- and one part of the keys, 128 keys at a time: S = Q K^T into one of
// two tensor-memory buffers, the softmax of a row by two threads, P back into
// S's columns as the tensor-memory operand of O += P V.  With 24/4 heads and
// d = 256, 128 rows do 256 flop for a cached e4m3 byte, about the device's
// ratio, so one tile serves both ends: many tokens are bound by the products,
// few (a group's members over their shared prompt) by the memory stream.
//
// From 129 rows on (d 128 and 256) a pair of CTAs has 256 rows: each fills half of
// every K tile's keys and half of every V tile's columns, and the first issues
// the products of both (cta_group::2).
//
// K and V tiles are chunks of [128 keys x 128 columns] (a pair's CTA: [64 keys x d]
// of K, [128 keys x d/2] of V) in a ring of four to six slots in shared memory, in
// the order of use K0 K1 V0 K2 V1 ...  Two groups of four warps fill them in turn: bf16 rows by asynchronous copies, e4m3 rows through
// registers, as f16 (exact: e4m3 is a subset).  Rows are found per key, so any
// page size works; a missing key's row is zeros.
//
// A key's scale multiplies its scores; a pair, whose softmax is what there is
// least of, folds it into the key's f16 values instead, relative to the tile's
// largest, where no key of the tile lies more than 15 binades below it: codes down
// to 2^-9 times 2^-15 are f16 numbers, so the fold is exact.  Value scales stay out of the product, whose
// small rows may be the ones that count: y = x + ev (base 2) is the score and the
// exponent of the value row, w = 2^(y - m) the weight that multiplies codes.
// Exponents are counted from the largest so far, B (of the part's tiles up to this
// one): a tile's share of the softmax's sum is sum w 2^(B - ev) = sum 2^(x - (m - B)),
// added in float32 with its reference m - B beside it, so that neither the sum nor
// the weights leave float32's range at either end of the scales.  For that ev - B
// is held at -80 at least: a value row 2^80 times smaller than the largest so far
// counts as 2^-80 of it.  Weights are f16, held 2^11 times their value
// and at most 2^15: 11 bits down to 2^-25 of the largest, so a sum of many small
// weights beside a large one is not lost.  bf16: P in bf16, as in the replay
// kernels.  Each row's maximum only moves when exceeded by 2^4
// (e4m3) or 2^8 (bf16), so that O is rarely rescaled.
//
// Warp roles (640 threads): 0 and 2 find the keys' rows, scales and presence;
// 1 issues the products; 2 also owns tensor memory; 4-11 fill chunks, 12-19
// softmax.  The roles' loops are kept short (one copy of each, waits of six
// instructions): together they have to stay in the instruction cache.  With
// unrolled loops and inlined timers a tile of e4m3 keys took 11,500 cycles,
// most of them the issuing thread's misses (61 % hits).
//
// Measured (24/4 heads, d 256): 2048 tokens over 32,768 e4m3 keys 1.33 ms = 1.2
// PFLOP/s (tensor pipe 60 % busy, issue slots 64 %), 1.39 where no tile is folded, 2.3
// where every value row is zeros; in bf16 1.23 ms.  8 tokens over 262,144 keys 154 us
// = 3.5 TB/s (bound by filling the f16 tiles), in bf16 183 us = 5.9 TB/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "ls_cached.cuh"
#include "ls_internal.h"
#include "ls_tc.cuh"

namespace ls {
namespace {
using namespace tc;

constexpr int kBM = 128, kBN = 128, kThreads = 640;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBar = 8;  // barriers per ring (more than chunks), and tiles of key tables
constexpr int kValueSpan = 80;  // binades below the largest value scale that are told apart

// PAIR: two CTAs (cta_group::2) share a tile of 256 rows; each has half of
// every K tile's keys and half of every V tile's columns.
template <int D, bool PAIR>
struct TcShape {
  static constexpr int CW = PAIR || D < 128 ? D : 128;  // columns of a chunk (of both CTAs' for V)
  static constexpr int NCH = D / CW;                    // chunks of a K or V tile
  static constexpr int NC = PAIR ? (D == 256 ? 4 : 6) : D == 256 ? 4 : 5;  // chunks of the ring
  static constexpr uint32_t kBoxV = kBN * 128;          // [128 keys x 64 columns] of 16-bit values
  static constexpr uint32_t kBoxK = PAIR ? kBoxV / 2 : kBoxV;
  static constexpr uint32_t kChunk = kBN * CW * (PAIR ? 1 : 2);
  static constexpr uint32_t kQ = kBM * D * 2;
  static constexpr uint32_t kSmem = kQ + NC * kChunk + 1024;
  static_assert(!PAIR || D >= 128, "half of V's columns is at least a box");
  static_assert(kSmem + 20480 <= 227 * 1024, "shared memory, with 20 KB of tables");
  static_assert(NC < kBar, "a chunk's barriers are free before its slot is");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two pairs of e4m3 codes as two f16 pairs, times an f16 pair where SCALE.
template <bool SCALE>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t scale, uint32_t& lo, uint32_t& hi) {
  if constexpr (!SCALE) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    return;
  }
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t"
      "mul.rn.f16x2 %0, %0, %3;\n\tmul.rn.f16x2 %1, %1, %3;\n\t}"
      : "=&r"(lo), "=&r"(hi)
      : "r"(w), "r"(scale));
}
// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives on the barrier at this address in the pair's first CTA.  What it
// announces is in tensor memory (behind tcgen05.fence::before_thread_sync) or
// in this CTA's shared memory behind each writer's fence.proxy.async; no data
// of other kinds pass, so the arrival needs no fence of the cluster's scope,
// which cost 1,200 cycles a tile.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
      : "memory");
}
// mbar_wait_short for a barrier that the other CTA arrives on too.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 131072;\n"
      "W_%=:\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "sub.u32 n, n, 1;\n\tsetp.ne.and.u32 q, n, 0, !p;\n\t@q bra W_%=;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool PAIR>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_ss(d, a, b, idesc, acc);
}
template <bool PAIR>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_ts(d, a, b, idesc, acc);
}
// Arrives once the products so far are done: in a pair, in both CTAs.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}

constexpr int log2_of(int x) { return x <= 1 ? 0 : 1 + log2_of(x / 2); }

// Position of K_j / V_j in the order of use, and what stands at position u.
__device__ __forceinline__ int unit_of_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int unit_of_v(int j, int n) { return j < n - 1 ? 2 * j + 2 : 2 * n - 1; }
__device__ __forceinline__ void unit_at(int u, int n, int& j, bool& is_v) {
  if (u == 0) {
    j = 0, is_v = false;
  } else if (u & 1) {
    j = (u + 1) / 2;
    is_v = j >= n;
    if (is_v) j = n - 1;
  } else {
    j = (u - 2) / 2, is_v = true;
  }
}

template <int D, bool E4, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) cached_tc_kernel(const CachedParams p) {
  using L = TcShape<D, PAIR>;
  constexpr int kCtas = PAIR ? 2 : 1;
  constexpr bool FOLD = PAIR;
  constexpr float kOff = E4 ? 11.f : 0.f;
  constexpr float kSlack = E4 ? 4.f : 8.f;
  // registers: 96 a thread at launch, 61,440 in all; 64 + 2 x 72 + 2 x 136 per
  // group of 128 threads make all of them
  constexpr int kRegsControl = 64, kRegsFill = 72, kRegsSoftmax = 136;
  static_assert(128 * (kRegsControl + 2 * kRegsFill + 2 * kRegsSoftmax) <= kThreads * 96, "register split");
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_q, bar_back, bar_full[kBar], bar_done[kBar], bar_rows[kBar], bar_tile[kBar], bar_s[2], bar_p[2], bar_o,
      bar_last, bar_pair[4], bar_drain;
  __shared__ uint32_t tmem_base_s;
  __shared__ int row_s[kBar][kBN];
  // a key's scale: folded: 2^ek over the tile's largest, twice in f16; else the float32
  __shared__ __align__(16) uint32_t kh_s[E4 ? kBar : 1][kBN];
  __shared__ float kmax_s[kBar];                 // FOLD: 2^(the tile's largest ek), 0 for a tile that is not folded
  __shared__ int base_s[kBar];                   // the largest ev of the tiles so far
  __shared__ __align__(16) float ev_s[E4 ? kBar : 1][kBN], vi_s[E4 ? kBar : 1][kBN];
  __shared__ uint32_t there_s[kBar][4];
  __shared__ float top_s[2][2][kBM], back_s[kBM];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sQ = (smem_u32(smem_raw) + 1023u) & ~1023u, sRing = sQ + L::kQ;
  const int b = blockIdx.z, kvh = blockIdx.y;
  // the kernel that joins the parts may be launched; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int part = (int)(blockIdx.x / kCtas) % p.ns, tile = (int)(blockIdx.x / kCtas) / p.ns;
  const Seq s = load_seq(p, b, tid == 0 && kvh == 0 && blockIdx.x == 0);
  const int nrows = s.n * p.gq, t0 = tile * kBM * kCtas, t1 = t0 + kBM * kCtas < nrows ? t0 + kBM * kCtas : nrows;
  if (t0 >= nrows) return;  // both CTAs of a pair
  // this CTA's rows (a pair's second may have none, and then only fills its share)
  const int r0 = t0 + rank * kBM, r1 = r0 + kBM < nrows ? r0 + kBM : nrows;
  int kb, ke;
  part_range(p, s, part, (t1 - 1) / p.gq, kb, ke);
  const int ntiles = ke > kb ? (ke - kb + kBN - 1) / kBN : 0;
  const int nchunks = 2 * ntiles * L::NCH;

  if (tid == 0) {
    // what the products wait for is counted in the pair's first CTA
    mbar_init(smem_u32(&bar_q), 8 * kCtas);
    mbar_init(smem_u32(&bar_back), 8);
    for (int i = 0; i < kBar; ++i) {
      mbar_init(smem_u32(&bar_full[i]), 4 * kCtas);
      mbar_init(smem_u32(&bar_done[i]), 1);
      mbar_init(smem_u32(&bar_rows[i]), 1);
      mbar_init(smem_u32(&bar_tile[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_p[i]), 8 * kCtas);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bar_pair[i]), 64);
    mbar_init(smem_u32(&bar_o), 1);
    mbar_init(smem_u32(&bar_last), 1);
    mbar_init(smem_u32(&bar_drain), 1);
    fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base_s)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(smem_u32(&tmem_base_s), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tbase = tmem_base_s;
  const uint32_t tS = tbase + 256;
  // where a role's wait gave up; it then leaves, and the others' waits end likewise
  int gave_up = 0;
  auto arrive = [&](uint64_t& bar) {
    if constexpr (PAIR)
      arrive_first(smem_u32(&bar));
    else
      mbar_arrive(smem_u32(&bar));
  };
  auto wait = [&](uint64_t& bar, int parity, int line) -> bool {  // whole warps
    if (mbar_wait_short_warp(smem_u32(&bar), parity)) return true;
    gave_up = line;
    return false;
  };

  if (warp < 4) {
    fewer_registers<kRegsControl>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- key tables
      // two warps, every other tile each: a tile takes two loads that depend
      // on one another (page id, scales), about as long as its products
      const int32_t* pages = p.page_table + (int64_t)b * p.pages_per_seq;
      const uint32_t pool_pages = (uint32_t)p.c.pool_pages;  // a pool's rows number below 2^31
      const uint32_t head_row = (uint32_t)kvh * p.c.page_size, page_rows = (uint32_t)p.c.hkv * p.c.page_size;
#pragma unroll 1
      for (int j = warp >> 1; j < ntiles; j += 2) {
        const int sl = j % kBar, key0 = kb + j * kBN + lane;
        int row[4], ek[4], ev[4];
        bool bad = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t key = key0 + x * 32;
          const uint32_t page = p.page_mul ? __umulhi(key, p.page_mul) >> p.page_shift : key;
          row[x] = (int)key < ke ? __ldg(pages + page) : -1;  // the page's slot for now
          ek[x] = (int)(key - page * p.c.page_size);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool in = (uint32_t)row[x] < pool_pages;
          bad |= !in && key0 + x * 32 < ke;
          row[x] = in ? (int)(row[x] * page_rows + head_row + ek[x]) : -1;
        }
        if (bad) atomicOr(p.status, kStatusBadPage);
        if constexpr (E4) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            ek[x] = row[x] >= 0 ? __ldg(p.c.k_exp + row[x]) : 0;
            ev[x] = row[x] >= 0 ? __ldg(p.c.v_exp + row[x]) : 0;
          }
        }
        int top = -127;  // the largest scale of the tile's keys
        bool folded = false;
        if constexpr (E4 && FOLD) {
          int low = 127;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const bool in = row[x] >= 0 && ek[x] != -128;
            top = in && ek[x] > top ? ek[x] : top;
            low = in && ek[x] < low ? ek[x] : low;
          }
          top = __reduce_max_sync(0xffffffffu, top);
          low = __reduce_min_sync(0xffffffffu, low);
          folded = top - low <= 15;  // also where there is none
          top = top == -127 ? 0 : top;
        }
        int base = -126;  // the largest value scale of the tile's keys
        if constexpr (E4) {
          // A value row of zeros, which the cache holds with exponent 0, adds nothing
          // to O and must not raise the base: it counts as the smallest.  Whether a
          // row with this exponent is one, its codes say (mostly the first few).
          uint32_t zero = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) zero |= row[x] >= 0 && ev[x] == 0 ? 1u << x : 0u;
          if (__any_sync(0xffffffffu, zero != 0)) {
            const uint4* codes = static_cast<const uint4*>(p.c.v);
#pragma unroll 1
            for (int c = 0; c < D / 16 && __any_sync(0xffffffffu, zero != 0); c += 2) {
              uint4 z[8];
#pragma unroll
              for (int x = 0; x < 8; ++x)
                z[x] = zero >> (x >> 1) & 1u ? __ldg(codes + (int64_t)row[x >> 1] * (D / 16) + c + (x & 1)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if ((z[x].x | z[x].y | z[x].z | z[x].w) & 0x7f7f7f7fu) zero &= ~(1u << (x >> 1));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) ev[x] = zero >> x & 1u ? -126 : ev[x];
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) base = row[x] >= 0 && ev[x] > base ? ev[x] : base;
          base = __reduce_max_sync(0xffffffffu, base);
        }
        // the tables of tile j - kBar are used up once its O is done
        if (j >= kBar && !mbar_wait_lazy_warp<200>(smem_u32(&bar_tile[sl]), (j / kBar - 1) & 1)) {
          gave_up = __LINE__;
          break;
        }
        if constexpr (E4) {
          // and of the tiles before, from the other warp's table
          if (j > 0) {
            if (!wait(bar_rows[(j - 1) % kBar], ((j - 1) / kBar) & 1, __LINE__)) break;
            base = max(base, base_s[(j - 1) % kBar]);
          }
          if (lane == 0) base_s[sl] = base;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          row_s[sl][x * 32 + lane] = row[x];
          const uint32_t m = __ballot_sync(0xffffffffu, row[x] >= 0);
          if (lane == 0) there_s[sl][x] = m;
          if constexpr (E4) {
            // 2^(ek - top) in f16 bits, or 2^ek
            const int dk = row[x] >= 0 ? top - ek[x] : 0;
            const uint32_t h = ek[x] == -128 ? 0x7fffu : dk <= 14 ? (uint32_t)(15 - dk) << 10 : 0x200u;
            kh_s[sl][x * 32 + lane] = folded ? h | h << 16 : __float_as_uint(exp_scale(ek[x]));
            // a NaN row reaches only the rows that see it: through the exponent
            const bool nan = ev[x] == -128;
            const int e = row[x] >= 0 ? max(ev[x] - base, -kValueSpan) : 0;
            ev_s[sl][x * 32 + lane] = nan ? exp_scale(-128) : (float)e;
            vi_s[sl][x * 32 + lane] = nan ? 1.f : exp_scale(-e);
          }
        }
        if (E4 && lane == 0) kmax_s[sl] = folded ? exp_scale(top) : 0.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_rows[sl]));
      }
    } else if (warp == 1 && lane == 0 && rank == 0 && ntiles > 0) {
      // ---------------------------------------------------------- products
      constexpr uint32_t kF16 = (1u << 7) | (1u << 10);  // the operands' type bits: bf16, cleared for f16
      constexpr uint32_t idesc_s = idesc_bf16(kBM * kCtas, kBN, false) & ~(E4 ? kF16 : 0u);
      constexpr uint32_t idesc_o = idesc_bf16(kBM * kCtas, L::CW, true) & ~(E4 ? kF16 : 0u);
      auto ready = [&](uint32_t bar, uint32_t parity) { return PAIR ? wait_cluster(bar, parity) : mbar_wait_short(bar, parity); };
      // descriptors count in 16 bytes: a tile's differ by constants
      const uint64_t qd = sdesc_sw128(sQ, 16, 1024);
      bool ok = ready(smem_u32(&bar_q), 0);
      for (int j = -1; ok && j < ntiles; ++j) {
        // S_{j+1} goes to the buffer that held P_{j-1}, read by products issued before
        if (j + 1 < ntiles) {
#pragma unroll 1
          for (int h = 0; h < L::NCH; ++h) {
            const int c = unit_of_k(j + 1) * L::NCH + h;
            ok = ready(smem_u32(&bar_full[c % kBar]), (c / kBar) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = sdesc_sw128(sRing + (c % L::NC) * L::kChunk, 16, 1024);
            const uint64_t qh = qd + (h * 2 * (kBM * 128) >> 4);
#pragma unroll
            for (int kk = 0; kk < L::CW / 16; ++kk)
              product_ss<PAIR>(tS + ((j + 1) & 1) * kBN, qh + (((kk >> 2) * (kBM * 128) + (kk & 3) * 32) >> 4),
                     kd + (((kk >> 2) * L::kBoxK + (kk & 3) * 32) >> 4), idesc_s, (h > 0 || kk > 0) ? 1u : 0u);
            if (h == L::NCH - 1) commit<PAIR>(smem_u32(&bar_s[(j + 1) & 1]));
            commit<PAIR>(smem_u32(&bar_done[c % kBar]));
          }
        }
        if (!ok) gave_up = __LINE__;
        if (j < 0 || !ok) continue;
        ok = ready(smem_u32(&bar_p[j & 1]), (j >> 1) & 1);
#pragma unroll 1
        for (int h = 0; ok && h < L::NCH; ++h) {
          const int c = unit_of_v(j, ntiles) * L::NCH + h;
          ok = ready(smem_u32(&bar_full[c % kBar]), (c / kBar) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sdesc_sw128(sRing + (c % L::NC) * L::kChunk, L::kBoxV, 1024);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            product_ts<PAIR>(tbase + h * L::CW, tS + (j & 1) * kBN + kk * 8, vd + (kk * 2048 >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
          commit<PAIR>(smem_u32(&bar_done[c % kBar]));
        }
        if (!ok) {
          gave_up = __LINE__;
          break;
        }
        commit<PAIR>(smem_u32(&bar_tile[j % kBar]));
        commit<PAIR>(smem_u32(&bar_o));
        if (j == ntiles - 1) commit<PAIR>(smem_u32(&bar_last));
      }
      // no product is under way when the pair ends, not even after a wait gave up; to
      // this CTA alone (what the other was sent, its warp 2 waits for)
      if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&bar_drain)) : "memory");
      else
        mma_commit(smem_u32(&bar_drain));
      ready(smem_u32(&bar_drain), 0);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ chunks
    // four warps take the even chunks, four the odd ones
    fewer_registers<kRegsFill>();
    const int w = tid & 127, group = (warp - 4) >> 2;
    // a thread's NP pieces of a chunk (16 codes or 8 bf16 columns each): piece
    // pc of rows rr, rr + rs, ...  A pair's CTA has 64 keys of K and all its
    // columns, 128 keys of V and half its columns.
    constexpr int PC = E4 ? 16 : 8, ES = E4 ? 1 : 2;
    constexpr int NP = (PAIR ? 64 * D : kBN * L::CW) / PC / 128;
    constexpr int kLogK = log2_of(L::CW / PC), kLogV = PAIR ? kLogK - 1 : kLogK;
    int copied = -1;  // bf16: the chunk whose copies are under way
    auto filled = [&](int c) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive(bar_full[c % kBar]);
    };
    int pc, rr, rs;      // of the chunk to load next
    const char* src = nullptr;
    const int* rows = nullptr;
    const uint32_t* scales = nullptr;  // of the rows of a K chunk that is folded
    auto source = [&](int c) -> bool {  // and waits for its rows
      int j;
      bool is_v;
      unit_at(c / L::NCH, ntiles, j, is_v);
      const int lg = is_v ? kLogV : kLogK;
      if constexpr (E4) {
        // four threads on four pieces of a row, the next four on the next row's:
        // their two 16-byte halves then fall on all banks (rows r and r + 1 differ
        // in the swizzle's lowest bit)
        pc = (w & 3) | ((w >> 3) & ((1 << (lg - 2)) - 1)) << 2, rr = (w >> 2 & 1) | (w >> (lg + 1)) << 1;
        scales = is_v ? nullptr : &kh_s[j % kBar][rr + (PAIR ? rank * 64 : 0)];
      } else {
        pc = w & ((1 << lg) - 1), rr = w >> lg;
      }
      rs = 128 >> lg;
      src = static_cast<const char*>(is_v ? p.c.v : p.c.k) +
            ((c % L::NCH) * L::CW + pc * PC + (PAIR && is_v ? rank * (D / 2) : 0)) * ES;
      rows = &row_s[j % kBar][rr + (PAIR && !is_v ? rank * 64 : 0)];
      const bool in = wait(bar_rows[j % kBar], (j / kBar) & 1, __LINE__);
      if constexpr (E4 && FOLD)
        if (kmax_s[j % kBar] == 0.f) scales = nullptr;
      return in;
    };
    // e4m3: the pieces of the next chunk; each is loaded as soon as its place is
    // converted, so that a group always has about a chunk in flight
    uint4 v[E4 ? NP : 1];
    int at_row[E4 ? NP : 1];
    uint32_t at_scale[E4 ? NP : 1] = {};
    auto fetch = [&](int i) {
      const int row = at_row[i];
      v[i] = row >= 0 ? load_once(reinterpret_cast<const uint4*>(src + (int64_t)row * D)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto find = [&] {  // the rows of all pieces at once, ahead of the loads that need them
#pragma unroll
      for (int i = 0; i < NP; ++i) at_row[i] = rows[i * rs];
    };
    // The scale of piece i, read for the chunk at hand before the next one's source.
    auto find_scales = [&] {
#pragma unroll
      for (int i = 0; i < NP; ++i) at_scale[i] = scales ? scales[i * rs] : 0x3c003c00u;  // 1
    };
    bool ok = true;
    if (E4 && group < nchunks) {
      ok = source(group);
      if (ok) {
        find();
#pragma unroll
        for (int i = 0; i < NP; ++i) fetch(i);
      }
    }
#pragma unroll 1
    for (int c = group; ok && c < nchunks; c += 2) {
      const int next = E4 ? c + 2 : c;
      const int my_pc = pc, my_rr = rr, my_rs = rs;
      if constexpr (E4 && FOLD) find_scales();
      if (next < nchunks) ok = source(next);
      if (ok && c >= L::NC && !mbar_wait_lazy_warp<20>(smem_u32(&bar_done[(c - L::NC) % kBar]), ((c - L::NC) / kBar) & 1)) {
        gave_up = __LINE__;
        ok = false;
      }
      if (!ok) break;
      const uint32_t slot = sRing + (c % L::NC) * L::kChunk;
      const uint32_t box = PAIR && (E4 ? my_rs : rs) == (128 >> kLogK) && kLogK != kLogV ? L::kBoxK : L::kBoxV;
      if constexpr (E4) {
        if (next < nchunks) find();
        // rs is a multiple of 8: a thread's rows have one place in the swizzle,
        // and a piece's halves stand in neighbouring places
        uint32_t d0 = slot + (my_pc >> 2) * box + sw128_offset(my_rr, (my_pc & 3) * 2);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          uint4 x, y;
          codes_f16<FOLD>(v[i].x, at_scale[i], x.x, x.y);
          codes_f16<FOLD>(v[i].y, at_scale[i], x.z, x.w);
          codes_f16<FOLD>(v[i].z, at_scale[i], y.x, y.y);
          codes_f16<FOLD>(v[i].w, at_scale[i], y.z, y.w);
          st_shared_v4(d0, x);
          st_shared_v4(d0 ^ 16u, y);
          d0 += my_rs * 128;
          if (next < nchunks) fetch(i);
        }
        filled(c);
      } else {
        const uint32_t dst = slot + (pc >> 3) * box;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int row = rows[i * rs];
          copy16(dst + sw128_offset(rr + i * rs, pc & 7), src + (int64_t)(row < 0 ? 0 : row) * D * 2, row >= 0);
        }
        copy_commit();
        if (copied >= 0) {
          copy_wait<1>();
          filled(copied);
        }
        copied = c;
      }
    }
    if constexpr (!E4) {
      copy_wait<0>();
      if (copied >= 0) filled(copied);
    }
  } else {
    // ------------------------------------------------------------ softmax
    more_registers<kRegsSoftmax>();
    const int sw = warp - 12, q4 = sw & 3, hf = sw >> 2;
    const int i = q4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    // queries: a warp takes 16 rows, eight columns a lane, all copied to their
    // places at once; e4m3 turns them into f16 there
    const uint32_t my_q = sQ + (lane >> 3) * (kBM * 128);
#pragma unroll 4
    for (int x = 0; x < 16; ++x) {
      const int r = sw * 16 + x, t = r0 + r;
      const int tok = t < r1 ? t / p.gq : 0, hh = t < r1 ? t - tok * p.gq : 0;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(s.q0 + tok) * p.q_stride + (int64_t)(kvh * p.gq + hh) * D + lane * 8;
      if (lane < D / 8) copy16(my_q + sw128_offset(r, lane & 7), src, t < r1);
    }
    copy_commit();
    copy_wait<0>();
    if constexpr (E4) {
#pragma unroll 2
      for (int x = 0; x < 16; ++x) {
        const int r = sw * 16 + x;
        const uint32_t at = my_q + sw128_offset(r, lane & 7);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (lane < D / 8) v = ld_shared_v4(at);
        // f16 with the row's power of two taken out: its largest element in [1, 4)
        uint32_t e[4] = {v.x, v.y, v.z, v.w}, top = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) top = max(top, max((e[y] << 16) & 0x7fffffffu, e[y] & 0x7fff0000u));
        top = __reduce_max_sync(0xffffffffu, top);
        int f = 254 - (int)(top >> 23);
        f = f < 1 ? 1 : f > 253 ? 253 : f;
        const float to = __int_as_float(f << 23);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          e[y] = pack_f16x2(__uint_as_float(e[y] << 16) * to, __uint_as_float(e[y] & 0xffff0000u) * to);
        if (lane < D / 8) st_shared_v4(at, make_uint4(e[0], e[1], e[2], e[3]));
        if (lane == 0) back_s[r] = __int_as_float((254 - f) << 23) * p.scale_log2;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_u32(&bar_back));
      arrive(bar_q);
    }

    bool ok = wait(bar_back, 0, __LINE__);  // back_s of rows that other warps wrote
    const bool row_ok = r0 + i < r1;
    const int tok = row_ok ? (r0 + i) / p.gq : 0, hh = row_ok ? r0 + i - tok * p.gq : 0;
    // a row past the end has zero queries; seeing every key keeps its warp on the short path
    const int lim = row_ok ? row_limit(p, s, tok) : INT32_MAX;
    const float crow = E4 ? back_s[i] : p.scale_log2;
    // the row's maximum, its sum and what the sum is relative to
    float m_run = -CUDART_INF_F, l_run = 0.f, r_run = -CUDART_INF_F;
    if (r0 + q4 * 32 >= r1) {
      // a warp without rows only keeps step: its rows of P may hold anything,
      // since each row of O depends on its own row of P alone
      for (int j = 0; ok && j < ntiles; ++j) {
        ok = wait(bar_s[j & 1], (j >> 1) & 1, __LINE__);
        if (ok && lane == 0) arrive(bar_p[j & 1]);
      }
    }
    const bool busy = r0 + q4 * 32 < r1;
    for (int j = 0; ok && busy && j < ntiles; ++j) {
      const int bf = j & 1, sl = j % kBar, key0 = kb + j * kBN + hf * 64;
      ok = wait(bar_rows[sl], (j / kBar) & 1, __LINE__) && wait(bar_s[bf], (j >> 1) & 1, __LINE__);
      if (!ok) break;
      tc_fence_after();
      uint64_t y[32];  // scores of this half's 64 keys, two by two
      {
        uint32_t a0[32], a1[32];
        const uint32_t sa = tS + lanes + bf * kBN + hf * 64;
        tmem_ld32(sa, a0);
        tmem_ld32(sa + 32, a1);
        tmem_wait_ld_r(a0);
        reg_dep(a1);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          y[c] = f2(__uint_as_float(a0[2 * c]), __uint_as_float(a0[2 * c + 1]));
          y[16 + c] = f2(__uint_as_float(a1[2 * c]), __uint_as_float(a1[2 * c + 1]));
        }
      }
      if constexpr (E4) {
        const bool by_key = !FOLD || kmax_s[sl] == 0.f;  // the keys' scales are still to be multiplied
        const float ct = by_key ? crow : crow * kmax_s[sl];
        const uint64_t c2 = f2(ct, ct);
        const ulonglong2* kf = reinterpret_cast<const ulonglong2*>(&kh_s[sl][hf * 64]);
        const ulonglong2* ev = reinterpret_cast<const ulonglong2*>(&ev_s[sl][hf * 64]);
        if (by_key) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const ulonglong2 f = kf[c];
            y[2 * c] = f2_mul(y[2 * c], f.x);
            y[2 * c + 1] = f2_mul(y[2 * c + 1], f.y);
          }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const ulonglong2 e = ev[c];
          y[2 * c] = f2_fma(y[2 * c], c2, e.x);
          y[2 * c + 1] = f2_fma(y[2 * c + 1], c2, e.y);
        }
      }
      // keys that exist and that this row sees
      const int nv = lim - key0;
      uint64_t see = (uint64_t)there_s[sl][hf * 2] | (uint64_t)there_s[sl][hf * 2 + 1] << 32;
      if (nv < 64) see &= nv > 0 ? ~0ull >> (64 - nv) : 0ull;
      float mq[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
      if (!__all_sync(0xffffffffu, see == ~0ull)) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float a, bb;
          f2_split(y[c], a, bb);
          y[c] = f2(see >> (2 * c) & 1 ? a : -CUDART_INF_F, see >> (2 * c + 1) & 1 ? bb : -CUDART_INF_F);
        }
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float a, bb;
        f2_split(y[c], a, bb);
        mq[c & 3] = max3f(mq[c & 3], a, bb);
      }
      float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
      // both halves of a row meet: they exchange their maxima, and each has
      // read its half of S before P overwrites it
      top_s[bf][hf][i] = mx;
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_pair[q4]));
      ok = wait(bar_pair[q4], j & 1, __LINE__);
      if (!ok) break;
      tc_fence_after();
      mx = fmaxf(mx, top_s[bf][hf ^ 1][i]);
      const float base = E4 ? (float)base_s[sl] : 0.f;
      if constexpr (E4)
        mx += base;
      else
        mx *= crow;
      float alpha = 1.f;
      bool rescale = false;
      if (mx > m_run + kSlack) {
        if (m_run != -CUDART_INF_F) {
          alpha = ex2(m_run - mx);
          rescale = true;
        }
        if constexpr (!E4) l_run *= alpha;
        m_run = mx;
      }
      if (__any_sync(0xffffffffu, rescale)) {
        // S_j done means PV_{j-2} done, so bar_o has completed j-1 or j phases
        ok = wait(bar_o, (j - 1) & 1, __LINE__);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = hf * (D / 2); c0 < (hf + 1) * (D / 2); c0 += 32) {
          uint32_t rr[32];
          tmem_ld32(tbase + lanes + c0, rr);
          tmem_wait_ld_r(rr);
#pragma unroll
          for (int c = 0; c < 32; ++c) rr[c] = __float_as_uint(__uint_as_float(rr[c]) * alpha);
          tmem_st32(tbase + lanes + c0, rr);
        }
        tmem_wait_st();
      }
      // a row that has seen no key keeps its reference at 0: -infinity gives a
      // weight of 0, and a NaN stays one.  e4m3: r is the sum's reference too, so
      // that what its subtraction rounds stays out of the result
      const float r = m_run - base, ref = kOff - (m_run == -CUDART_INF_F ? 0.f : r);
      const uint64_t nref = f2(ref, ref), sc2 = f2(crow, crow);
      uint64_t acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
      const ulonglong2* vi = reinterpret_cast<const ulonglong2*>(&vi_s[E4 ? sl : 0][hf * 64]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int x = half * 16 + 2 * c;
          float e[4];
          if constexpr (E4) {
            f2_split(f2_add(y[x], nref), e[0], e[1]);
            f2_split(f2_add(y[x + 1], nref), e[2], e[3]);
          } else {
            f2_split(f2_fma(y[x], sc2, nref), e[0], e[1]);
            f2_split(f2_fma(y[x + 1], sc2, nref), e[2], e[3]);
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) e[z] = ex2(e[z]);
          if constexpr (E4) {
            const ulonglong2 f = vi[half * 8 + c];
            acc[0] = f2_fma(f2(e[0], e[1]), f.x, acc[0]);
            acc[1] = f2_fma(f2(e[2], e[3]), f.y, acc[1]);
            pk[2 * c] = pack_f16x2(e[0], e[1]);
            pk[2 * c + 1] = pack_f16x2(e[2], e[3]);
          } else {
            acc[0] = f2_add(acc[0], f2(e[0], e[1]));
            acc[1] = f2_add(acc[1], f2(e[2], e[3]));
            pk[2 * c] = pack_bf16x2(e[0], e[1]);
            pk[2 * c + 1] = pack_bf16x2(e[2], e[3]);
          }
        }
        tmem_st16(tS + lanes + bf * kBN + hf * 32 + half * 16, pk);
      }
      float p0, p1, p2, p3;
      f2_split(acc[0], p0, p1);
      f2_split(acc[1], p2, p3);
      const float sum = (p0 + p1) + (p2 + p3);
      if constexpr (E4) {
        // the larger reference holds for both; 0 where no key was seen yet
        const float rn = fmaxf(r_run, r), at = rn == -CUDART_INF_F ? 0.f : rn;
        l_run = l_run * ex2(r_run - at) + sum * ex2(r - at);
        r_run = rn;
      } else {
        l_run += sum;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(bar_p[bf]);
    }
    // ---- the row sums of both halves, then this half of O's columns
    float l = 0.f;
    if (ok && ntiles > 0 && busy) {
      ok = wait(bar_last, 0, __LINE__);
      tc_fence_after();
      if (ok) {
        top_s[ntiles & 1][hf][i] = l_run;
        mbar_arrive(smem_u32(&bar_pair[q4]));
        ok = wait(bar_pair[q4], ntiles & 1, __LINE__);
      }
      if (ok) l = top_s[ntiles & 1][0][i] + top_s[ntiles & 1][1][i];
    }
    const int64_t out = (int64_t)(s.q0 + tok) * p.hq + kvh * p.gq + hh;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float seen = E4 ? r_run : m_run, lref = seen == -CUDART_INF_F ? 0.f : seen;
    const float to = E4 ? ex2(m_run - seen) : 1.f;  // from O's reference to the sum's
#pragma unroll 1
    for (int c0 = hf * (D / 2); c0 < (hf + 1) * (D / 2); c0 += 32) {
      uint32_t rr[32];
      __syncwarp();
      if (ok && ntiles > 0 && busy) {
        tmem_ld32(tbase + lanes + c0, rr);
        tmem_wait_ld_r(rr);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) rr[c] = 0u;
      }
      if (!row_ok) continue;
      // a row without keys: its O was never weighted, and 0 times it is 0
      float v[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = l == 0.f ? 0.f : __uint_as_float(rr[c]) * inv * to;
      if (p.ns > 1 || p.o_dtype == LS_DTYPE_F32) {
        float* dst = (p.ns > 1 ? p.o_parts + (int64_t)part * p.total_q * p.hq * D : static_cast<float*>(p.o)) + out * D + c0;
#pragma unroll
        for (int c = 0; c < 32; c += 4) *reinterpret_cast<float4*>(dst + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + out * D + c0;
#pragma unroll
        for (int c = 0; c < 32; c += 8)
          *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack_bf16x2(v[c], v[c + 1]), pack_bf16x2(v[c + 2], v[c + 3]),
                                                          pack_bf16x2(v[c + 4], v[c + 5]), pack_bf16x2(v[c + 6], v[c + 7]));
      }
    }
    if (row_ok && hf == 0) {
      const float z = l == 0.f ? -CUDART_INF_F : (lref + log2f(E4 ? l * 0x1p-11f : l)) * kLn2;
      if (p.ns > 1)
        p.lse_parts[(int64_t)part * p.total_q * p.hq + out] = z;
      else
        p.lse[out] = z;
    }
  }
  // What the products announce has arrived before a CTA ends, whether or not it has rows:
  // an arrival must not find its shared memory given back.  bar_last comes with the last
  // product; by then each other barrier stands at its last phase or the one before.
  if (warp == 2 && ntiles > 0) {
    bool in = wait(bar_last, 0, __LINE__) && wait(bar_o, (ntiles - 1) & 1, __LINE__);
#pragma unroll 1
    for (int x = 1; in && x <= kBar; ++x) {
      const int c = nchunks - x, j = ntiles - x;
      if (c >= 0) in = wait(bar_done[c % kBar], (c / kBar) & 1, __LINE__);
      if (in && j >= 0) in = wait(bar_tile[j % kBar], (j / kBar) & 1, __LINE__);
      if (in && j >= 0 && x <= 2) in = wait(bar_s[j & 1], (j >> 1) & 1, __LINE__);
    }
  }
  if (gave_up && (lane == 0 || warp == 1)) {
    atomicOr(p.status, kStatusTimeout);
    atomicCAS(p.status + 1, 0u, ((uint32_t)kKCachedTc << 16) | (uint32_t)gave_up);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tbase) : "memory");
    else
      tmem_dealloc(tbase, 512);
  }
}

template <int D, bool E4, bool PAIR>
cudaError_t run_tc(const CachedParams& p, cudaStream_t s) {
  using L = TcShape<D, PAIR>;
  auto* kernel = cached_tc_kernel<D, E4, PAIR>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.max_q * p.gq, per = kBM * (PAIR ? 2 : 1);
  const int64_t ctas = (rows + per - 1) / per * p.ns * (PAIR ? 2 : 1);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  LaunchScope ls(kKCachedTc, s);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, p.c.hkv, p.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = PAIR ? 2 : 1, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// 30,000 keys, one CTA's tiles against pairs': d 256, 144 rows 57 and 49 us, 768 rows
// 125 and 102; d 128, 96 rows 43 and 66 (a pair's second half would be empty), 160 rows
// 72 and 66, 512 rows 125 and 109 (e4m3; bf16 alike).
bool cached_tc_pairs(int64_t rows, int d) { return rows > kBM && d >= 128; }

cudaError_t launch_cached_tc(const CachedParams& p, cudaStream_t s) {
  const bool e4 = p.c.format == LS_CACHE_E4M3, pair = cached_tc_pairs((int64_t)p.max_q * p.gq, p.c.head_dim);
  switch (p.c.head_dim) {
    case 64: return e4 ? run_tc<64, true, false>(p, s) : run_tc<64, false, false>(p, s);
    case 128:
      if (pair) return e4 ? run_tc<128, true, true>(p, s) : run_tc<128, false, true>(p, s);
      return e4 ? run_tc<128, true, false>(p, s) : run_tc<128, false, false>(p, s);
    default:
      if (pair) return e4 ? run_tc<256, true, true>(p, s) : run_tc<256, false, true>(p, s);
      return e4 ? run_tc<256, true, false>(p, s) : run_tc<256, false, false>(p, s);
  }
}

}  // namespace ls
