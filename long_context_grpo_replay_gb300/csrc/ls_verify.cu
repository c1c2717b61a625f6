// Verification of drafted tokens against the target's logits, and the draw of
// the token after them.
//
//   p_r(v) = exp(s z_rv - lse_r);  a draft x is accepted while u_r q_r(x) < p_r(x);
//   next token: least v with sum_{j<=v} w_j > u sum_j w_j,  w = max(p - q, 0) or p.
//
// Two kernels.  verify_rows_kernel reads every logit once: a (maximum, sum) pair
// for each row and 2 KB of it, in base 2.  verify_draw_kernel, a cluster of up to eight
// blocks for each sequence, joins them, tests the drafts and draws from the one
// row where they end.
//
// The draw compares u with a running sum that has a step for every token, 10^5
// of them in [0, 1): with sums good to 2^-24 one draw in a hundred would give a
// neighbour of the definition's token.  So the draw's weights are formed anew, to
// 2^-30 of each (2^-33 rms), and summed as exactly:
//   e = 2^(s log2(e) (z - max)) = 2^(k/256) (1 + d),  d = 2^f - 1,  |f| <= 2^-8,
// k/256 being z's product rounded to that grid less the maximum's (both exact),
// f what is left of both, formed by fused multiply-adds; 2^(j/256) comes from a
// table of pairs (Tang's method: P. T. P. Tang, Table-driven implementation of the
// exponential function, ACM TOMS 15, 1989) and d from three terms (the fourth is
// below 2^-38).  A weight, scaled so that all of them sum to less than 1, is split
// at 2^-22: sums of the upper parts are exact in float32.  A lower part is 2^-8.5 of
// its weight at most, and 2^-23: below that a weight is all lower part, good to
// 2^-24 of itself, 2^-47 of the row.  A thread adds up to 256 of them in float32, in
// longer segments 64 at a time; beyond that they are integers in units of 2^-61, whose
// sums do not depend on their order.  Roundings that fall as they may leave about
// 2^-31 of the row; at worst, where all of a thread's parts are alike, 2^-17.6 of what
// the lower parts sum to (2^-20.6 in longer segments).
//   After a rejection w = max(e - q Z, 0) needs Z, the sum of all e, before the
// first of them is known: the pass takes the row's float32 sum Z0, and as Z is
// within about 2^-20 of it (2^-17 at most up to 2^17 tokens), each partial sum is put
// right afterwards by (Z - Z0) times the sum of its q where e > q Z0 (tokens as near
// that border weigh 2^-20 of theirs, so that their side does not matter).
//   Measured: 64 sequences of up to 5 rows x 128,000 (54 MB) 29.2 us: the rows' pass 8
// (4.3 TB/s with cold caches), the draw 20, of which half is the weights' arithmetic
// (34 instructions an element, three issued a cycle on the SMs that hold four blocks)
// and half the chain of a block's loads, barriers and scans.  Packed pairs with a copy
// of the table in each bank take a seventh fewer instructions and more registers (30.6
// against 26.4 us of the draw with cold caches).

#include <cuda_bf16.h>

#include "ls_cluster.cuh"
#include "ls_internal.h"
#include "ls_tc.cuh"

namespace ls {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kEach = 4, kVectors = 32 * kEach, kChunkBytes = 16 * kVectors;  // a warp's in the pass over the rows
constexpr int kMaxCluster = 8;
constexpr int kTile = 256;  // elements a warp takes at a time in the draw, eight a lane
constexpr int kShort = 32, kChain = 8;  // tiles whose lower parts a lane sums in float32: of a whole segment, of a longer one at a time

// ---------------------------------------------------------------- 2^(j/256)
struct Table {
  float2 v[256];  // as a pair: its 24 upper bits, and the rest
};
// From square roots of 2 in integers of 62 bits (each off by less than 2^-60).
constexpr uint64_t root(uint64_t x) {  // sqrt(x * 2^62)
  const unsigned __int128 n = (unsigned __int128)x << 62;
  uint64_t r = 0;
  for (int b = 62; b >= 0; --b) {
    const uint64_t t = r | (1ull << b);
    if ((unsigned __int128)t * t <= n) r = t;
  }
  return r;
}
constexpr Table make_table() {
  Table t{};
  uint64_t roots[8] = {};
  uint64_t x = 1ull << 63;  // 2 * 2^62
  for (int i = 7; i >= 0; --i) x = root(x), roots[i] = x;  // roots[i] = 2^(2^i / 256)
  for (int j = 0; j < 256; ++j) {
    uint64_t y = 1ull << 62;
    for (int i = 0; i < 8; ++i)
      if (j >> i & 1) y = (uint64_t)((unsigned __int128)y * roots[i] >> 62);
    const uint64_t upper = (y + (1ull << 38)) >> 39;
    t.v[j] = float2{(float)upper * 0x1p-23f, (float)((int64_t)y - (int64_t)(upper << 39)) * 0x1p-62f};
  }
  return t;
}
__device__ constexpr Table kExp2 = make_table();

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (maximum, sum of 2^(c (z - maximum))) of two sets.  A NaN stays in the sum.
__device__ __forceinline__ float2 join(float2 a, float2 b, float c) {
  const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * ex2((a.x - base) * c) + b.y * ex2((b.x - base) * c));
}
__device__ __forceinline__ float2 join_warp(float2 a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = join(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o)), c);
  return a;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// The elements of a 16-byte piece in pairs of floats, and their largest (a NaN aside).
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ float largest(const uint4& w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ uint64_t pair(const uint4& w, int i) {
    return i ? tc::f2(__uint_as_float(w.z), __uint_as_float(w.w)) : tc::f2(__uint_as_float(w.x), __uint_as_float(w.y));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  static __device__ __forceinline__ float largest(const uint4& w) {
    const __nv_bfloat162 m = __hmax2(__hmax2(two(w.x), two(w.y)), __hmax2(two(w.z), two(w.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint64_t pair(const uint4& w, int i) {
    const uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return tc::f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
};

// A warp takes 2 KB of a row by itself: all of it loaded at once, the maximum of the
// lanes first, the exponentials relative to it, on packed pairs.  A row starts
// anywhere: its 16-byte pieces are dealt out, the elements before the first and after
// the last go to its first warp.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_rows_kernel(const VerifyParams p) {
  constexpr int E = Piece<T>::E;
  asm volatile("griddepcontrol.launch_dependents;");  // the draw's blocks set up while the last rows are read
  const int64_t part = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (part >= p.d.total_q * p.chunks) return;
  const int64_t r = part / p.chunks;
  const int chunk = (int)(part - r * p.chunks), lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(p.logits) + r * p.d.logits_stride;
  const int before = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
  const int head = before < p.d.vocab ? before : p.d.vocab;
  const int vectors = (p.d.vocab - head) / E, tail = p.d.vocab - head - vectors * E;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  uint4 w[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = chunk * kVectors + i * 32 + lane;
    constexpr uint32_t low = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -infinity
    w[i] = at < vectors ? __ldcs(body + at) : make_uint4(low, low, low, low);
  }
  float z = -INFINITY;
  if (chunk == 0) {
    if (lane < head) z = value(row[lane]);
    if (lane >= 16 && lane < 16 + tail) z = value(row[head + vectors * E + lane - 16]);
  }
  float m = z;
#pragma unroll
  for (int i = 0; i < kEach; ++i) m = fmaxf(m, Piece<T>::largest(w[i]));
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  const uint64_t base2 = tc::f2(-base, -base), c2 = tc::f2(p.c, p.c);
  float sum = ex2((z - base) * p.c);
  uint64_t more = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      float lo, hi;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(tc::f2_mul(tc::f2_add(Piece<T>::pair(w[i], j), base2), c2)));
      more = tc::f2_add(more, tc::f2(ex2(lo), ex2(hi)));
    }
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(more));
  sum += lo + hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) p.parts[part] = make_float2(m, sum);
}

// ---------------------------------------------------------------- the draw
struct Row {
  float base;      // taken off every logit first where it is not 0: the maximum, where the products would leave the grid
  float bias;      // 1.5 * 2^15 less the maximum's product on the grid of 2^-8
  float rest;      // the rest of that product
  float least;     // logits below it count as it: 2^-90 of the largest weight, nothing in units of 2^-61
  float c, c_low;
  uint32_t scale;  // exponent bits of 2^-k, with 2^-k Z in [0.5, 1)
  float z0;        // 2^-k Z0
};
constexpr uint32_t kGrid = 0x47400000u;  // 1.5 * 2^15: a float near it is a multiple of 2^-8

__device__ __forceinline__ Row make_row(float top, float sum, float c, float c_low) {
  Row r;
  r.c = c, r.c_low = c_low;
  r.base = fabsf(top) * c > 8192.f ? top : 0.f;
  const float m = top - r.base, hi = m * c;
  const float grid = rintf(hi * 256.f) * 0x1p-8f;
  r.rest = (hi - grid) + fmaf(m, c_low, fmaf(m, c, -hi));
  r.bias = __uint_as_float(kGrid) - grid;
  r.least = fmaxf(m - 90.f / c, -3.402823466e38f);
  const uint32_t bits = __float_as_uint(sum);
  r.scale = (253u - (bits >> 23)) << 23;                         // 127 - (exponent + 1)
  r.z0 = __uint_as_float((bits & 0x7fffffu) | 0x3f000000u);
  return r;
}

// e = 2^(c (z - top)) in the row's units, as a sum of two floats: the lower one is
// up to 2^-8.5 of the upper.
__device__ __forceinline__ void weight(float z, const Row& r, const float2* table, float& upper, float& lower) {
  if (r.base != 0.f) z -= r.base;
  const float s = fmaxf(z, r.least);
  const float t = fmaf(s, r.c, r.bias);
  const float f = fmaf(s, r.c, r.bias - t) + fmaf(s, r.c_low, -r.rest);
  const uint32_t k = __float_as_uint(t);
  const float2 w = table[k & 255u];
  const float d = f * fmaf(f, fmaf(f, 0.0555041087f, 0.240226507f), 0.693147181f);  // powers of ln 2 over factorials
  const float scale = __uint_as_float(((k & 0xffffff00u) << 15) + r.scale);
  upper = w.x * scale;
  lower = fmaf(w.x, d, w.y) * scale;
}
// The multiples of 2^-22 nearest to x in [0, 1).
__device__ __forceinline__ float on_grid(float x) { return (x + 3.f) - 3.f; }

// 2^61 times a float below 2, towards 0, by its bits (a conversion to 64 bits runs on the slow double pipe).
__device__ __forceinline__ int64_t fixed(float x) {
  const uint32_t u = __float_as_uint(x);
  const int shift = (int)((u >> 23) & 255u) - 89;  // the 24 bits count 2^(e - 150)
  const uint64_t m = (u & 0x7fffffu) | 0x800000u;
  const int64_t y = (int64_t)(shift >= 0 ? m << shift : shift > -24 ? m >> -shift : 0);
  return (int32_t)u < 0 ? -y : y;
}
__device__ __forceinline__ int64_t fixed(float a, float b) { return fixed(a) + fixed(b); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Sums of the lanes before and with this one.
__device__ __forceinline__ uint64_t warp_prefix(uint64_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// floor(u * c) for c < 2^62; c - 1 for u >= 1, 0 for what is not above 0.
__device__ __forceinline__ uint64_t part_of(float u, uint64_t c) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return c - 1;
  const uint32_t b = __float_as_uint(u);
  const int e = (int)(b >> 23);
  if (e == 0) return 0;
  const uint64_t x = __umul64hi((uint64_t)((b & 0x7fffffu) | 0x800000u) << 40, c);
  return 126 - e > 63 ? 0 : x >> (126 - e);
}

// Elements v .. v+7 of a row, as they lie; `outside` for those before or after it.
// whole: p + v is 16-byte aligned.
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int v, int end, bool whole, uint32_t outside) {
  Raw8<T> r;
  if (whole && v >= 0 && v + 8 <= end) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 a = reinterpret_cast<const uint4*>(p + v)[i];
      r.w[4 * i] = a.x, r.w[4 * i + 1] = a.y, r.w[4 * i + 2] = a.z, r.w[4 * i + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t x = outside;
      if (v + i >= 0 && v + i < end) {
        if constexpr (sizeof(T) == 4)
          x = reinterpret_cast<const uint32_t*>(p)[v + i];
        else
          x = reinterpret_cast<const uint16_t*>(p)[v + i];
      }
      if constexpr (sizeof(T) == 4)
        r.w[i] = x;
      else
        r.w[i / 2] |= x << (16 * (i & 1));
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ float element(const Raw8<T>& r, int i) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(r.w[i]);
  else
    return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}
// A row's logits, and the drafts' probabilities beside them (null: none).
template <typename T>
struct Source {
  const T* z;
  const float* q;
  int end;
  bool whole;  // q is aligned where z is
  __device__ __forceinline__ Raw8<T> logits(int v) const { return load8(z, v, end, true, sizeof(T) == 4 ? 0xff800000u : 0xff80u); }
  __device__ __forceinline__ Raw8<float> shares(int v) const { return load8(q, v, end, whole, 0u); }
};

struct Sums {
  uint64_t e, w;  // of all weights, and of those that the draw is from
  float q;
};
// This lane's part of the elements lo .. stop-1 (lo where a 16-byte piece begins, perhaps before the row).
// Long: of more than kShort tiles; the lower parts' sums are put aside after every kChain.
template <bool Q, bool Long, typename T>
__device__ __forceinline__ Sums segment(const Source<T>& src, int lo, int stop, const Row& r, const float2* table) {
  float e0 = 0.f, e1 = 0.f, w0 = 0.f, w1 = 0.f, sum_q = 0.f, all_q = 0.f;
  int64_t e = 0, w = 0;
  int v = lo + (threadIdx.x & 31) * 8;
  Raw8<T> x = src.logits(v);
  Raw8<float> y{};
  if constexpr (Q) y = src.shares(v);
  auto add = [&](int till) {
    for (; v < till; v += kTile) {
      const Raw8<T> x1 = src.logits(v + kTile);  // under this tile's arithmetic
      Raw8<float> y1{};
      if constexpr (Q) y1 = src.shares(v + kTile);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, b;
        weight(element(x, i), r, table, a, b);
        const float a0 = on_grid(a), a1 = (a - a0) + b;
        e0 += a0, e1 += a1;
        if constexpr (Q) {
          const float q = fmaxf(element(y, i), 0.f), s = q * r.z0, s0 = on_grid(s);
          const float d0 = a0 - s0, d1 = a1 - ((s - s0) + fmaf(q, r.z0, -s));
          if (d0 + d1 > 0.f) w0 += d0, w1 += d1, sum_q += q;
        }
      }
      x = x1, y = y1;
    }
  };
  if constexpr (Long) {
    while (v < stop) {
      add(min(stop, v + kChain * kTile));
      e += fixed(e1), e1 = 0.f;
      if constexpr (Q) w += fixed(w1), w1 = 0.f, all_q += sum_q, sum_q = 0.f;
    }
  } else {
    add(stop);
  }
  Sums s;
  s.e = (uint64_t)(e + fixed(e0, e1));
  if constexpr (Q) {
    w += fixed(w0, w1);
    s.w = w > 0 ? (uint64_t)w : 0;
  } else {
    s.w = s.e;
  }
  s.q = all_q + sum_q;
  return s;
}

// The token of elements from .. stop-1 in which the running sum of the weights passes t
// (all of a block): its index in the thread that has it, below 0 in the others.  over_q:
// weights are max(e - q Z, 0), Z = z_hi + z_lo; but: an element that weighs nothing.  its:
// the token's logit, in the same thread.
template <typename T>
__device__ __forceinline__ int look(const Source<T>& src, const Row& w, const float2* table, int64_t from, int stop, uint64_t t,
                                    bool over_q, float z_hi, float z_lo, int but, uint64_t* scan, int* most_of, float& its) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int found = -1, last = -1;  // the last token so far that weighs anything
  for (int lo = (int)from, turn = 0; found == -1; lo += kThreads * 8) {
    if (lo >= stop) {
      // The sum that t was taken from may be past the tiles' own by rounding: their last token then.  And rounding may
      // have left a sum where no token is to be drawn (the rejected draft's part, tokens that weigh less than a unit):
      // the next one behind comes out, or else the row's last, by p alone (a remainder's last segments hold nothing else).
      if (last >= 0 || turn == 2) break;
      if (turn == 0 && stop < src.end)
        turn = 1, lo = stop, stop = src.end, t = 0;
      else
        turn = 2, lo = (int)-(-from & 7), stop = src.end, t = ~0ull, over_q = false;  // from where a piece begins
    }
    const int v = lo + tid * 8;
    uint64_t x[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0;
    Raw8<T> raw{};
    if (v < stop) {
      raw = src.logits(v);
      Raw8<float> share{};
      if (over_q) share = src.shares(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, b;
        weight(element(raw, i), w, table, a, b);
        int64_t e = 0;
        if (over_q) {
          const float y = fmaxf(element(share, i), 0.f), s = y * z_hi, rest = fmaf(y, z_lo, fmaf(y, z_hi, -s));
          const float a0 = on_grid(a), s0 = on_grid(s), d0 = a0 - s0, d1 = ((a - a0) + b) - ((s - s0) + rest);
          if (d0 + d1 > 0.f) e = fixed(d0, d1);
        } else if (v + i != but) {
          e = fixed(a, b);
        }
        if (v + i < stop && e > 0) x[i] = (uint64_t)e, sum += x[i];
      }
    }
    int mine = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (x[i]) mine = v + i;
    uint64_t upto = warp_prefix(sum);
    if (lane == 31) scan[warp] = upto;
    const int most = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) most_of[warp] = most;
    __syncthreads();
    uint64_t total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) upto += scan[i];
      total += scan[i];
      last = max(last, most_of[i]);
    }
    if (t < total) {
      found = -2;  // in this tile, by one thread
      uint64_t run = upto - sum;
      if (t >= run && t < upto)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          run += x[i];
          if (found < 0 && run > t) found = v + i, its = element(raw, i);
        }
    } else {
      t -= total;
    }
    __syncthreads();
  }
  if (found == -1 && last >= 0 && tid == 0) found = last, its = value(src.z[last]);
  return found;
}

template <typename T, bool Long>
__global__ void __launch_bounds__(kThreads, 4) verify_draw_kernel(const VerifyParams p) {
  using Team = Cluster<0>;
  __shared__ float2 table[256];
  __shared__ float2 row_of[kWarps];
  __shared__ int passes[kWarps];
  __shared__ uint64_t seg_e[kWarps], seg_w[kWarps], scan[kWarps];
  __shared__ float seg_q[kWarps];
  __shared__ int picked, use_p;
  __shared__ uint64_t target, z_all;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = Team::rank(), blocks = Team::size();
  table[tid] = kExp2.v[tid];
  const int64_t first = p.q_start[b], n64 = p.q_start[b + 1] - first;
  const bool bad = first < 0 || n64 < 0 || first + n64 > p.d.total_q || n64 > p.d.max_q;
  if (bad || n64 == 0) {  // all blocks of the cluster
    if (rank == 0 && tid == 0) {
      if (bad) atomicOr(p.status, kStatusBadIndex);
      p.n_emitted[b] = 0;
      if (p.keep) p.keep[b] = p.kv_len[b];
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // who comes after this kernel comes after the rows' too
    return;
  }
  const int n = (int)n64, V = p.d.vocab;
  const T* logits = static_cast<const T*>(p.logits);
  // A warp a row: what its draft is, and what is said of it.
  struct Draft {
    int64_t x;
    float z, q, u;
  };
  auto draft_of = [&](int i) {
    Draft d{-1, 0.f, 1.f, 0.f};
    if (i + 1 < n) {
      const int64_t r = first + i;
      d.x = p.tokens[r + 1], d.u = p.u[r];
      if (d.x >= 0 && d.x < V) {
        d.z = value(logits[r * p.d.logits_stride + d.x]);
        if (p.probs) d.q = fmaxf(p.probs[r * p.d.draft_stride + d.x], 0.f);
      }
    }
    return d;
  };
  Draft draft0 = draft_of(warp);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' pairs are there
  // the drafts, a warp a row, up to the first that does not pass
  int stop = -1;
  float2 row{};
  for (int i0 = 0; stop < 0; i0 += kWarps) {
    const int i = i0 + warp;
    if (i < n) {
      const int64_t r = first + i;
      float2 a = make_float2(-INFINITY, 0.f);
      for (int x = lane; x < p.chunks; x += 32) a = join(a, p.parts[r * p.chunks + x], p.c);
      a = join_warp(a, p.c);
      bool pass = false;
      const Draft t = i0 ? draft_of(i) : draft0;
      if (i + 1 < n) {
        if (t.x >= 0 && t.x < V) {
          const float d = t.z - a.x, x = d * p.c;
          // below 2^-149 it is 0, whatever d * c_low is: that may overflow where c_low is negative
          pass = t.u * t.q * a.y < (x < -160.f ? 0.f : exp2f(fmaf(d, p.c, d * p.c_low)));
          if (pass && rank == 0 && lane == 0) {
            p.emitted[r] = t.x;
            if (p.logp) p.logp[r] = d * p.d.logit_scale - logf(a.y);
          }
        } else if (rank == 0 && lane == 0) {
          atomicOr(p.status, kStatusBadIndex);
        }
      }
      if (lane == 0) row_of[warp] = a, passes[warp] = pass;
    }
    __syncthreads();
    for (int w = 0; w < kWarps && i0 + w < n && stop < 0; ++w)
      if (!passes[w]) stop = i0 + w, row = row_of[w];
    __syncthreads();
  }
  const int64_t r = first + stop;
  const bool rejected = stop + 1 < n, some = row.x > -INFINITY && row.y > 0.f && row.y < INFINITY;
  if (rank == 0) {  // what came out, but for the new token
    for (int i = stop + 1 + tid; i < n; i += kThreads) {
      p.emitted[first + i] = -1;
      if (p.logp) p.logp[first + i] = 0.f;
    }
    if (tid == 0) {
      p.n_emitted[b] = stop + (some ? 1 : 0);
      if (p.keep) p.keep[b] = p.kv_len[b] - n + stop + 1;
      if (!some) {
        atomicOr(p.status, kStatusBadIndex);
        p.emitted[r] = -1;
        if (p.logp) p.logp[r] = 0.f;
      }
    }
  }
  if (!some) return;  // all blocks of the cluster
  const Row w = make_row(row.x, row.y, p.c, p.c_low);
  const T* z = logits + r * p.d.logits_stride;
  const float* q = p.probs && rejected ? p.probs + r * p.d.draft_stride : nullptr;
  const int64_t next = rejected && !p.probs ? p.tokens[r + 1] : -1;
  const int draft = next >= 0 && next < V ? (int)next : -1;  // an id outside takes nothing out of the row
  // each warp its segment of the row; segments begin where 16-byte pieces do, `shift` elements before the row
  const int shift = (int)(reinterpret_cast<uintptr_t>(z) & 15) / (int)sizeof(T);
  const Source<T> src{z, q, V, (reinterpret_cast<uintptr_t>(q - shift) & 15) == 0};
  const int segments = (int)blocks * kWarps, tiles = (V + shift + kTile - 1) / kTile;
  const int each = (tiles + segments - 1) / segments * kTile;
  {
    const int64_t lo = (int64_t)((int)rank * kWarps + warp) * each - shift;
    const int stop = (int)(lo + each < V ? lo + each : V);
    Sums s{};
    if (lo < V) s = q ? segment<true, Long>(src, (int)lo, stop, w, table) : segment<false, Long>(src, (int)lo, stop, w, table);
    s.e = warp_sum(s.e), s.w = warp_sum(s.w), s.q = warp_sum(s.q);
    if (draft >= 0 && draft >= lo && draft < lo + each) {
      float a, b;
      weight(value(z[draft]), w, table, a, b);
      const uint64_t x = (uint64_t)fixed(a, b);
      s.w = s.w > x ? s.w - x : 0;
    }
    if (lane == 0) seg_e[warp] = s.e, seg_w[warp] = s.w, seg_q[warp] = s.q;
  }
  Team::sync();
  if (warp == 0) {  // two segments a lane, neighbours
    uint64_t e[2], x[2];
    float sq[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = 2 * lane + i;
      const bool in = s < segments;
      e[i] = in ? Team::at(seg_e + s % kWarps, s / kWarps) : 0;
      x[i] = in ? Team::at(seg_w + s % kWarps, s / kWarps) : 0;
      sq[i] = in ? Team::at(seg_q + s % kWarps, s / kWarps) : 0.f;
    }
    const uint64_t all = warp_sum(e[0] + e[1]);
    const float off = (float)((int64_t)all - fixed(w.z0)) * 0x1p-61f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t right = q ? (int64_t)x[i] - fixed(off * sq[i]) : (int64_t)x[i];
      x[i] = right > 0 ? (uint64_t)right : 0;
    }
    const bool none = warp_sum(x[0] + x[1]) <= all >> 30;  // 2^-30 of the row: it may be rounding alone
    if (none) x[0] = e[0], x[1] = e[1];
    const uint64_t upto = warp_prefix(x[0] + x[1]), total = __shfl_sync(0xffffffffu, upto, 31);
    const uint64_t t = part_of(p.u_next[b], total), before = upto - x[0] - x[1];
    const unsigned here = __ballot_sync(0xffffffffu, t < upto);  // t < total: a lane has it
    if (lane == __ffs(here) - 1) {
      const int second = t >= before + x[0];
      picked = 2 * lane + second;
      target = t - before - (second ? x[0] : 0);
      use_p = none;
      z_all = all;
    }
  }
  __syncwarp();
  Team::arrive();  // this block has read the others' sums
  __syncthreads();
  // the block that holds the segment looks into it
  if (picked / kWarps == (int)rank) {
    const int64_t from = (int64_t)picked * each - shift;
    const int stop = (int)(from + each < V ? from + each : V);
    const float z_hi = (float)z_all * 0x1p-61f, z_lo = (float)((int64_t)z_all - fixed(z_hi)) * 0x1p-61f;
    float its = 0.f;
    const int found = look(src, w, table, from, stop, target, q && !use_p, z_hi, z_lo, use_p ? -1 : draft, scan, passes, its);
    if (found >= 0) {
      p.emitted[r] = found;
      if (p.logp) p.logp[r] = (its - row.x) * p.d.logit_scale - logf(row.y);
    }
  }
  Team::wait();  // the others have read this block's
}

// ---------------------------------------------------------------- one row a sequence
// Where no sequence has a draft (max_q is 1) the rows to draw from are known: one pass
// takes each row's weights in pieces of 1024, relative to the piece's own maximum, and
// the draw puts the pieces together.  Against the kernels above, which read the row
// twice: 256 rows of 50,003 in 20.5 us against 32.3.
constexpr int kOne = 1024, kOneShift = 11;  // weights of a piece are in units of 2^-61 of 2^11 times its largest
struct Part {
  uint64_t sum;
  float top;  // not finite: the row has no distribution; -infinity: the piece has no token
  uint32_t none;
};
static_assert(sizeof(Part) == 2 * sizeof(float2), "the workspace holds a Part in the place of two pairs");

__device__ __forceinline__ float nan_max(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float warp_nan_max(float x) {
  float y;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) one_rows_kernel(const VerifyParams p) {
  __shared__ float2 table[256];
  asm volatile("griddepcontrol.launch_dependents;");
  table[threadIdx.x] = kExp2.v[threadIdx.x];
  const int64_t part = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool in = part < p.d.total_q * p.chunks;
  const int64_t r = in ? part / p.chunks : 0;
  const int piece = (int)(part - r * p.chunks), lane = threadIdx.x & 31;
  const T* z = static_cast<const T*>(p.logits) + r * p.d.logits_stride;
  const int shift = (int)(reinterpret_cast<uintptr_t>(z) & 15) / (int)sizeof(T);
  const Source<T> src{z, nullptr, in ? p.d.vocab : 0, false};
  Raw8<T> x[kOne / 256];
#pragma unroll
  for (int i = 0; i < kOne / 256; ++i) x[i] = src.logits(piece * kOne - shift + i * 256 + lane * 8);
  __syncthreads();
  if (!in) return;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kOne / 256; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = nan_max(m, element(x[i], j));
  m = warp_nan_max(m);
  uint64_t sum = 0;
  if (m > -INFINITY && m < INFINITY) {
    const Row w = make_row(m, (float)kOne, p.c, p.c_low);
    float e0 = 0.f, e1 = 0.f;
#pragma unroll
    for (int i = 0; i < kOne / 256; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a, b;
        weight(element(x[i], j), w, table, a, b);
        const float a0 = on_grid(a);
        e0 += a0, e1 += (a - a0) + b;
      }
    sum = warp_sum((uint64_t)fixed(e0, e1));
  }
  if (lane == 0) {
    Part out;
    out.sum = sum, out.top = m, out.none = 0;
    reinterpret_cast<Part*>(p.parts)[part] = out;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) one_draw_kernel(const VerifyParams p) {
  __shared__ float2 table[256];
  __shared__ float tops[kWarps];
  __shared__ uint64_t scan[kWarps], target;
  __shared__ int most[kWarps], picked;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = p.d.vocab;
  table[tid] = kExp2.v[tid];
  const int64_t first = p.q_start[b], n = p.q_start[b + 1] - first;
  const bool bad = first < 0 || n < 0 || first + n > p.d.total_q || n > p.d.max_q;
  const float u = p.u_next[b];
  if (tid == 0) {
    if (bad) atomicOr(p.status, kStatusBadIndex);
    if (bad || n == 0) p.n_emitted[b] = 0;
    if (p.keep) p.keep[b] = p.kv_len[b];  // a row that is drawn from drops nothing
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are there, and who comes after this kernel comes after them
  if (bad || n == 0) return;
  const Part* parts = reinterpret_cast<const Part*>(p.parts) + first * p.chunks;
  const int each = (p.chunks + kThreads - 1) / kThreads, c0 = min(tid * each, p.chunks), c1 = min(c0 + each, p.chunks);
  float top = -INFINITY;
  for (int c = c0; c < c1; ++c) top = nan_max(top, parts[c].top);
  top = warp_nan_max(top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) top = nan_max(top, tops[i]);
  const bool some = top > -INFINITY && top < INFINITY;
  if (tid == 0) {
    p.n_emitted[b] = some;
    if (!some) {
      atomicOr(p.status, kStatusBadIndex);
      p.emitted[first] = -1;
      if (p.logp) p.logp[first] = 0.f;
    }
  }
  if (!some) return;
  const Row w = make_row(top, (float)V, p.c, p.c_low);  // units in which the whole row stays below 2^61
  auto weight_of = [&](int c) -> uint64_t {
    const Part x = parts[c];
    float a, b;
    weight(x.top, w, table, a, b);
    const uint64_t f = (uint64_t)fixed(a, b);
    return __umul64hi(x.sum, f) << (3 + kOneShift) | (x.sum * f) >> (61 - kOneShift);
  };
  uint64_t sum = 0;
  for (int c = c0; c < c1; ++c) sum += weight_of(c);
  uint64_t upto = warp_prefix(sum), total = 0;
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) upto += scan[i];
    total += scan[i];
  }
  const uint64_t t = part_of(u, total);
  if (t < upto && t >= upto - sum) {
    uint64_t run = upto - sum;
    for (int c = c0; c < c1; ++c) {
      const uint64_t x = weight_of(c);
      if (t < run + x) {
        picked = c, target = t - run;
        break;
      }
      run += x;
    }
  }
  __syncthreads();
  const T* z = static_cast<const T*>(p.logits) + first * p.d.logits_stride;
  const int shift = (int)(reinterpret_cast<uintptr_t>(z) & 15) / (int)sizeof(T);
  const Source<T> src{z, nullptr, V, false};
  const int64_t from = (int64_t)picked * kOne - shift;
  float its = 0.f;
  const int found = look(src, w, table, from, (int)(from + kOne < V ? from + kOne : V), target, false, 0.f, 0.f, -1, scan, most, its);
  if (found >= 0) {
    p.emitted[first] = found;
    if (p.logp)
      p.logp[first] = (its - top) * p.d.logit_scale - logf((float)total * 0x1p-61f / __uint_as_float(w.scale));
  }
}

}  // namespace

// Pieces of a row.
int verify_chunks(const ls_verify_desc& d) {
  if (d.max_q <= 1) return (int)(((int64_t)d.vocab + 7 + kOne - 1) / kOne);
  const int64_t bytes = (int64_t)d.vocab * (d.dtype == LS_DTYPE_F32 ? 4 : 2);
  return (int)((bytes + kChunkBytes - 1) / kChunkBytes);
}
size_t verify_scratch(const ls_verify_desc& d) {
  return (size_t)d.total_q * verify_chunks(d) * (d.max_q <= 1 ? sizeof(Part) : sizeof(float2));
}

cudaError_t launch_draft_verify(const VerifyParams& p, cudaStream_t s) {
  const bool wide = p.d.dtype == LS_DTYPE_F32, one = p.d.max_q <= 1;
  if (p.d.total_q > 0) {
    LaunchScope ls(kKVerifyRows, s);
    const unsigned grid = (unsigned)((p.d.total_q * p.chunks + kWarps - 1) / kWarps);
    auto kernel = one ? (wide ? one_rows_kernel<float> : one_rows_kernel<__nv_bfloat16>)
                      : (wide ? verify_rows_kernel<float> : verify_rows_kernel<__nv_bfloat16>);
    kernel<<<grid, kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls(kKVerifyDraw, s);
  // Blocks of a sequence: as many as let all sequences' run at once, four an SM.
  int blocks = one ? 1 : kMaxCluster;
  while (blocks > 1 && (int64_t)blocks * p.d.batch > 4 * device_sms()) blocks /= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = one ? dim3(p.d.batch) : dim3(blocks, p.d.batch), cfg.blockDim = dim3(kThreads), cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (p.d.total_q > 0) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (!one) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = blocks, at[n].val.clusterDim.y = 1, at[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = at, cfg.numAttrs = n;
  // A row's segments of more than kShort tiles (524,000 tokens over eight blocks, 65,000 over one) take the form that keeps
  // its float32 sums short; in it 64 x 5 rows of 128,000 take 29.2 us instead of 28.6, 310 x 2 of 152,064 160 instead of 157.
  const bool many = (int64_t)p.d.vocab + 7 > (int64_t)kShort * kTile * kWarps * blocks;
  auto kernel = one ? (wide ? one_draw_kernel<float> : one_draw_kernel<__nv_bfloat16>)
                : many ? (wide ? verify_draw_kernel<float, true> : verify_draw_kernel<__nv_bfloat16, true>)
                       : (wide ? verify_draw_kernel<float, false> : verify_draw_kernel<__nv_bfloat16, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace ls
