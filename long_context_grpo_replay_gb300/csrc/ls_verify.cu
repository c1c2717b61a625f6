// Verification of drafted tokens against the target's logits, and the draw of
// the token after them.
//
//   p_r(v) = exp(s z_rv - lse_r);  a draft x is accepted while u_r q_r(x) < p_r(x);
//   next token: least v with sum_{j<=v} w_j > u sum_j w_j,  w = max(p - q, 0) or p.
//
// Two kernels.  verify_rows_kernel reads every logit once: a (maximum, sum) pair
// for each row and 16 KB of it, in base 2.  verify_draw_kernel, a cluster of eight
// blocks for each sequence, joins them, tests the drafts and draws from the one
// row where they end.
//
// The draw compares u with a running sum that has a step for every token, 10^5
// of them in [0, 1): with sums good to 2^-24 one draw in a hundred would give a
// neighbour of the definition's token.  So the draw's weights are formed anew as
// integers in units of about 2^-61, whose sums do not depend on their order:
//   w = 2^(n + j/256) (1 + d),  s log2(e) (z - max) = n + j/256 + r, |r| <= 2^-9,
//   d = 2^r - 1 by three terms (the fourth is below 2^-42),
// the argument as a pair of floats (a difference and a product with their exact
// remainders), 2^(j/256) from a table (Tang's method: P. T. P. Tang, Table-driven
// implementation of the exponential function, ACM TOMS 15, 1989), d in float32:
// at most 2^-31 of each weight (2^-34.6 on average).  After a rejection w = max(e - q Z, 0) needs Z, the sum of
// all e, before the first of them is known: the pass takes the row's float32 sum
// Z0, and as Z is within 2^-20 of it, each partial sum is put right afterwards by
// (Z - Z0) times the sum of its q where e > q Z0 (tokens within 2^-20 of that
// border weigh 2^-20 of theirs, so that their side does not matter).
#include <cuda_bf16.h>

#include "ls_cluster.cuh"
#include "ls_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunkBytes = 16384, kVectors = kChunkBytes / 16, kEach = kVectors / kThreads;
constexpr int kCluster = 8, kSegments = kCluster * kWarps;

// ---------------------------------------------------------------- 2^(j/256)
struct Table {
  uint64_t v[256];
};
// 2^(j/256) * 2^61, from square roots of 2 in integers (each off by less than 2^-60).
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
    t.v[j] = (y + 1) >> 1;
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

__device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}

// Block (row, chunk).  A row starts anywhere: its 16-byte pieces are dealt out to
// the chunks, the elements before the first and after the last go to chunk 0.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_rows_kernel(const VerifyParams p) {
  constexpr int E = 16 / sizeof(T);
  __shared__ float2 warps[kWarps];
  const int chunk = blockIdx.x % p.chunks, tid = threadIdx.x;
  const int64_t r = blockIdx.x / p.chunks;
  const T* row = static_cast<const T*>(p.logits) + r * p.d.logits_stride;
  const int before = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
  const int head = before < p.d.vocab ? before : p.d.vocab;
  const int vectors = (p.d.vocab - head) / E, tail = p.d.vocab - head - vectors * E;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  uint4 w[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = chunk * kVectors + i * kThreads + tid;
    if (at < vectors) w[i] = __ldcs(body + at);
  }
  float2 a = make_float2(-INFINITY, 0.f);
  if (chunk == 0) {
    float z = -INFINITY;
    if (tid < head) z = value(row[tid]);
    if (tid >= 32 && tid < 32 + tail) z = value(row[head + vectors * E + tid - 32]);
    a = make_float2(z, z == -INFINITY ? 0.f : z - z + 1.f);  // NaN for NaN and +infinity
  }
  float m = a.x;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (chunk * kVectors + i * kThreads + tid < vectors) {
      float x[E];
      unpack(w[i], x);
#pragma unroll
      for (int e = 0; e < E; ++e) m = fmaxf(m, x[e]);
    }
  const float base = m == -INFINITY ? 0.f : m;
  float sum = a.y * ex2((a.x - base) * p.c);
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (chunk * kVectors + i * kThreads + tid < vectors) {
      float x[E];
      unpack(w[i], x);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += ex2((x[e] - base) * p.c);
    }
  a = join_warp(make_float2(m, sum), p.c);
  if ((tid & 31) == 0) warps[tid >> 5] = a;
  __syncthreads();
  if (tid < 32) {
    a = join_warp(tid < kWarps ? warps[tid] : make_float2(-INFINITY, 0.f), p.c);
    if (tid == 0) p.parts[blockIdx.x] = a;
  }
}

// ---------------------------------------------------------------- the draw
struct Row {
  float top;      // the row's maximum
  float c, c_low;
  int32_t k;      // weights are e * 2^(61 - k), Z in [2^60, 2^61) of them
  uint32_t z0;    // 24 bits: Z0 = z0 * 2^37
};

// e = 2^(c (z - top)) in the row's units.
__device__ __forceinline__ uint64_t weight(float z, const Row& r, const uint64_t* table) {
  const float s = z - r.top, back = s - z, rest = (z - (s - back)) - (r.top + back);
  const float hi = s * r.c;
  if (!(hi > -62.f)) return 0;
  const float lo = fmaf(s, r.c, -hi) + fmaf(s, r.c_low, rest * r.c);
  const float t = hi + 49152.f;  // 1.5 * 2^15: rounds to a multiple of 2^-8
  const int k = __float_as_int(t) - __float_as_int(49152.f);
  const float f = (hi - (t - 49152.f)) + lo;
  const uint64_t w = table[k & 255];
  const float d = f * fmaf(f, fmaf(f, 0.0555041087f, 0.240226507f), 0.693147181f);  // 2^f - 1: powers of ln 2
  const float wide = __uint_as_float(0x3f000000u + (uint32_t)(w >> 38));            // the table's value in [1, 2)
  const int64_t more = (int64_t)__float2int_rn(d * wide * 0x1p39f) << 22;
  const int shift = r.k - (k >> 8);
  return shift > 63 ? 0 : (w + more) >> shift;
}

// q as m * 2^(e - 150); not a number below 2 (or NaN): more than any weight.
struct Share {
  uint32_t m;
  int32_t e;
};
__device__ __forceinline__ Share share(float q) {
  const uint32_t u = __float_as_uint(q), e = u >> 23;
  Share s;
  s.e = (int32_t)e;
  s.m = e == 0 || e > 255 ? 0 : (u & 0x7fffffu) | 0x800000u;  // below 2^-126, or with a sign: 0
  return s;
}
__device__ __forceinline__ int64_t times_z0(Share q, uint32_t z0) {
  if (q.m == 0) return 0;
  if (q.e >= 128) return INT64_MAX;
  const uint64_t x = (uint64_t)q.m * z0;
  const int shift = q.e - 113;
  return shift >= 0 ? (int64_t)(x << shift) : shift < -63 ? 0 : (int64_t)(x >> -shift);
}
__device__ __forceinline__ int64_t times_z(Share q, uint64_t z) {
  if (q.m == 0) return 0;
  if (q.e >= 128) return INT64_MAX;
  const uint64_t x = __umul64hi((uint64_t)q.m << 40, z);
  const int shift = q.e - 126;
  return shift >= 0 ? (int64_t)(x << shift) : shift < -63 ? 0 : (int64_t)(x >> -shift);
}

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

// Four elements from p, or fewer before `end`, as floats (zeros after it).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int at, int end, bool whole, float (&x)[4]) {
  if (whole && at + 4 <= end) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + at);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(p + at);
      x[0] = __uint_as_float(a.x << 16), x[1] = __uint_as_float(a.x & 0xffff0000u);
      x[2] = __uint_as_float(a.y << 16), x[3] = __uint_as_float(a.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = at + i < end ? value(p[at + i]) : 0.f;
  }
}

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) verify_draw_kernel(const VerifyParams p) {
  using Team = Cluster<kCluster>;
  __shared__ uint64_t table[256];
  __shared__ float2 row_of[kWarps];
  __shared__ int passes[kWarps];
  __shared__ uint64_t seg_e[kWarps], seg_w[kWarps], scan[kWarps];
  __shared__ float seg_q[kWarps];
  __shared__ int picked, use_p;
  __shared__ uint64_t target, z_all;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = Team::rank();
  table[tid] = kExp2.v[tid];
  const int64_t first = p.q_start[b], n64 = p.q_start[b + 1] - first;
  const bool bad = first < 0 || n64 < 0 || first + n64 > p.d.total_q || n64 > p.d.max_q;
  if (bad || n64 == 0) {  // all blocks of the cluster
    if (rank == 0 && tid == 0) {
      if (bad) atomicOr(p.status, kStatusBadIndex);
      p.n_emitted[b] = 0;
      if (p.keep) p.keep[b] = p.kv_len[b];
    }
    return;
  }
  const int n = (int)n64, V = p.d.vocab;
  const T* logits = static_cast<const T*>(p.logits);
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
      if (i + 1 < n) {
        const int64_t x = p.tokens[r + 1];
        if (x >= 0 && x < V) {
          const float d = value(logits[r * p.d.logits_stride + x]) - a.x;
          const double e = exp2f(fmaf(d, p.c, d * p.c_low));
          const double q = p.probs ? p.probs[r * p.d.draft_stride + x] : 1.f;
          pass = (double)p.u[r] * q * a.y < e;
          if (pass && rank == 0 && lane == 0) {
            p.emitted[r] = x;
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
  Row w;
  w.top = row.x, w.c = p.c, w.c_low = p.c_low;
  w.k = (int)(__float_as_uint(row.y) >> 23) - 126;
  w.z0 = (__float_as_uint(row.y) & 0x7fffffu) | 0x800000u;
  const T* z = logits + r * p.d.logits_stride;
  const float* q = p.probs && rejected ? p.probs + r * p.d.draft_stride : nullptr;
  const int64_t draft = rejected && !p.probs ? p.tokens[r + 1] : -1;
  const bool whole = (reinterpret_cast<uintptr_t>(z) & (4 * sizeof(T) - 1)) == 0 && (reinterpret_cast<uintptr_t>(q) & 15) == 0;
  // each warp its segment
  const int each = (V + kSegments * 128 - 1) / (kSegments * 128) * 128;
  {
    const int64_t lo = (int64_t)((int)rank * kWarps + warp) * each;
    const int end = (int)(lo + each < V ? lo + each : V);
    uint64_t sum_e = 0, sum_w = 0;
    float sum_q = 0.f;
    for (int64_t at = lo + lane * 4; at < end; at += 128) {
      float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
      load4(z, (int)at, end, whole, x);
      if (q) load4(q, (int)at, end, whole, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at + i >= end) continue;
        const uint64_t e = weight(x[i], w, table);
        sum_e += e;
        if (q) {
          const int64_t over = (int64_t)e - times_z0(share(y[i]), w.z0);
          if (over > 0) sum_w += (uint64_t)over, sum_q += y[i];
        } else if (at + i != draft) {
          sum_w += e;
        }
      }
    }
    sum_e = warp_sum(sum_e), sum_w = warp_sum(sum_w), sum_q = warp_sum(sum_q);
    if (lane == 0) seg_e[warp] = sum_e, seg_w[warp] = sum_w, seg_q[warp] = sum_q;
  }
  Team::sync();
  if (warp == 0) {  // two segments a lane, neighbours
    uint64_t e[2], x[2];
    float sq[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = 2 * lane + i;
      e[i] = Team::at(seg_e + s % kWarps, s / kWarps);
      x[i] = Team::at(seg_w + s % kWarps, s / kWarps);
      sq[i] = Team::at(seg_q + s % kWarps, s / kWarps);
    }
    const uint64_t all = warp_sum(e[0] + e[1]);
    const float off = (float)((int64_t)all - ((int64_t)w.z0 << 37));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t fixed = q ? (int64_t)x[i] - __float2ll_rn(off * sq[i]) : (int64_t)x[i];
      x[i] = fixed > 0 ? (uint64_t)fixed : 0;
    }
    const bool none = warp_sum(x[0] + x[1]) < (1ull << 31);  // of 2^61: rounding alone
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
  __syncthreads();
  // the block that holds the segment looks into it
  if (picked / kWarps == (int)rank) {
    const int64_t lo64 = (int64_t)picked * each;
    const int lo = (int)lo64, end = (int)(lo64 + each < V ? lo64 + each : V);
    const int per = (each + kThreads - 1) / kThreads;
    const uint64_t all = z_all;
    auto weigh = [&](int v) -> uint64_t {
      const uint64_t e = weight(value(z[v]), w, table);
      if (use_p) return e;
      if (q) {
        const int64_t over = (int64_t)e - times_z(share(q[v]), all);
        return over > 0 ? (uint64_t)over : 0;
      }
      return v == draft ? 0 : e;
    };
    uint64_t sum = 0;
    int last = -1;  // the last token of this thread's that weighs anything
    const int a0 = lo + tid * per, a1 = a0 + per < end ? a0 + per : end;
    for (int v = a0; v < a1; ++v) {
      const uint64_t x = weigh(v);
      if (x) last = v;
      sum += x;
    }
    uint64_t upto = warp_prefix(sum);
    if (lane == 31) scan[warp] = upto;
    passes[warp] = __reduce_max_sync(0xffffffffu, last);
    __syncthreads();
    uint64_t total = 0;
    int most = -1;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) upto += scan[i];
      total += scan[i];
      most = max(most, passes[i]);
    }
    // the segment's own sum may differ from the corrected one by rounding: its last token then
    const uint64_t t = target < total ? target : total - 1;
    int found = -1;
    if (total == 0) {
      if (tid == 0) found = lo;
    } else if (t < upto && t >= upto - sum) {
      uint64_t run = upto - sum;
      for (int v = a0; v < a1 && found < 0; ++v) {
        run += weigh(v);
        if (run > t) found = v;
      }
      if (found < 0) found = most;
    }
    if (found >= 0) {
      p.emitted[r] = found;
      if (p.logp) p.logp[r] = (value(z[found]) - w.top) * p.d.logit_scale - logf(row.y);
    }
  }
  Team::sync();  // the sums are read by other blocks
}

}  // namespace

int verify_chunks(const ls_verify_desc& d) {
  const int64_t bytes = (int64_t)d.vocab * (d.dtype == LS_DTYPE_F32 ? 4 : 2);
  return (int)((bytes + kChunkBytes - 1) / kChunkBytes);
}

cudaError_t launch_draft_verify(const VerifyParams& p, cudaStream_t s) {
  if (p.d.total_q > 0) {
    LaunchScope ls(kKVerifyRows, s);
    const unsigned grid = (unsigned)(p.d.total_q * p.chunks);
    if (p.d.dtype == LS_DTYPE_F32)
      verify_rows_kernel<float><<<grid, kThreads, 0, s>>>(p);
    else
      verify_rows_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls(kKVerifyDraw, s);
  const dim3 grid(kCluster, p.d.batch);
  if (p.d.dtype == LS_DTYPE_F32)
    verify_draw_kernel<float><<<grid, kThreads, 0, s>>>(p);
  else
    verify_draw_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ls
