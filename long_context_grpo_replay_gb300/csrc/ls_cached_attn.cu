// Attention of new tokens over a paged cache: the float32 CUDA-core kernel
// for any mix of types, and the matrix-instruction kernel for few query rows.
//
//   x_ij = scale * q_i . k_j   (j < limit of row i),
//   o_i = sum_j exp(x_ij) v_j / sum_j exp(x_ij),  lse_i = log sum_j exp(x_ij).
//
// Rows of one (sequence, KV head) are its tokens' gq heads, so that every key
// is read once for all heads that share it.  The keys of a sequence are cut
// into parts over CTAs; each part gives a normalised o and an lse in float32,
// and one more kernel joins them exactly.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "ls_cached.cuh"
#include "ls_internal.h"

namespace ls {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A part's (or the whole) result of four columns of one row.
__device__ __forceinline__ void write_o4(const CachedParams& p, int part, int64_t row, int c, float4 v) {
  const int d = p.c.head_dim;
  if (p.ns > 1) {
    *reinterpret_cast<float4*>(p.o_parts + ((int64_t)part * p.total_q * p.hq + row) * d + c) = v;
  } else if (p.o_dtype == LS_DTYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * d + c) = v;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + row * d + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}
__device__ __forceinline__ void write_lse(const CachedParams& p, int part, int64_t row, float v) {
  if (p.ns > 1)
    p.lse_parts[(int64_t)part * p.total_q * p.hq + row] = v;
  else
    p.lse[row] = v;
}

// ===========================================================================
// CUDA-core kernel: float32 arithmetic for any cache format and query type.
// A CTA of four warps takes 16 rows and one part of the keys, 32 keys at a
// time in shared memory as float32; a warp owns four rows.  Scores: a lane
// owns a key; P V: a lane owns columns.  Bound by shared-memory reads; it is
// the float32 path and the plain one, not the fast one.
// ===========================================================================
constexpr int kSimtRows = 16, kSimtKeys = 32;

template <int FMT>
__device__ __forceinline__ float4 load_cache4(const void* pool, int64_t at, float s) {
  if constexpr (FMT == LS_CACHE_F32) {
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(pool) + at));
  } else if constexpr (FMT == LS_CACHE_BF16) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(pool) + at));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pool) + at));
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
    return make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
  }
}

template <typename TQ, int FMT>
__global__ void __launch_bounds__(128) cached_simt_kernel(const CachedParams p) {
  extern __shared__ float sm[];
  __shared__ int rows_s[kSimtKeys];
  __shared__ bool nan_s[kSimtKeys];  // e4m3: the value row is marked NaN
  const int d = p.c.head_dim, ks = d + 4;
  float* sq = sm;                        // [16][d]
  float* sk = sq + kSimtRows * d;        // [32][d + 4]
  float* sv = sk + kSimtKeys * ks;       // [32][d]
  const int b = blockIdx.z, kvh = blockIdx.y;
  // the kernel that joins the parts may be launched; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;");
  const int part = blockIdx.x % p.ns, tile = blockIdx.x / p.ns;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq s = load_seq(p, b, tid == 0 && kvh == 0 && blockIdx.x == 0);
  const int nrows = s.n * p.gq, r0 = tile * kSimtRows;
  if (r0 >= nrows) return;
  const int r1 = r0 + kSimtRows < nrows ? r0 + kSimtRows : nrows;
  int kb, ke;
  part_range(p, s, part, (r1 - 1) / p.gq, kb, ke);

  for (int x = tid * 4; x < kSimtRows * d; x += 128 * 4) {
    const int r = r0 + x / d;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < r1) {
      const int i = r / p.gq, hh = r - i * p.gq;
      const TQ* src = static_cast<const TQ*>(p.q) + (int64_t)(s.q0 + i) * p.q_stride + (int64_t)(kvh * p.gq + hh) * d + x % d;
      if constexpr (sizeof(TQ) == 4) {
        v = *reinterpret_cast<const float4*>(src);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                        __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
      }
    }
    *reinterpret_cast<float4*>(sq + x) = v;
  }
  int lim[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + warp * 4 + j;
    lim[j] = r < r1 ? row_limit(p, s, r / p.gq) : 0;
  }
  float m[4], l[4], acc[4][8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = -CUDART_INF_F;
    l[j] = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[j][c] = 0.f;
  }
  const int nc = d / 32;
  for (int k0 = kb; k0 < ke; k0 += kSimtKeys) {
    __syncthreads();  // the previous tile is used up
    if (tid < kSimtKeys) {
      const int row = k0 + tid < ke ? pool_row(p, b, kvh, k0 + tid) : -1;
      rows_s[tid] = row;
      if constexpr (FMT == LS_CACHE_E4M3) nan_s[tid] = row >= 0 && __ldg(p.c.v_exp + row) == -128;
    }
    __syncthreads();
    for (int x = tid * 4; x < kSimtKeys * d; x += 128 * 4) {
      const int key = x / d, c = x - key * d, row = rows_s[key];
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), v = a;
      if (row >= 0) {
        float ek = 1.f, ev = 1.f;
        if constexpr (FMT == LS_CACHE_E4M3) {
          ek = exp_scale(__ldg(p.c.k_exp + row));
          // a NaN row reaches only the rows that see it: through their weights
          ev = nan_s[key] ? 0.f : exp_scale(__ldg(p.c.v_exp + row));
        }
        a = load_cache4<FMT>(p.c.k, (int64_t)row * d + c, ek);
        v = load_cache4<FMT>(p.c.v, (int64_t)row * d + c, ev);
      }
      *reinterpret_cast<float4*>(sk + key * ks + c) = a;
      *reinterpret_cast<float4*>(sv + key * d + c) = v;
    }
    __syncthreads();
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < d; c += 4) {
      const float4 kk = *reinterpret_cast<const float4*>(sk + lane * ks + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 qq = *reinterpret_cast<const float4*>(sq + (warp * 4 + j) * d + c);
        x[j] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, x[j]))));
      }
    }
    const bool there = rows_s[lane] >= 0;
    if constexpr (FMT == LS_CACHE_E4M3) {
      if (nan_s[lane]) x[0] = x[1] = x[2] = x[3] = __int_as_float(0x7fffffff);
    }
    float pr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = there && k0 + lane < lim[j] ? x[j] * p.scale_log2 : -CUDART_INF_F;
      float top = y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m[j], top);
      pr[j] = 0.f;
      if (mn != -CUDART_INF_F) {
        const float alpha = exp2f(m[j] - mn);
        pr[j] = exp2f(y - mn);
        float sum = pr[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[j] = l[j] * alpha + sum;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] *= alpha;
        m[j] = mn;
      } else {
        // a score that is NaN leaves the maximum at -infinity: carry it
        float sum = y != y ? y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[j] += sum;
      }
    }
    for (int key = 0; key < kSimtKeys; ++key) {
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __shfl_sync(0xffffffffu, pr[j], key);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c >= nc) break;
        const float v = sv[key * d + c * 32 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j][c] = fmaf(w[j], v, acc[j][c]);
      }
    }
  }
  __syncthreads();
  // columns of a row are spread over the lanes: through shared memory for
  // 16-byte stores
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < nc) sq[(warp * 4 + j) * d + c * 32 + lane] = acc[j][c] * inv;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + warp * 4 + j;
    if (r >= r1) continue;
    const int i = r / p.gq, hh = r - i * p.gq;
    const int64_t row = (int64_t)(s.q0 + i) * p.hq + kvh * p.gq + hh;
    // an empty part's o is not read by the merge
    if (p.ns == 1 || l[j] != 0.f)
      for (int c = lane * 4; c < d; c += 128) {
        const float4 v = *reinterpret_cast<const float4*>(sq + (warp * 4 + j) * d + c);
        write_o4(p, part, row, c, v);
      }
    if (lane == 0)
      write_lse(p, part, row, l[j] == 0.f ? -CUDART_INF_F : m[j] == -CUDART_INF_F ? l[j] : (m[j] + log2f(l[j])) * kLn2);
  }
}

// ===========================================================================
// Matrix-instruction kernel for few rows (a decoding step, drafted tokens):
// bound by the cache's bytes, so it is built around the memory stream.
//
// A CTA has NW warps and one part of the keys; each warp streams its own
// blocks of 16 keys (block w, w + NW, ...) through its own ring of ST stages
// in shared memory with 16-byte asynchronous copies and keeps its own running
// maximum, sum and output, so the loop has no barrier wider than a warp.  The
// warps' results are joined once at the end.
//
// Keys are the M dimension of m16n8k16: S^T = K Q^T with eight query rows as
// N, so the six rows of a 24/4-head decoding step waste two columns of eight
// instead of ten of sixteen.  O^T = V^T P^T likewise; P^T is S^T's layout
// transposed, one movmatrix per eight keys.  Which dimension stands where
// inside a product is free as long as both operands agree, and is chosen so
// that a lane reads 16 contiguous bytes of its key's row.
//
// e4m3: codes become f16 (exact, one conversion per pair), the scales stay
// out of the products: K's multiplies the score, V's exponent is added to the
// score's exponent.  Per key (base 2, x_j the score, ev_j the value row's exponent)
//   w_j = 2^(x_j + ev_j - mo),   l = sum_j 2^(x_j - mx),   o = 2^(mo - mx) sum_j w_j code_j / l,
// with mo the running maximum of x_j + ev_j.  The softmax's sum has exponentials
// and a reference of its own, so that neither overflows or vanishes however far
// apart the value rows' scales are; each lane keeps its own mx, which float32 lets
// lag by 2^40.  The weights are f16, 2^11 times their value and at most 2^15 (mo
// moves once it is exceeded by 2^4): 11 bits down to 2^-25 of the largest.
// Queries go to f16 with a power of two per row taken out.
// bf16: the values as they are, P rounded to bf16 once.
//
// Measured (24/4 heads, d 256, e4m3): 1,000,003 keys in 300 us (6.85 TB/s, a copy's
// rate); 32 sequences up to 16,384 keys in 116.5 us (5.2 TB/s; 132 where every value
// row is zeros and is looked at); 8 sequences of 1 to 5 tokens over bf16 pages of 16,
// 8 x 128, in 38 us.
// ===========================================================================
template <bool E4>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  if constexpr (E4)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two pairs of e4m3 codes (low and high half of w) as two f16 pairs.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool E4>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (E4) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
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

// The maximum over the eight lanes that hold a block's keys for the same query rows.
__device__ __forceinline__ float key_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

template <int D, bool E4>
struct MmaShape {
  static constexpr int kRowBytes = D * (E4 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;      // 16-byte pieces of a row
  static constexpr int kStage = 2 * 16 * kRowBytes;   // K and V of 16 keys
  // two CTAs to an SM, so that one streams while the other starts or ends:
  // about 96 KB of ring each
  static constexpr int NW = kStage > 8192 ? 2 : 4;
  static constexpr int ST = kStage * NW * 6 <= 96 * 1024 ? 6 : 3;
  static constexpr int kRing = NW * ST * kStage;
  static constexpr int VD = E4 && D >= 128 ? 16 : 8;  // V columns of a lane's piece
  static constexpr int NU = D / (8 * VD);
};

template <int D, bool E4, int NT>
__global__ void __launch_bounds__(MmaShape<D, E4>::NW * 32, 2) cached_mma_kernel(const CachedParams p) {
  using L = MmaShape<D, E4>;
  constexpr int NW = L::NW, ST = L::ST, RB = L::kRowBytes, CPR = L::kChunks, VD = L::VD;
  constexpr int KS = D / 16;                 // products per score block, and m-tiles of O^T
  constexpr float kOff = E4 ? 11.f : 0.f;    // weights are held 2^kOff times their value
  constexpr float kSlack = 4.f, kSumSlack = 40.f;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int8_t exps[NW][ST][32];        // K exponents of 16 keys, V exponents of 16 keys
  __shared__ uint32_t there_s[NW][ST];       // which of the 16 keys exist
  __shared__ float3 ml[NW][8 * NT];          // reference of o, of the sum, the sum

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.z, kvh = blockIdx.y;
  // the kernel that joins the parts may be launched; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;");
  const int part = blockIdx.x % p.ns, tile = blockIdx.x / p.ns;
  const Seq s = load_seq(p, b, tid == 0 && kvh == 0 && blockIdx.x == 0);
  const int nrows = s.n * p.gq, r0 = tile * 8 * NT;
  if (r0 >= nrows) return;
  const int r1 = r0 + 8 * NT < nrows ? r0 + 8 * NT : nrows;
  int kb, ke;
  part_range(p, s, part, (r1 - 1) / p.gq, kb, ke);
  const int nblk = ke > kb ? (ke - kb + 15) / 16 : 0;

  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + warp * ST * L::kStage;
  const char* kp = static_cast<const char*>(p.c.k);
  const char* vp = static_cast<const char*>(p.c.v);

  // The pool row of key (lane & 15) of block blk, -1 past the end.
  auto lookup = [&](int blk) -> int {
    const int key = kb + blk * 16 + (lane & 15);
    return blk < nblk && key < ke ? pool_row(p, b, kvh, key) : -1;
  };
  auto issue = [&](int row, int st) {
    const uint32_t dk = base + st * L::kStage, dv = dk + 16 * RB;
#pragma unroll
    for (int j = 0; j < 16 * CPR / 32; ++j) {
      const int x = j * 32 + lane, r = x / CPR, c = x % CPR;
      const int rr = __shfl_sync(0xffffffffu, row, r);
      const int64_t off = (int64_t)(rr < 0 ? 0 : rr) * RB + c * 16;
      const int ck = CPR >= 8 ? c ^ ((r & 1) << 2) : c;
      const int cv = CPR >= 8 ? c ^ (r & 6) : c ^ ((r >> 1) & 3);
      copy16(dk + r * RB + ck * 16, kp + off, rr >= 0);
      copy16(dv + r * RB + cv * 16, vp + off, rr >= 0);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, row >= 0);
    if (lane == 0) there_s[warp][st] = mask;
  };
  auto load_exp = [&](int row) -> int8_t {
    if (!E4 || row < 0) return 0;
    return __ldg((lane < 16 ? p.c.k_exp : p.c.v_exp) + row);
  };

  // the first ST-1 blocks on their way before anything else is waited for
  int8_t first_exp[ST - 1];
  int row_next;
  {
    int rows[ST];
#pragma unroll
    for (int x = 0; x < ST; ++x) rows[x] = lookup(warp + x * NW);
#pragma unroll
    for (int x = 0; x < ST - 1; ++x) {
      issue(rows[x], x);
      copy_commit();
    }
#pragma unroll
    for (int x = 0; x < ST - 1; ++x) first_exp[x] = load_exp(rows[x]);
    row_next = rows[ST - 1];
  }

  // queries: B fragments of every product, and each row's factor and limit
  uint32_t qf[KS][NT][2];
  float crow[NT][2];
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + nt * 8 + g;
    const bool ok = r < r1;
    const int i = ok ? r / p.gq : 0, hh = ok ? r - i * p.gq : 0;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(s.q0 + i) * p.q_stride + (int64_t)(kvh * p.gq + hh) * D;
    uint2 w[KS];
    uint32_t top = 0;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int dim = E4 ? (kk / 4) * 64 + t * 16 + (kk % 4) * 4 : (kk / 2) * 32 + t * 8 + (kk % 2) * 4;
      w[kk] = ok ? *reinterpret_cast<const uint2*>(src + dim) : make_uint2(0u, 0u);
      if constexpr (E4) {
        top = max(top, max((w[kk].x << 16) & 0x7fffffffu, w[kk].x & 0x7fff0000u));
        top = max(top, max((w[kk].y << 16) & 0x7fffffffu, w[kk].y & 0x7fff0000u));
      }
    }
    float back = 1.f;
    if constexpr (E4) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row's largest element goes to [1, 4): exponent field of the factor
      int f = 254 - (int)(top >> 23);
      f = f < 1 ? 1 : f > 253 ? 253 : f;
      const float to = __int_as_float(f << 23);
      back = __int_as_float((254 - f) << 23);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        qf[kk][nt][0] = pack2<true>(__uint_as_float(w[kk].x << 16) * to, __uint_as_float(w[kk].x & 0xffff0000u) * to);
        qf[kk][nt][1] = pack2<true>(__uint_as_float(w[kk].y << 16) * to, __uint_as_float(w[kk].y & 0xffff0000u) * to);
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) qf[kk][nt][0] = w[kk].x, qf[kk][nt][1] = w[kk].y;
    }
    const int lm = ok ? row_limit(p, s, i) : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // of rows 2t and 2t+1, which this lane's scores belong to
      crow[nt][h] = __shfl_sync(0xffffffffu, back, (2 * t + h) * 4) * p.scale_log2;
      lim[nt][h] = __shfl_sync(0xffffffffu, lm, (2 * t + h) * 4);
    }
  }

  float o[NT][KS][4];
  float m[NT][2], mx[NT][2], l[NT][2];  // bf16: l is relative to m, mx is not used
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) m[nt][h] = mx[nt][h] = -CUDART_INF_F, l[nt][h] = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
  }

  // ring: ST-1 blocks ahead; a block's exponents are loaded with it and put
  // into shared memory one block later, its pool rows one block earlier, so
  // no load is waited for where it is issued
#pragma unroll
  for (int x = 0; x < ST - 1; ++x) exps[warp][x][lane] = first_exp[x];
  int8_t exp_next = 0;
  int st = 0, pend = -1;
  for (int blk = warp; blk < nblk; blk += NW) {
    copy_wait<ST - 2>();
    if (E4 && pend >= 0) exps[warp][pend][lane] = exp_next;
    __syncwarp();
    pend = st == 0 ? ST - 1 : st - 1;  // the stage used in the last turn
    issue(row_next, pend);
    copy_commit();
    exp_next = load_exp(row_next);
    row_next = lookup(blk + ST * NW);

    const uint32_t sk = base + st * L::kStage, sv = sk + 16 * RB;
    const uint32_t there = there_s[warp][st];
    float x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[nt][c] = 0.f;
#pragma unroll
    for (int u = 0; u < CPR / 4; ++u) {
      const int c = CPR >= 8 ? (4 * u + t) ^ ((g & 1) << 2) : 4 * u + t;
      const uint4 wa = lds16(sk + g * RB + c * 16), wb = lds16(sk + (g + 8) * RB + c * 16);
      const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, e[4] = {wb.x, wb.y, wb.z, wb.w};
      if constexpr (E4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          codes_f16(a[i], a0, a2);
          codes_f16(e[i], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16<true>(x[nt], a0, a1, a2, a3, qf[4 * u + i][nt][0], qf[4 * u + i][nt][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16<false>(x[nt], a[2 * i], e[2 * i], a[2 * i + 1], e[2 * i + 1], qf[2 * u + i][nt][0], qf[2 * u + i][nt][1]);
      }
    }
    // scores of keys g and g+8, rows 2t and 2t+1
    float ks[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f};
    if constexpr (E4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = exps[warp][st][16 + g + 8 * h];
        // a NaN row reaches only the rows that see it: through their scores
        ks[h] = exp_scale(e == -128 ? e : exps[warp][st][g + 8 * h]);
        ev[h] = (float)e;
      }
    }
    const int key = kb + blk * 16 + g;
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float y[2][2], top[2];  // [row][key half]
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool sees = (there >> (g + 8 * h) & 1u) && key + 8 * h < lim[nt][r];
          const float v = x[nt][2 * h + r] * (E4 ? crow[nt][r] * ks[h] : crow[nt][r]);
          y[r][h] = sees ? v : -CUDART_INF_F;
        }
        if constexpr (E4) {
          const float tx = fmaxf(y[r][0], y[r][1]), nx = tx > mx[nt][r] + kSumSlack ? tx : mx[nt][r];
          const float at = nx == -CUDART_INF_F ? 0.f : nx;
          l[nt][r] = fmaf(l[nt][r], ex2(mx[nt][r] - at), ex2(y[r][0] - at) + ex2(y[r][1] - at));
          mx[nt][r] = nx;
          y[r][0] += ev[0], y[r][1] += ev[1];
        }
        top[r] = key_max(fmaxf(y[r][0], y[r][1]));
      }
      if (__any_sync(0xffffffffu, top[0] > m[nt][0] + kSlack || top[1] > m[nt][1] + kSlack)) {
        if constexpr (E4) {
          // A value row of zeros, which the cache holds with exponent 0, adds nothing to
          // o and must not raise the reference (below it, its weight is harmless).
          const uint32_t none = __ballot_sync(0xffffffffu, exps[warp][st][lane] == 0) >> 16 & there;
          if (none) {
            uint32_t zeros = 0;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint32_t any = 0;
#pragma unroll 4
              for (int c = t; c < CPR; c += 4) {
                const uint4 z = lds16(sv + (g + 8 * h) * RB + c * 16);
                any |= z.x | z.y | z.z | z.w;
              }
              any |= __shfl_xor_sync(0xffffffffu, any, 1);
              any |= __shfl_xor_sync(0xffffffffu, any, 2);
              if ((none >> (g + 8 * h) & 1u) && (any & 0x7f7f7f7fu) == 0) zeros |= 1u << h;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (zeros & 1u) y[r][0] = -CUDART_INF_F;
              if (zeros & 2u) y[r][1] = -CUDART_INF_F;
              top[r] = key_max(fmaxf(y[r][0], y[r][1]));
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (!(top[r] > m[nt][r] + kSlack)) continue;
          const float alpha = ex2(m[nt][r] - top[r]);
          m[nt][r] = top[r];
          if constexpr (!E4) l[nt][r] *= alpha;
#pragma unroll
          for (int i = 0; i < KS; ++i) o[nt][i][r] *= alpha, o[nt][i][2 + r] *= alpha;
        }
      }
      float w[2][2];  // [key half][row]
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // where no key is seen yet the maximum stands at 0, so that -infinity
        // gives a weight of 0 and a NaN stays one
        const float ref = (m[nt][r] == -CUDART_INF_F ? 0.f : m[nt][r]) - kOff;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[h][r] = ex2(y[r][h] - ref);
          if constexpr (!E4) l[nt][r] += w[h][r];
        }
      }
      pb[nt][0] = transpose8(pack2<E4>(w[0][0], w[0][1]));
      pb[nt][1] = transpose8(pack2<E4>(w[1][0], w[1][1]));
    }
#pragma unroll
    for (int u = 0; u < L::NU; ++u) {
      uint32_t v[4][4];  // keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 2 * t + (q & 1) + (q >> 1) * 8;
        if constexpr (VD * (E4 ? 1 : 2) == 16) {
          const uint4 z = lds16(sv + r * RB + (((g + 8 * u) ^ (r & 6)) * 16));
          v[q][0] = z.x, v[q][1] = z.y, v[q][2] = z.z, v[q][3] = z.w;
        } else {  // 64 e4m3 columns: eight to a lane
          const uint2 z = lds8(sv + r * RB + (((g >> 1) ^ ((r >> 1) & 3)) * 16) + (g & 1) * 8);
          v[q][0] = z.x, v[q][1] = z.y, v[q][2] = v[q][3] = 0u;
        }
      }
      if constexpr (E4) {
#pragma unroll
        for (int i = 0; i < VD / 4; ++i) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t a0, a1, a2, a3;
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            codes_f16(__byte_perm(v[0][i], v[1][i], sel), a0, a1);
            codes_f16(__byte_perm(v[2][i], v[3][i], sel), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16<true>(o[nt][u * (VD / 2) + 2 * i + half], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410), a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
          const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410), a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16<false>(o[nt][u * 4 + i], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      }
    }
    st = st == ST - 1 ? 0 : st + 1;
  }

  // join the warps' results: [warp][row][D] in the ring, which no copy writes any more
  copy_wait<0>();
  __syncthreads();
  constexpr int OS = D + 4;
  float* so = reinterpret_cast<float*>(ring);
  static_assert(NW * 8 * NT * OS * 4 <= L::kRing, "the warps' results fit the ring");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // each lane's sum is relative to a reference of its own (e4m3)
      float top = E4 ? mx[nt][r] : m[nt][r], sum = l[nt][r];
      if constexpr (E4) {
        top = key_max(top);
        if (mx[nt][r] != -CUDART_INF_F) sum *= ex2(mx[nt][r] - top);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int row = nt * 8 + 2 * t + r;
      if (g == 0) ml[warp][row] = make_float3(m[nt][r], top, sum);
      float* dst = so + (warp * 8 * NT + row) * OS;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int dim = (i / (VD / 2)) * 8 * VD + g * VD + (i % (VD / 2)) * 2;
        *reinterpret_cast<float2*>(dst + dim) = make_float2(o[nt][i][r], o[nt][i][2 + r]);
      }
    }
  }
  __syncthreads();
  for (int x = tid; x < (r1 - r0) * (D / 4); x += NW * 32) {
    const int row = x / (D / 4), c = (x % (D / 4)) * 4;
    float top = -CUDART_INF_F, topx = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w][row].x), topx = fmaxf(topx, ml[w][row].y);
    const float ref = top == -CUDART_INF_F ? 0.f : top, refx = topx == -CUDART_INF_F ? 0.f : topx;
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float3 a = ml[w][row];
      // a warp that saw no key has a weight of 0, but passes a NaN on
      const float f = a.x == -CUDART_INF_F ? 0.f : ex2(a.x - ref), fx = a.y == -CUDART_INF_F ? 1.f : ex2(a.y - refx);
      const float4 z = *reinterpret_cast<const float4*>(so + (w * 8 * NT + row) * OS + c);
      sum = fmaf(fx, a.z, sum);
      v.x = fmaf(f, z.x, v.x), v.y = fmaf(f, z.y, v.y), v.z = fmaf(f, z.z, v.z), v.w = fmaf(f, z.w, v.w);
    }
    const int r = r0 + row, i = r / p.gq, hh = r - i * p.gq;
    const int64_t out = (int64_t)(s.q0 + i) * p.hq + kvh * p.gq + hh;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    // from o's reference to the sum's, by halves: the whole may pass float32's range
    const float to = top == -CUDART_INF_F ? 1.f : ex2(0.5f * (ref - kOff - refx));
    v.x = v.x * inv * to * to, v.y = v.y * inv * to * to, v.z = v.z * inv * to * to, v.w = v.w * inv * to * to;
    if (p.ns == 1 || sum != 0.f) write_o4(p, part, out, c, v);
    if (c == 0) write_lse(p, part, out, sum == 0.f ? -CUDART_INF_F : (refx + log2f(sum)) * kLn2);
  }
}

__device__ __forceinline__ void store_joined(int o_dtype, void* o, int64_t at, float4 v) {
  if (o_dtype == LS_DTYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(o) + at) = v;
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
}

// ===========================================================================
// Joins the parts of each row exactly: o = sum_s w_s o_s / sum_s w_s with
// w_s = exp(lse_s - max).  A CTA has one row; its threads take four columns
// each and share the parts in groups, so that the few rows of a decoding step
// still have many loads in flight.  Parts without keys (lse -infinity, o not
// written) are skipped; a NaN part makes the row NaN.  The kernel is there while the
// parts are still being written: it reads them by ordinary loads, which the wait's
// memory clobber keeps behind it (not as data that nothing writes while it runs).
// ===========================================================================
__global__ void __launch_bounds__(256) cached_join_kernel(int ns, int64_t n_rows, int d, const float* o_parts,
                                                          const float* lse_parts, int o_dtype, void* o,
                                                          float* lse) {
  __shared__ float w[kCachedMaxParts], total_s;
  __shared__ float4 acc_s[256];
  // launched while the parts' kernel still runs: wait for its results
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, cols = d >> 2, groups = 256 / cols;
  if (tid < 32) {
    float v[4], top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = tid + 32 * i;
      v[i] = s < ns ? lse_parts[(int64_t)s * n_rows + row] : -CUDART_INF_F;
      top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = expf(v[i] - ref);
      w[tid + 32 * i] = f;
      sum += f;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (tid == 0) {
      total_s = sum;
      lse[row] = sum == 0.f ? -CUDART_INF_F : ref + logf(sum);
    }
  }
  __syncthreads();
  const int c = (tid % cols) * 4, group = tid / cols;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = group; s < ns; s += groups) {
    const float f = w[s];
    if (f == 0.f) continue;
    const float4 z = *reinterpret_cast<const float4*>(o_parts + ((int64_t)s * n_rows + row) * d + c);
    a.x = fmaf(f, z.x, a.x), a.y = fmaf(f, z.y, a.y), a.z = fmaf(f, z.z, a.z), a.w = fmaf(f, z.w, a.w);
  }
  acc_s[tid] = a;
  __syncthreads();
  if (group != 0) return;
  for (int i = 1; i < groups; ++i) {
    const float4 z = acc_s[tid + i * cols];
    a.x += z.x, a.y += z.y, a.z += z.z, a.w += z.w;
  }
  const float inv = total_s == 0.f ? 0.f : 1.f / total_s;
  store_joined(o_dtype, o, row * d + c, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
}

// The same for many rows and few parts: one thread per four columns, which
// reads its row's few weights itself.
__global__ void __launch_bounds__(256) cached_join_rows_kernel(int ns, int64_t n_rows, int d, const float* o_parts,
                                                               const float* lse_parts, int o_dtype, void* o,
                                                               float* lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cols = d >> 2, c = (int)(threadIdx.x % cols) * 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / cols) + threadIdx.x / cols;
  if (row >= n_rows) return;
  float top = -CUDART_INF_F;
  for (int s = 0; s < ns; ++s) top = fmaxf(top, lse_parts[s * n_rows + row]);
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    const float f = expf(lse_parts[s * n_rows + row] - ref);
    sum += f;
    if (f == 0.f) continue;
    const float4 z = *reinterpret_cast<const float4*>(o_parts + (s * n_rows + row) * d + c);
    a.x = fmaf(f, z.x, a.x), a.y = fmaf(f, z.y, a.y), a.z = fmaf(f, z.z, a.z), a.w = fmaf(f, z.w, a.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  store_joined(o_dtype, o, row * d + c, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
  if (c == 0) lse[row] = sum == 0.f ? -CUDART_INF_F : ref + logf(sum);
}

template <int D, bool E4, int NT>
cudaError_t run_mma(const CachedParams& p, cudaStream_t s) {
  using L = MmaShape<D, E4>;
  cudaError_t e = cudaFuncSetAttribute(cached_mma_kernel<D, E4, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kRing);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)p.max_q * p.gq + 8 * NT - 1) / (8 * NT);
  if (tiles * p.ns > INT32_MAX) return cudaErrorInvalidConfiguration;
  LaunchScope ls(kKCachedMma, s);
  cached_mma_kernel<D, E4, NT><<<dim3((unsigned)(tiles * p.ns), p.c.hkv, p.batch), L::NW * 32, L::kRing, s>>>(p);
  return cudaGetLastError();
}

// Most rows that this kernel takes; more go to cached_tc_kernel.  By time (24/4 heads
// for d 256, 32/8 else), this kernel against that one, for one sequence of 100,000
// keys, 8 of 12,000 and one of 3,000.  At the most rows: e4m3, d 256, 12 rows: 68
// against 72 us, 61 against 90, 20 and 20; d 128, 24 rows: 74 against 86, 90 against
// 123, 20 and 20; d 64, 32 rows: 66 against 78, 72 against 113, 18 and 18.  bf16, d
// 256, 6 rows: 96 against 90, 90 against 98, 16 against 18; d 128, 24 rows: 96 against
// 88, 102 against 107, 18 and 18; d 64, 16 rows: 55 against 59, 57 against 90, 14
// against 16.  Beyond, on 100,000 keys: e4m3, d 256, 18 rows 86 against 72; d 128, 28
// rows 117 against 84; d 64, 48 rows 104 against 74; bf16, d 128, 28 rows 121 against 88.
template <int D, bool E4>
constexpr int kMmaRows = E4 ? (D == 256 ? 16 : D == 128 ? 24 : 32) : (D == 256 ? 8 : D == 128 ? 24 : 16);

// Tiles of as many rows as there are, in eights.
template <int D, bool E4>
cudaError_t run_mma_d(const CachedParams& p, cudaStream_t s) {
  constexpr int kMost = kMmaRows<D, E4>;
  const int64_t rows = (int64_t)p.max_q * p.gq;
  if (rows <= 8) return run_mma<D, E4, 1>(p, s);
  if constexpr (kMost > 8)
    if (rows <= 16) return run_mma<D, E4, 2>(p, s);
  if constexpr (kMost > 16)
    if (rows <= kMost) return run_mma<D, E4, kMost / 8>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace

int cached_mma_rows(int d, int format) {
  const bool e4 = format == LS_CACHE_E4M3;
  switch (d) {
    case 64: return e4 ? kMmaRows<64, true> : kMmaRows<64, false>;
    case 128: return e4 ? kMmaRows<128, true> : kMmaRows<128, false>;
    default: return e4 ? kMmaRows<256, true> : kMmaRows<256, false>;
  }
}

cudaError_t launch_cached_mma(const CachedParams& p, cudaStream_t s) {
  const bool e4 = p.c.format == LS_CACHE_E4M3;
  switch (p.c.head_dim) {
    case 64: return e4 ? run_mma_d<64, true>(p, s) : run_mma_d<64, false>(p, s);
    case 128: return e4 ? run_mma_d<128, true>(p, s) : run_mma_d<128, false>(p, s);
    default: return e4 ? run_mma_d<256, true>(p, s) : run_mma_d<256, false>(p, s);
  }
}

cudaError_t launch_cached_join(const CachedParams& p, cudaStream_t s) {
  LaunchScope ls(kKCachedJoin, s);
  const int64_t rows = p.total_q * p.hq;
  cudaLaunchConfig_t cfg{};
  // a CTA a row where rows are few; from four rows an SM on, as many rows as a
  // CTA's threads have columns for (49,152 rows of 256, 3 parts: 90 -> 36 us)
  const bool few = rows < 4 * (int64_t)device_sms() || p.ns > 16;
  const int64_t per = few ? 1 : 256 / (p.c.head_dim / 4);
  cfg.gridDim = dim3((unsigned)((rows + per - 1) / per));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? cached_join_kernel : cached_join_rows_kernel, (int)p.ns, rows, (int)p.c.head_dim, (const float*)p.o_parts,
                            (const float*)p.lse_parts, (int)p.o_dtype, p.o, p.lse);
}

cudaError_t launch_cached_simt(const CachedParams& p, cudaStream_t s) {
  const int d = p.c.head_dim;
  const int smem = (kSimtRows * d + kSimtKeys * (d + 4) + kSimtKeys * d) * (int)sizeof(float);
  const int64_t tiles = ((int64_t)p.max_q * p.gq + kSimtRows - 1) / kSimtRows;
  if (tiles * p.ns > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tiles * p.ns), p.c.hkv, p.batch);
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchScope ls(kKCachedSimt, s);
    kernel<<<grid, 128, smem, s>>>(p);
    return cudaGetLastError();
  };
  if (p.q_dtype == LS_DTYPE_F32) {
    if (p.c.format == LS_CACHE_E4M3) return go(cached_simt_kernel<float, LS_CACHE_E4M3>);
    if (p.c.format == LS_CACHE_BF16) return go(cached_simt_kernel<float, LS_CACHE_BF16>);
    return go(cached_simt_kernel<float, LS_CACHE_F32>);
  }
  if (p.c.format == LS_CACHE_E4M3) return go(cached_simt_kernel<__nv_bfloat16, LS_CACHE_E4M3>);
  if (p.c.format == LS_CACHE_BF16) return go(cached_simt_kernel<__nv_bfloat16, LS_CACHE_BF16>);
  return go(cached_simt_kernel<__nv_bfloat16, LS_CACHE_F32>);
}

}  // namespace ls
