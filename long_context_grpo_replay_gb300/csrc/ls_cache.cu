// The quantised K/V cache: rows written into page slots as e4m3 codes with a
// power-of-two scale per row and KV head, and read back by slot.
//
//   e = min { e >= -126 : max|x| <= 448 * 2^e },  code = rne_e4m3(x * 2^-e),
//   value = code * 2^e.
//
// A power of two costs nothing in precision, because e4m3 keeps its relative
// precision over 15 binades, and makes both directions exact but for the one
// rounding of the code: x * 2^-e never rounds in float32 where the code is
// not zero, and code * 2^e is a bf16 number.  The scale is one byte a row.
//
// Both kernels only move bytes: a group of lanes takes a token's K and V row of
// one head (writing: sixteen elements a lane, so that codes leave in 16-byte
// pieces; reading: eight), all loads before the first use.  A row's maximum is
// log2 of the group's lanes in shuffles; no shared memory.  Measured: 131,075
// tokens of 4 x 256 written from bf16 in 129 us (6.25 TB/s), 60,001 read to bf16
// in 61.5 us (6.0 TB/s); a copy runs at 6.75.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ls_internal.h"

namespace ls {
namespace {

constexpr int8_t kNanRow = -128;  // exponent of a row that held an infinity or a NaN

struct Row8 {
  float x[8];
};

__device__ __forceinline__ Row8 load8(const float* p) {
  Row8 r;
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  r.x[0] = a.x, r.x[1] = a.y, r.x[2] = a.z, r.x[3] = a.w;
  r.x[4] = b.x, r.x[5] = b.y, r.x[6] = b.z, r.x[7] = b.w;
  return r;
}
__device__ __forceinline__ Row8 load8(const __nv_bfloat16* p) {
  Row8 r;
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = __uint_as_float(w[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ void store8(float* p, const Row8& r) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(r.x[0], r.x[1], r.x[2], r.x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(r.x[4], r.x[5], r.x[6], r.x[7]));
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Row8& r) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(bf2(r.x[0], r.x[1]), bf2(r.x[2], r.x[3]),
                                                 bf2(r.x[4], r.x[5]), bf2(r.x[6], r.x[7])));
}

// Exponent of a row from the bits of its largest magnitude.
__device__ __forceinline__ int row_exp(uint32_t amax) {
  if (amax >= 0x7f800000u) return kNanRow;
  if (amax == 0u) return 0;
  // amax = 1.m * 2^(E-127), 448 = 1.75 * 2^8
  const int e = (int)(amax >> 23) - ((amax & 0x7fffffu) <= 0x600000u ? 135 : 134);
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126..127

// Sixteen elements of a row as they lie in memory.
template <typename T>
struct Raw16 {
  static constexpr int N = (int)sizeof(T);  // 16-byte pieces
  uint4 w[N];
};
template <typename T>
__device__ __forceinline__ Raw16<T> load16(const T* p) {
  Raw16<T> r;
#pragma unroll
  for (int i = 0; i < Raw16<T>::N; ++i) r.w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ float2 pair_of(const Raw16<float>& r, int i) {
  const uint4 w = r.w[i >> 1];
  return i & 1 ? make_float2(__uint_as_float(w.z), __uint_as_float(w.w)) : make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
}
__device__ __forceinline__ float2 pair_of(const Raw16<__nv_bfloat16>& r, int i) {
  const uint4 w = r.w[i >> 2];
  const uint32_t u = (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w;
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Writes a group's row (LANES lanes of sixteen elements) into the cache.
template <int FMT, int LANES, typename T>
__device__ __forceinline__ void put_row(const Raw16<T>& r, unsigned mask, bool first, void* pool, int8_t* exps, int64_t dst,
                                        int part) {
  const int64_t at = dst * (LANES * 16) + part * 16;
  if constexpr (FMT == LS_CACHE_E4M3) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = pair_of(r, i);
      m = max(m, max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu));
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
    const int e = row_exp(m);
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    if (e != kNanRow) {
      const float s = pow2(-e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = pair_of(r, i);
        c[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x.x * s, x.y * s), __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(pool) + at) = make_uint4(c[0], c[1], c[2], c[3]);
    if (first) exps[dst] = (int8_t)e;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Row8 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = pair_of(r, h * 4 + i);
        x.x[2 * i] = y.x, x.x[2 * i + 1] = y.y;
      }
      if constexpr (FMT == LS_CACHE_BF16)
        store8(static_cast<__nv_bfloat16*>(pool) + at + h * 8, x);
      else
        store8(static_cast<float*>(pool) + at + h * 8, x);
    }
  }
}

// One group of D/16 lanes per (token, head): its K row and its V row.
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256) cache_write_kernel(
    const ls_kv_cache c, const T* __restrict__ k, const T* __restrict__ v, int64_t k_stride,
    int64_t v_stride, const int64_t* __restrict__ slots, uint32_t n_rows, int64_t pool_slots, uint32_t* status) {
  constexpr int LANES = D / 16;
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int part = threadIdx.x % LANES;
  const unsigned mask = ((1u << LANES) - 1u) << (lane / LANES * LANES);
  if (row >= n_rows) return;  // a whole group leaves
  const uint32_t t = row / (uint32_t)c.hkv;
  const int head = (int)(row - t * c.hkv);
  const int64_t slot = __ldg(slots + t);
  const Raw16<T> rk = load16(k + (int64_t)t * k_stride + head * D + part * 16);
  const Raw16<T> rv = load16(v + (int64_t)t * v_stride + head * D + part * 16);
  if (slot < 0) return;
  if (slot >= pool_slots) {
    if (part == 0 && status) atomicOr(status, kStatusBadIndex);
    return;
  }
  const uint32_t page = (uint32_t)slot / (uint32_t)c.page_size;  // rows of the pool number below 2^31
  const int64_t dst = (int64_t)((page * c.hkv + head) * c.page_size + ((uint32_t)slot - page * c.page_size));
  put_row<FMT, LANES>(rk, mask, part == 0, c.k, c.k_exp, dst, part);
  put_row<FMT, LANES>(rv, mask, part == 0, c.v, c.v_exp, dst, part);
}

__device__ __forceinline__ Row8 load_codes(const uint8_t* p, int e) {
  Row8 r;
  const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p));
  const float s = e == kNanRow ? __int_as_float(0x7fffffff) : pow2(e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffffu), __NV_E4M3);
    r.x[2 * i] = __half2float(__half(__half_raw{h.x})) * s;
    r.x[2 * i + 1] = __half2float(__half(__half_raw{h.y})) * s;
  }
  return r;
}

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256) cache_read_kernel(
    const ls_kv_cache c, T* __restrict__ k, T* __restrict__ v, const int64_t* __restrict__ slots,
    uint32_t n_rows, int64_t pool_slots, uint32_t* status) {
  constexpr int LANES = D / 8;
  const uint32_t row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int part = threadIdx.x % LANES;
  if (row >= n_rows) return;
  const uint32_t t = row / (uint32_t)c.hkv;
  const int head = (int)(row - t * c.hkv);
  const int64_t slot = __ldg(slots + t);
  Row8 rk, rv;
  if (slot < 0 || slot >= pool_slots) {
    if (slot >= 0 && part == 0 && status) atomicOr(status, kStatusBadIndex);
#pragma unroll
    for (int i = 0; i < 8; ++i) rk.x[i] = rv.x[i] = 0.f;
  } else {
    const uint32_t page = (uint32_t)slot / (uint32_t)c.page_size;
    const int64_t src = (int64_t)((page * c.hkv + head) * c.page_size + ((uint32_t)slot - page * c.page_size));
    if constexpr (FMT == LS_CACHE_E4M3) {
      rk = load_codes(static_cast<const uint8_t*>(c.k) + src * D + part * 8, __ldg(c.k_exp + src));
      rv = load_codes(static_cast<const uint8_t*>(c.v) + src * D + part * 8, __ldg(c.v_exp + src));
    } else if constexpr (FMT == LS_CACHE_BF16) {
      rk = load8(static_cast<const __nv_bfloat16*>(c.k) + src * D + part * 8);
      rv = load8(static_cast<const __nv_bfloat16*>(c.v) + src * D + part * 8);
    } else {
      rk = load8(static_cast<const float*>(c.k) + src * D + part * 8);
      rv = load8(static_cast<const float*>(c.v) + src * D + part * 8);
    }
  }
  store8(k + (int64_t)row * D + part * 8, rk);
  store8(v + (int64_t)row * D + part * 8, rv);
}

// Calls f with the format and the head dimension as constants.
template <typename F>
cudaError_t with_shape(const ls_kv_cache& c, F f) {
  auto by_d = [&](auto fmt) {
    switch (c.head_dim) {
      case 64: return f(fmt, std::integral_constant<int, 64>{});
      case 128: return f(fmt, std::integral_constant<int, 128>{});
      default: return f(fmt, std::integral_constant<int, 256>{});
    }
  };
  switch (c.format) {
    case LS_CACHE_E4M3: return by_d(std::integral_constant<int, LS_CACHE_E4M3>{});
    case LS_CACHE_BF16: return by_d(std::integral_constant<int, LS_CACHE_BF16>{});
    default: return by_d(std::integral_constant<int, LS_CACHE_F32>{});
  }
}

}  // namespace

cudaError_t launch_cache_write(const ls_kv_cache& c, int src_dtype, const void* k, const void* v,
                               int64_t k_stride, int64_t v_stride, const int64_t* slots,
                               int64_t n_tok, uint32_t* status, cudaStream_t s) {
  const int64_t rows = n_tok * c.hkv;
  const int64_t blocks = (rows * (c.head_dim / 16) + 255) / 256;
  if (rows > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int64_t pool_slots = c.pool_pages * c.page_size;
  return with_shape(c, [&](auto fmt, auto d) {
    LaunchScope ls(kKCacheWrite, s);
    if (src_dtype == LS_DTYPE_F32)
      cache_write_kernel<float, fmt.value, d.value><<<(unsigned)blocks, 256, 0, s>>>(
          c, static_cast<const float*>(k), static_cast<const float*>(v), k_stride, v_stride, slots, (uint32_t)rows, pool_slots, status);
    else
      cache_write_kernel<__nv_bfloat16, fmt.value, d.value><<<(unsigned)blocks, 256, 0, s>>>(
          c, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), k_stride, v_stride, slots,
          (uint32_t)rows, pool_slots, status);
    return cudaGetLastError();
  });
}

cudaError_t launch_cache_read(const ls_kv_cache& c, const int64_t* slots, int64_t n_tok,
                              int dst_dtype, void* k, void* v, uint32_t* status, cudaStream_t s) {
  const int64_t rows = n_tok * c.hkv;
  const int64_t blocks = (rows * (c.head_dim / 8) + 255) / 256;
  if (rows > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int64_t pool_slots = c.pool_pages * c.page_size;
  return with_shape(c, [&](auto fmt, auto d) {
    LaunchScope ls(kKCacheRead, s);
    if (dst_dtype == LS_DTYPE_F32)
      cache_read_kernel<float, fmt.value, d.value><<<(unsigned)blocks, 256, 0, s>>>(
          c, static_cast<float*>(k), static_cast<float*>(v), slots, (uint32_t)rows, pool_slots, status);
    else
      cache_read_kernel<__nv_bfloat16, fmt.value, d.value><<<(unsigned)blocks, 256, 0, s>>>(
          c, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), slots, (uint32_t)rows, pool_slots, status);
    return cudaGetLastError();
  });
}

}  // namespace ls
