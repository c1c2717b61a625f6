// Recurrent step of the gated-DeltaNet state: one or a few new tokens of each
// sequence move its state S [dv][dk] on (the recurrence of ls_gdn.cu),
//   u = S k,  w = v - a u,  S <- a S + b w k^T,  o = S q,  a = exp(g).
//
// A row of S needs k, q and its own element of v alone, so rows are spread over
// the whole device: a CTA takes 32 rows of one (sequence, head), eight lanes a
// row with sixteen columns each in registers, all of a CTA's 16 KB loaded before
// the first use.  The tokens then run over the registers; row products are
// sixteen FMAs and three shuffles.
#include <cuda_bf16.h>

#include "ls_internal.h"

namespace ls {
namespace {

constexpr int kD = 128;        // dk = dv
constexpr int kRows = 32;      // rows of a CTA
constexpr int kLanes = 8;      // lanes of a row
constexpr int kTokens = 8;     // tokens staged at a time
constexpr int kThreads = kRows * kLanes;

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Eight elements at p (16-byte aligned) to shared memory as float.
__device__ __forceinline__ void stage8(const float* p, float* to) {
  *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(p);
  *reinterpret_cast<float4*>(to + 4) = *reinterpret_cast<const float4*>(p + 4);
}
__device__ __forceinline__ void stage8(const __nv_bfloat16* p, float* to) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float x) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, x))));
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_decode_kernel(const GdnDecodeParams p) {
  __shared__ __align__(16) float ks[kTokens][kD], qs[kTokens][kD];
  __shared__ float vs[kTokens][kRows], as[kTokens], bs[kTokens];
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int row = blockIdx.x * kRows + tid / kLanes, lane = tid % kLanes;
  const int64_t first = p.q_start[b];
  const int64_t n_all = p.q_start[b + 1] - first;
  const int64_t n = p.n_use ? p.n_use[b] : n_all;
  const int64_t in = p.state_in[b];
  int64_t out = p.state_out ? p.state_out[b] : -1;
  if (first < 0 || n_all < 0 || first + n_all > p.d.total_q || n_all > p.d.max_q || n < 0 || n > n_all ||
      in < -1 || in >= p.d.n_states) {
    if (tid == 0 && p.status) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  if (out >= p.d.n_states) {
    if (tid == 0 && p.status) atomicOr(p.status, kStatusBadIndex);
    out = -1;
  }
  if ((n == 0 || !p.o) && (out < 0 || (n == 0 && out == in))) return;
  const int64_t at = ((int64_t)h * kD + row) * (kD / 4) + lane;  // of a state's float4s
  const int64_t state = (int64_t)p.d.heads * kD * (kD / 4);
  float4 s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    s[j] = in < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : reinterpret_cast<const float4*>(p.states)[in * state + at + j * kLanes];
  const int kh = h / (p.d.heads / p.d.key_heads);
  for (int64_t t0 = 0; t0 < n; t0 += kTokens) {
    const int nt = n - t0 < kTokens ? (int)(n - t0) : kTokens;
    if (t0) __syncthreads();
    {  // a warp a token: sixteen lanes k, sixteen q
      const int t = tid >> 5, part = (tid & 15) * 8;
      if (t < nt) {
        const int64_t tok = first + t0 + t;
        if (tid & 16)
          stage8(static_cast<const T*>(p.q) + tok * p.d.q_stride + kh * kD + part, &qs[t][part]);
        else
          stage8(static_cast<const T*>(p.k) + tok * p.d.k_stride + kh * kD + part, &ks[t][part]);
        vs[t][tid & 31] = value(static_cast<const T*>(p.v)[tok * p.d.v_stride + h * kD + blockIdx.x * kRows + (tid & 31)]);
        if ((tid & 31) == 0) as[t] = expf(p.g[tok * p.d.heads + h]), bs[t] = p.beta[tok * p.d.heads + h];
      }
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float a = as[t];
      float4 k[4];
      float u = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[j] = *reinterpret_cast<const float4*>(&ks[t][(j * kLanes + lane) * 4]);
        u = dot4(s[j], k[j], u);
      }
      u = row_sum(u);
      const float bw = bs[t] * (vs[t][tid / kLanes] - a * u);
      float acc = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j].x = fmaf(a, s[j].x, bw * k[j].x), s[j].y = fmaf(a, s[j].y, bw * k[j].y);
        s[j].z = fmaf(a, s[j].z, bw * k[j].z), s[j].w = fmaf(a, s[j].w, bw * k[j].w);
        if (p.o) acc = dot4(s[j], *reinterpret_cast<const float4*>(&qs[t][(j * kLanes + lane) * 4]), acc);
      }
      if (p.o) {
        acc = row_sum(acc);
        if (lane == 0) put(static_cast<T*>(p.o) + ((first + t0 + t) * p.d.heads + h) * kD + row, acc);
      }
    }
  }
  if (out >= 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<float4*>(p.states)[out * state + at + j * kLanes] = s[j];
  }
}

}  // namespace

cudaError_t launch_gdn_decode(const GdnDecodeParams& p, cudaStream_t s) {
  LaunchScope ls(kKGdnDecode, s);
  const dim3 grid(kD / kRows, p.d.heads, p.d.batch);
  if (p.d.dtype == LS_DTYPE_F32)
    gdn_decode_kernel<float><<<grid, kThreads, 0, s>>>(p);
  else
    gdn_decode_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ls
