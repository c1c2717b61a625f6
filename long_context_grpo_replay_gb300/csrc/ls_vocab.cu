// Vocabulary log-probabilities on the CUDA cores: float32 arithmetic for any
// dtype, row stride and alignment, and what both routes share (joining the
// pieces' softmax statistics).
//
//   x_nv = s * h_n . w_v,  lse_n = log sum_v exp(x_nv),  logp_n = x_nt - lse_n,
//   D_nv = s * dlogp_n * ([v = t_n] - exp(x_nv - lse_n)),  dh = D w,  dw = D^T h.
//
// The logits are never in memory: the forward's product keeps, per row and
// tile of the vocabulary, the tile's maximum and its sum of exponentials; the
// backward forms them again, a piece of the vocabulary at a time, turns them
// into D in the product's epilogue, and uses D in two products.
//
// One tiled product serves all three: 128 x 128, 64 x 64 or 16 x 256 outputs for
// 256 threads, 16 or 32 of the inner dimension at a time through two shared
// buffers, 8 x 8 or 4 x 4 outputs a thread; few rows' dh is cut along the
// vocabulary into float32 sums.  Bound by FMA issue (1024 x 2048 x 16384: 53.7
// TFLOP/s, a library float32 product 58), for few rows by the weight's bytes.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "ls_internal.h"
#include "ls_tc.cuh"

namespace ls {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kQuantum = 32;  // splits of the inner dimension are multiples of it

__device__ __forceinline__ float ldf(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p)) << 16);
}
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// An operand of the product: element (i, k), i the output's index.
template <typename T>
struct Operand {
  const T* p;
  int64_t si, sk;  // strides of i and k; one of them is 1
  int64_t n;       // extent of i
  bool quads;      // four neighbours of the contiguous index can be read at once
};
template <typename T>
Operand<T> operand(const T* p, int64_t si, int64_t sk, int64_t n) {
  const int64_t other = sk == 1 ? si : sk;
  return {p, si, sk, n, reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && other % 4 == 0};
}

__device__ __forceinline__ float4 ld4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

// C tile = sum_k A(m, k) B(n, k) over k in [kb, ke).  The next 16 (or 32) of k
// are loaded into registers while these are multiplied from shared memory.
template <int TM, int TX, typename TA, typename TB>
struct Product {
  static constexpr int TILE_M = 256 / TX * TM, TILE_N = TX * TM;
  // the 64 x 64 tile has 32 of the inner dimension at a time, for fewer barriers
  static constexpr int kBK = TM == 4 && TX == 16 ? 32 : 16, KQ = kBK / 4;
  float a[2][kBK][TILE_M + 4], b[2][kBK][TILE_N + 4];

  template <int TILE>
  static constexpr int quads() {  // of an operand's tile per thread
    return TILE * KQ >= 256 ? TILE * KQ / 256 : 1;
  }
  template <int TILE, typename T>
  __device__ __forceinline__ static void load(float4 (&r)[quads<TILE>()], const Operand<T>& o, int64_t i0, int64_t k0, int64_t ke) {
    // a quad lies along the contiguous index, and so do neighbouring threads
#pragma unroll
    for (int q = 0; q < quads<TILE>(); ++q) {
      const int x = threadIdx.x + q * 256;
      const bool kc = o.sk == 1;
      const int64_t i = i0 + (kc ? x / KQ : x % (TILE / 4) * 4), k = k0 + (kc ? x % KQ * 4 : x / (TILE / 4));
      const T* src = o.p + i * o.si + k * o.sk;
      const int64_t left = kc ? ke - k : o.n - i;  // of the contiguous index
      const bool there = (kc ? i < o.n : k < ke) && x < TILE * KQ;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (there && left >= 4 && o.quads) {
        v = ld4(src);
      } else if (there) {
        if (left > 0) v.x = ldf(src);
        if (left > 1) v.y = ldf(src + 1);
        if (left > 2) v.z = ldf(src + 2);
        if (left > 3) v.w = ldf(src + 3);
      }
      r[q] = v;
    }
  }
  template <int TILE>
  __device__ __forceinline__ static void store(float (&dst)[kBK][TILE + 4], const float4 (&r)[quads<TILE>()], bool kc) {
#pragma unroll
    for (int q = 0; q < quads<TILE>(); ++q) {
      const int x = threadIdx.x + q * 256;
      if (x >= TILE * KQ) break;
      if (kc) {
        const int i = x / KQ, k = x % KQ * 4;
        dst[k][i] = r[q].x, dst[k + 1][i] = r[q].y, dst[k + 2][i] = r[q].z, dst[k + 3][i] = r[q].w;
      } else {
        *reinterpret_cast<float4*>(&dst[x / (TILE / 4)][x % (TILE / 4) * 4]) = r[q];
      }
    }
  }

  // Row (column) of output i (j) of the thread's: four together, TM 8 in two groups half a tile apart.
  __device__ __forceinline__ static int at_m(int ty, int i) { return i / 4 * (TILE_M / 2) + ty * 4 + (i & 3); }
  __device__ __forceinline__ static int at_n(int tx, int j) { return j / 4 * (TILE_N / 2) + tx * 4 + (j & 3); }

  __device__ __forceinline__ void run(const Operand<TA>& A, const Operand<TB>& B, int64_t m0, int64_t n0,
                                      int64_t kb, int64_t ke, float (&acc)[TM][TM]) {
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    // outputs two by two along n: one packed instruction for two products, each
    // rounded as fmaf rounds it
    uint64_t sum[TM][TM / 2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM / 2; ++j) sum[i][j] = 0ull;
    float4 ra[quads<TILE_M>()], rb[quads<TILE_N>()];
    load<TILE_M>(ra, A, m0, kb, ke);
    load<TILE_N>(rb, B, n0, kb, ke);
    store<TILE_M>(a[0], ra, A.sk == 1);
    store<TILE_N>(b[0], rb, B.sk == 1);
    __syncthreads();
    int buf = 0;
    for (int64_t k0 = kb; k0 < ke; k0 += kBK, buf ^= 1) {
      const bool more = k0 + kBK < ke;
      if (more) {
        load<TILE_M>(ra, A, m0, k0 + kBK, ke);
        load<TILE_N>(rb, B, n0, k0 + kBK, ke);
      }
#pragma unroll
      for (int k = 0; k < kBK; ++k) {
        float x[TM];
        uint64_t y[TM / 2];
#pragma unroll
        for (int i = 0; i < TM; i += 4) {
          *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(&a[buf][k][at_m(ty, i)]);
          *reinterpret_cast<ulonglong2*>(y + i / 2) = *reinterpret_cast<const ulonglong2*>(&b[buf][k][at_n(tx, i)]);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const uint64_t xx = tc::f2(x[i], x[i]);
#pragma unroll
          for (int j = 0; j < TM / 2; ++j) sum[i][j] = tc::f2_fma(xx, y[j], sum[i][j]);
        }
      }
      if (more) {
        store<TILE_M>(a[buf ^ 1], ra, A.sk == 1);
        store<TILE_N>(b[buf ^ 1], rb, B.sk == 1);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM / 2; ++j) tc::f2_split(sum[i][j], acc[i][2 * j], acc[i][2 * j + 1]);
  }
};

// The number of this CTA's tile along the vocabulary, which may have more than the
// 65,535 of a grid's second dimension: the third counts those.
__device__ __forceinline__ uint32_t n_tile_of() { return blockIdx.z * gridDim.y + blockIdx.y; }

// Forward: per row and the columns of one warp, (maximum, sum of
// 2^(x - maximum)) of the logits in base 2, and the target's logit.
template <int TM, int TX, typename T>
__global__ void __launch_bounds__(256, 2) vocab_fwd_kernel(const ls_vocab_desc d, const Operand<T> A,
                                                        const Operand<T> B, const int64_t* targets, float2* parts, float* hit) {
  using P = Product<TM, TX, T, T>;
  constexpr int kLanes = TX < 32 ? TX : 32;  // of a warp that share a row; a row's warps leave statistics of their own
  __shared__ __align__(16) P sm;
  const uint32_t n_tile = n_tile_of();
  const int64_t m0 = (int64_t)blockIdx.x * P::TILE_M, n0 = (int64_t)n_tile * P::TILE_N;
  if (n0 >= B.n) return;
  float acc[TM][TM];
  sm.run(A, B, m0, n0, 0, d.hidden, acc);
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = m0 + P::at_m(ty, i);
    const int64_t target = row < d.n_rows ? __ldg(targets + row) : -1;
    float top = -CUDART_INF_F;
    float y[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t v = n0 + P::at_n(tx, j);
      const float x = acc[i][j] * d.logit_scale;
      if (v == target && v < d.vocab) hit[row] = x;
      y[j] = v < d.vocab ? x * kLog2e : -CUDART_INF_F;
      top = fmaxf(top, y[j]);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < TM; ++j) sum += exp2f(y[j] - ref);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x % kLanes == 0 && row < d.n_rows)
      parts[((int64_t)n_tile * (TX / kLanes) + threadIdx.x % TX / kLanes) * d.n_rows + row] = make_float2(top, sum);
  }
}

// lse and logp of 32 rows from their tiles' statistics: lane = row, eight
// warps share the tiles.
__global__ void __launch_bounds__(256) vocab_join_kernel(int n_tiles, int64_t n_rows, int64_t vocab,
                                                         int64_t ignore, const float2* __restrict__ parts,
                                                         const float* __restrict__ hit,
                                                         const int64_t* __restrict__ targets,
                                                         float* __restrict__ logp, float* __restrict__ lse,
                                                         uint32_t* status) {
  __shared__ float2 sm[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  float m = -CUDART_INF_F, l = 0.f;
  if (row < n_rows)
    for (int t = warp; t < n_tiles; t += 8) {
      const float2 a = __ldg(parts + (int64_t)t * n_rows + row);
      const float mn = fmaxf(m, a.x);
      const float ref = mn == -CUDART_INF_F ? 0.f : mn;
      l = l * exp2f(m - ref) + a.y * exp2f(a.x - ref);
      m = mn;
    }
  sm[warp][lane] = make_float2(m, l);
  __syncthreads();
  if (warp == 0 && row < n_rows) {
    for (int i = 1; i < 8; ++i) {
      const float2 a = sm[i][lane];
      const float mn = fmaxf(m, a.x);
      const float ref = mn == -CUDART_INF_F ? 0.f : mn;
      l = l * exp2f(m - ref) + a.y * exp2f(a.x - ref);
      m = mn;
    }
    const float z = ((m == -CUDART_INF_F ? 0.f : m) + log2f(l)) * kLn2;
    lse[row] = z;
    const int64_t target = __ldg(targets + row);
    const bool in = target >= 0 && target < vocab;
    if (!in && target != ignore) atomicOr(status, kStatusBadIndex);
    logp[row] = in ? hit[row] - z : 0.f;
  }
}

// D of a piece of the vocabulary: columns v0 .. v0 + np of the logits.
template <int TM, int TX, typename T>
__global__ void __launch_bounds__(256, 2) vocab_slope_kernel(const ls_vocab_desc d, const Operand<T> A,
                                                          const Operand<T> B, const int64_t* targets, const float* lse,
                                                          const float* d_logp, int64_t v0, int64_t np, float* out) {
  using P = Product<TM, TX, T, T>;
  __shared__ __align__(16) P sm;
  const uint32_t n_tile = n_tile_of();
  const int64_t m0 = (int64_t)blockIdx.x * P::TILE_M, n0 = (int64_t)n_tile * P::TILE_N;
  if (n0 >= B.n) return;
  float acc[TM][TM];
  sm.run(A, B, m0, n0, 0, d.hidden, acc);
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = m0 + P::at_m(ty, i);
    if (row >= d.n_rows) continue;
    const int64_t target = __ldg(targets + row);
    const float c = target >= 0 && target < d.vocab ? __ldg(d_logp + row) * d.logit_scale : 0.f;
    const float z = __ldg(lse + row);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t n = n0 + P::at_n(tx, j);
      if (n >= np) continue;
      const float p = exp2f((acc[i][j] * d.logit_scale - z) * kLog2e);
      // a row that takes no part has no gradient even where its logits are not finite
      out[row * np + n] = c == 0.f ? 0.f : c * ((v0 + n == target ? 1.f : 0.f) - p);
    }
  }
}

// out[z][m][n] = A B^T over split z's share of the inner dimension (+ what is there), rounded to TO once.
template <int TM, int TX, typename TA, typename TB, typename TO>
__global__ void __launch_bounds__(256, 2) vocab_product_kernel(Operand<TA> A, Operand<TB> B, int64_t K, int64_t per,
                                                            bool add, TO* out) {
  using P = Product<TM, TX, TA, TB>;
  __shared__ __align__(16) P sm;
  const int64_t m0 = (int64_t)blockIdx.x * P::TILE_M, n0 = (int64_t)blockIdx.y * P::TILE_N;
  float acc[TM][TM];
  const int64_t kb = blockIdx.z * per, ke = kb + per < K ? kb + per : K;
  out += (int64_t)blockIdx.z * A.n * B.n;
  sm.run(A, B, m0, n0, kb, ke, acc);
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + P::at_m(ty, i);
    if (m >= A.n) continue;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t n = n0 + P::at_n(tx, j);
      if (n >= B.n) continue;
      float v = acc[i][j];
      if constexpr (sizeof(TO) == 4)
        if (add) v += out[m * B.n + n];
      stf(out + m * B.n + n, v);
    }
  }
}

// dh from its float32 sums [split][n].
template <typename T>
__global__ void __launch_bounds__(256) vocab_sum_kernel(int splits, int64_t n, const float* __restrict__ sums, T* __restrict__ out) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x >= n) return;
  float a = 0.f;
  for (int s = 0; s < splits; ++s) a += __ldcs(sums + s * n + x);
  stf(out + x, a);
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Columns of a piece on the CUDA cores: D of a piece within 256 MB.
int64_t simt_piece(const ls_vocab_desc& d) {
  int64_t np = d.piece > 0 ? d.piece : (64ll << 20) / (d.n_rows > 0 ? d.n_rows : 1) / 128 * 128;
  if (np < 128 && d.piece == 0) np = 128;
  return np < d.vocab ? np : d.vocab;
}

// The product's tile: 16 x 256 for up to 16 rows (bound by the weight's bytes if
// the empty rows of a larger tile are left out), 64 x 64 where half of a 128-row
// tile would be empty or 128 x 128 ones would leave half the SMs idle (128 x 1024
// x 16384: 128 large tiles 120 us, 512 small ones 160), else 128 x 128.
enum Tile { kWide, kSmall, kLarge };
int tile_m(Tile t) { return t == kWide ? 16 : t == kSmall ? 64 : 128; }
int tile_n(Tile t) { return t == kWide ? 256 : t == kSmall ? 64 : 128; }
int64_t tiles_of(Tile t, int64_t m, int64_t n) {
  return ((m + tile_m(t) - 1) / tile_m(t)) * ((n + tile_n(t) - 1) / tile_n(t));
}
Tile pick_tile(int64_t m, int64_t n, int64_t splits = 1) {
  if (m <= 16) return kWide;
  if (m <= 64 || n <= 64 || tiles_of(kLarge, m, n) * splits < device_sms() / 2) return kSmall;
  return kLarge;
}
// Ways to cut dh's inner dimension, a piece of the vocabulary: where its tiles
// leave SMs idle, two CTAs an SM, 256 columns each at least.
int64_t most_splits(const ls_vocab_desc& d) {
  const int64_t s = simt_piece(d) / 256;
  return s < 1 ? 1 : s;
}
Tile dh_tile(const ls_vocab_desc& d) { return pick_tile(d.n_rows, d.hidden, most_splits(d)); }
int simt_splits(const ls_vocab_desc& d) {
  const int64_t tiles = tiles_of(dh_tile(d), d.n_rows, d.hidden);
  int64_t s = tiles > 0 ? 2 * device_sms() / tiles : 1;
  s = s < most_splits(d) ? s : most_splits(d);
  return s < 1 ? 1 : (int)s;
}
int64_t simt_per_split(const ls_vocab_desc& d) {
  const int64_t s = simt_splits(d);
  return round_up((size_t)((simt_piece(d) + s - 1) / s), kQuantum);
}

template <typename F>
cudaError_t with_tile(int64_t m, int64_t n, Tile t, bool layered, F f) {
  const int64_t mt = (m + tile_m(t) - 1) / tile_m(t), nt = (n + tile_n(t) - 1) / tile_n(t), layers = (nt + 65534) / 65535;
  if (mt > INT32_MAX || layers > (layered ? 65535 : 1)) return cudaErrorInvalidConfiguration;
  // as many tiles a layer, so that a few may lie past the end
  const dim3 grid((unsigned)mt, (unsigned)((nt + layers - 1) / layers), (unsigned)layers);
  using std::integral_constant;
  if (t == kWide)
    f(integral_constant<int, 4>{}, integral_constant<int, 64>{}, grid);
  else if (t == kSmall)
    f(integral_constant<int, 4>{}, integral_constant<int, 16>{}, grid);
  else
    f(integral_constant<int, 8>{}, integral_constant<int, 16>{}, grid);
  return cudaGetLastError();
}

// Statistics per row: one for 64 columns, or two for 256.
int64_t most_parts(const ls_vocab_desc& d) { return (d.vocab + 63) / 64 + 1; }

template <typename T>
cudaError_t simt_fwd(const VocabParams& p, cudaStream_t s) {
  const ls_vocab_desc& d = p.d;
  const auto A = operand(static_cast<const T*>(p.h), d.h_stride, 1, d.n_rows);
  const auto B = operand(static_cast<const T*>(p.w), d.w_stride, 1, d.vocab);
  float2* parts = static_cast<float2*>(p.scratch);
  const int64_t n_parts = most_parts(d);
  float* hit = reinterpret_cast<float*>(parts + n_parts * d.n_rows);
  int n_tiles = 0;
  {
    LaunchScope ls(kKVocabSimt, s);
    const Tile t = pick_tile(d.n_rows, d.vocab);
    const cudaError_t e = with_tile(d.n_rows, d.vocab, t, true, [&](auto tm, auto tx, dim3 grid) {
      n_tiles = (int)((d.vocab + tile_n(t) - 1) / tile_n(t)) * (tx.value < 32 ? 1 : tx.value / 32);
      vocab_fwd_kernel<tm.value, tx.value, T><<<grid, 256, 0, s>>>(d, A, B, p.targets, parts, hit);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_vocab_join(n_tiles, p, parts, hit, s);
}

template <typename T>
cudaError_t simt_bwd(const VocabParams& p, cudaStream_t s) {
  const ls_vocab_desc& d = p.d;
  const T* h = static_cast<const T*>(p.h);
  const T* w = static_cast<const T*>(p.w);
  const int64_t piece = simt_piece(d), per = simt_per_split(d);
  const int splits = (int)((piece + per - 1) / per);
  const bool direct = splits == 1 && piece == d.vocab;
  float* slope = static_cast<float*>(p.scratch);
  float* sums = slope + round_up((size_t)d.n_rows * piece, 64);
  for (int64_t v0 = 0; v0 < d.vocab; v0 += piece) {
    const int64_t np = d.vocab - v0 < piece ? d.vocab - v0 : piece;
    LaunchScope ls(kKVocabSimt, s);
    cudaError_t e = with_tile(d.n_rows, np, pick_tile(d.n_rows, np), true, [&](auto tm, auto tx, dim3 grid) {
      vocab_slope_kernel<tm.value, tx.value, T><<<grid, 256, 0, s>>>(d, operand(h, d.h_stride, 1, d.n_rows),
                                                           operand(w + v0 * d.w_stride, d.w_stride, 1, np), p.targets,
                                                           p.lse_in, p.d_logp, v0, np, slope);
    });
    if (e != cudaSuccess) return e;
    if (p.dh) {
      const auto A = operand(static_cast<const float*>(slope), np, 1, d.n_rows);
      const auto B = operand(w + v0 * d.w_stride, 1, d.w_stride, d.hidden);
      e = with_tile(d.n_rows, d.hidden, dh_tile(d), false, [&](auto tm, auto tx, dim3 grid) {
        ls.more_kernels(1);
        grid.z = (unsigned)((np + per - 1) / per);  // a shorter last piece has fewer
        if (direct)
          vocab_product_kernel<tm.value, tx.value, float, T, T><<<grid, 256, 0, s>>>(A, B, np, per, false, static_cast<T*>(p.dh));
        else
          vocab_product_kernel<tm.value, tx.value, float, T, float><<<grid, 256, 0, s>>>(A, B, np, per, v0 > 0, sums);
      });
      if (e != cudaSuccess) return e;
    }
    if (p.dw) {
      const auto A = operand(static_cast<const float*>(slope), 1, np, np);
      const auto B = operand(h, 1, d.h_stride, d.hidden);
      e = with_tile(np, d.hidden, pick_tile(np, d.hidden), false, [&](auto tm, auto tx, dim3 grid) {
        ls.more_kernels(1);
        vocab_product_kernel<tm.value, tx.value, float, T, T><<<grid, 256, 0, s>>>(A, B, d.n_rows, d.n_rows, false, static_cast<T*>(p.dw) + v0 * d.hidden);
      });
      if (e != cudaSuccess) return e;
    }
  }
  if (p.dh && !direct) {
    const int64_t n = d.n_rows * d.hidden;
    LaunchScope ls(kKVocabReduce, s);
    vocab_sum_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(splits, n, sums, static_cast<T*>(p.dh));
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_vocab_join(int n_tiles, const VocabParams& p, const float2* parts, const float* hit,
                              cudaStream_t s) {
  LaunchScope ls(kKVocabReduce, s);
  vocab_join_kernel<<<(unsigned)((p.d.n_rows + 31) / 32), 256, 0, s>>>(
      n_tiles, p.d.n_rows, p.d.vocab, p.d.ignore_index, parts, hit, p.targets, p.logp, p.lse, p.status);
  return cudaGetLastError();
}

size_t vocab_simt_scratch(const ls_vocab_desc& d, bool with_grad) {
  const size_t n = (size_t)d.n_rows, nf = (size_t)(d.n_rows < kVocabRows ? d.n_rows : kVocabRows);
  size_t need = (size_t)most_parts(d) * nf * sizeof(float2) + nf * sizeof(float);
  if (with_grad) {
    const size_t splits = (size_t)((simt_piece(d) + simt_per_split(d) - 1) / simt_per_split(d));
    const size_t g = (round_up(n * (size_t)simt_piece(d), 64) +
                      (splits > 1 || simt_piece(d) < d.vocab ? splits * n * (size_t)d.hidden : 0)) * sizeof(float);
    need = g > need ? g : need;
  }
  return round_up(need, 256);
}

cudaError_t launch_vocab_simt_fwd(const VocabParams& p, cudaStream_t s) {
  return p.d.dtype == LS_DTYPE_F32 ? simt_fwd<float>(p, s) : simt_fwd<__nv_bfloat16>(p, s);
}
cudaError_t launch_vocab_simt_bwd(const VocabParams& p, cudaStream_t s) {
  return p.d.dtype == LS_DTYPE_F32 ? simt_bwd<float>(p, s) : simt_bwd<__nv_bfloat16>(p, s);
}

}  // namespace ls
