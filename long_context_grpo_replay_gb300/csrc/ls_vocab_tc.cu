// Vocabulary log-probabilities on the tensor cores (bf16): one persistent
// tcgen05 product with three epilogues.
//
//   forward    X = h w^T              epilogue: per row and 256 columns, the
//                                     maximum and sum of 2^(x - maximum)
//   slope      X = h w_piece^T        epilogue: D = c ([v = t] - 2^(x - lse)),
//                                     bf16, the only copy of the piece
//   gradients  dh += D w_piece, dw_piece = D^T h
//
// A pair of CTAs (cta_group::2) has a 256 x 256 tile: each CTA loads its 128
// rows of A and its 128 rows of B, 64 of the inner dimension at a time, into
// a ring of six 32 KB stages, and holds its 128 rows of the float32 result in
// 256 of its tensor-memory columns; there are two such results, so that a
// tile's epilogue runs under the next tile's products.  A pair reads half the
// bytes that two lone CTAs would (64 bytes per clock and SM at full rate,
// against the 96 of a 128 x 256 tile), which is what keeps L2 off the path.
//
// An operand is read as it lies in memory, inner dimension contiguous ("K
// major") or not ("MN major": W in dh, D and h in dw), so nothing is
// transposed.  Rows and columns past the end load as zeros.
//
// Measured: 8192 x 4096 x 128,000 scored in 5.3 ms back to back (1.62 PFLOP/s, the
// power limit), 4.6 ms alone (1.87 PFLOP/s; a library product 1.89); 4096 x 4096 x
// 50,003 forward and backward in 4.1 ms, four products.
//
// Warp roles (256 threads): 0 loads, 1 issues products (in the pair's first
// CTA), 2 owns tensor memory, 4-7 run the epilogue, one thread a row.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <cstring>

#include "ls_internal.h"
#include "ls_tc.cuh"

namespace ls {
namespace {
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 256, kHalf = 128, kBK = 64, kStages = 6, kThreads = 256;
constexpr uint32_t kOperand = kHalf * kBK * 2;  // 16 KB: one CTA's share of A or B of a stage
constexpr uint32_t kStage = 2 * kOperand;
constexpr uint32_t kOutBox = 32 * 128;          // an epilogue warp's 32 rows x 64 columns of bf16
constexpr uint32_t kSmem = kStages * kStage + 4 * 2 * kOutBox + 1024;
constexpr uint32_t kMnBox = kBK * 128;          // [64 inner x 64 columns] of an MN-major operand

enum Epilogue { kStats, kSlope, kOut };

struct ProductParams {
  int32_t m, n;            // extents of the result
  int32_t k;               // inner extent
  int32_t m_tiles, n_tiles, splits;
  int32_t k_blocks;        // inner blocks of 64 per split
  int32_t m_fast;          // neighbouring tiles differ in m (else in n)
  int32_t a_boxes, b_boxes;  // an MN-major operand is loaded in one box, or in two of 64 columns
  // forward and slope
  int32_t v0, vocab;       // first column's token, vocabulary
  float scale, scale_log2;
  const int64_t* targets;
  float2* parts;
  float* hit;
  const float* lse;
  const float* d_logp;
  // gradients: rounded, through the output's map, or (sums not NULL) to / added
  // to float32 sums [split][m][n]
  float* sums;
  int32_t add;
  uint32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What it announces is in tensor memory, behind tcgen05.fence::before_thread_sync.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void load2_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void load2_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the products so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// Stores a swizzled [32 x 64] box of bf16 from shared memory; the map clips it.
__device__ __forceinline__ void store_box(const CUtensorMap* m, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1)
      : "memory");
}
// All but the last N of this thread's stores have read their shared memory.
template <int N>
__device__ __forceinline__ void store_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

template <int EPI, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    vocab_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const ProductParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[kStages], bar_empty[kStages], bar_done[2], bar_free[2];
  __shared__ uint32_t tmem_base_s, abort_s, never_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

  if (tid == 0) {
    abort_s = never_s = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bar_full[i]), 1);
      mbar_init(smem_u32(&bar_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_done[i]), 1);
      mbar_init(smem_u32(&bar_free[i]), 8);  // the epilogue warps of both CTAs
    }
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base_s)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tbase = tmem_base_s;
  const volatile uint32_t* abortp = &abort_s;
  auto fail = [&](int line) {
    atomicOr(p.status, kStatusTimeout);
    atomicCAS(p.status + 1, 0u, ((uint32_t)kKVocabTc << 16) | (uint32_t)line);
    abort_s = 1;
  };
  const int units = p.m_tiles * p.n_tiles * p.splits;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int all_blocks = (p.k + kBK - 1) / kBK;
  struct Unit {
    int m, n, split, kb, nk;
  };
  auto unit = [&](int u) -> Unit {
    Unit t;
    const int tiles = p.m_tiles * p.n_tiles;
    t.split = u / tiles;
    const int x = u - t.split * tiles;
    t.m = p.m_fast ? x % p.m_tiles : x / p.n_tiles;
    t.n = p.m_fast ? x / p.m_tiles : x % p.n_tiles;
    t.kb = t.split * p.k_blocks;
    t.nk = all_blocks - t.kb < p.k_blocks ? all_blocks - t.kb : p.k_blocks;
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      prefetch_tmap(&tmC);
      int it = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += pairs) {
        const Unit t = unit(u);
        const int ma = t.m * kTile + (int)rank * kHalf, nb = t.n * kTile + (int)rank * kHalf;
        for (int k = 0; k < t.nk; ++k, ++it) {
          const int s = it % kStages;
          if (it >= kStages && !mbar_wait(smem_u32(&bar_empty[s]), (it / kStages - 1) & 1, abortp)) {
            fail(__LINE__);
            ok = false;
            break;
          }
          const uint32_t full = map_to(smem_u32(&bar_full[s]), 0);
          if (rank == 0) mbar_expect_tx(smem_u32(&bar_full[s]), 2 * kStage);
          const uint32_t a = ring + s * kStage, b = a + kOperand;
          const int k0 = (t.kb + k) * kBK;
          if constexpr (!A_MN) {
            load2_2d(a, &tmA, full, k0, ma);
          } else if (p.a_boxes == 1) {
            load2_3d(a, &tmA, full, 0, k0, ma / 64);
          } else {
            load2_2d(a, &tmA, full, ma, k0);
            load2_2d(a + kMnBox, &tmA, full, ma + 64, k0);
          }
          if constexpr (!B_MN) {
            load2_2d(b, &tmB, full, k0, nb);
          } else if (p.b_boxes == 1) {
            load2_3d(b, &tmB, full, 0, k0, nb / 64);
          } else {
            load2_2d(b, &tmB, full, nb, k0);
            load2_2d(b + kMnBox, &tmB, full, nb + 64, k0);
          }
        }
      }
      // no copy may still be landing when the pair ends: the first CTA's
      // barriers count both CTAs' bytes, and the pair leaves together
      const int last = it - kStages < 0 ? 0 : it - kStages;
      if (rank == 0)
        for (int i = last; i < it; ++i)
          mbar_wait(smem_u32(&bar_full[i % kStages]), (i / kStages) & 1, &never_s);
      // nor an arrival of the products: each CTA waits for the last ones that it was sent
      for (int i = last; ok && i < it; ++i)
        if (!mbar_wait(smem_u32(&bar_empty[i % kStages]), (i / kStages) & 1, abortp)) {
          fail(__LINE__);
          ok = false;
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(kTile, kTile, B_MN, A_MN);
      int it = 0, n = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += pairs, ++n) {
        const Unit t = unit(u);
        const int b = n & 1;
        if (n >= 2 && !mbar_wait(smem_u32(&bar_free[b]), ((n >> 1) - 1) & 1, abortp)) {
          fail(__LINE__);
          break;
        }
        tc_fence_after();
        for (int k = 0; k < t.nk; ++k, ++it) {
          const int s = it % kStages;
          if (!mbar_wait(smem_u32(&bar_full[s]), (it / kStages) & 1, abortp)) {
            fail(__LINE__);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = ring + s * kStage, bb = a + kOperand;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t da = A_MN ? sdesc_sw128(a + kk * 2048, kMnBox, 1024) : sdesc_sw128(a + kk * 32, 16, 1024);
            const uint64_t db = B_MN ? sdesc_sw128(bb + kk * 2048, kMnBox, 1024) : sdesc_sw128(bb + kk * 32, 16, 1024);
            mma2_ss(tbase + b * kTile, da, db, idesc, (k > 0 || kk > 0) ? 1u : 0u);
          }
          commit2(smem_u32(&bar_empty[s]));
        }
        if (ok) commit2(smem_u32(&bar_done[b]));
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp - 4;
    const uint32_t out_box = ring + kStages * kStage + q * 2 * kOutBox;
    int n = 0, boxes = 0;
    for (int u = pair; u < units; u += pairs, ++n) {
      const Unit t = unit(u);
      const int b = n & 1;
      const int row = t.m * kTile + (int)rank * kHalf + q * 32 + lane, n0 = t.n * kTile;
      const bool row_ok = row < p.m;
      int64_t target = -1;
      float c = 0.f, z2 = 0.f;
      if constexpr (EPI != kOut) {
        if (row_ok) target = __ldg(p.targets + row);
        if (EPI == kSlope && row_ok) {
          c = target >= 0 && target < p.vocab ? __ldg(p.d_logp + row) * p.scale : 0.f;
          z2 = __ldg(p.lse + row) * kLog2e;
        }
      }
      if (!mbar_wait_warp(smem_u32(&bar_done[b]), (n >> 1) & 1, abortp)) {
        if (lane == 0) fail(__LINE__);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tbase + ((uint32_t)(q * 32) << 16) + b * kTile;
      const int cols = p.n - n0 < kTile ? p.n - n0 : kTile;
      const int hit = target >= p.v0 + n0 && target < p.v0 + n0 + cols ? (int)(target - p.v0 - n0) : -1;
      if constexpr (EPI == kStats) {
        float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(acc + c0, r);
          tmem_wait_ld_r(r);
          float y[32], mx = -CUDART_INF_F;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (c0 + j == hit) p.hit[row] = __uint_as_float(r[j]) * p.scale;
            y[j] = c0 + j < cols ? __uint_as_float(r[j]) * p.scale_log2 : -CUDART_INF_F;
            mx = fmaxf(mx, y[j]);
          }
          const float mn = fmaxf(top, mx), ref = mn == -CUDART_INF_F ? 0.f : mn;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) s4[j & 3] += ex2(y[j] - ref);
          sum = sum * ex2(top - ref) + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
          top = mn;
        }
        if (row_ok) p.parts[(int64_t)t.n * p.m + row] = make_float2(top, sum);
      } else if (EPI == kOut && p.sums) {
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(acc + c0, r);
          tmem_wait_ld_r(r);
          if (!row_ok) continue;
          // n is a multiple of 8: four columns are there or not
          float* dst = p.sums + ((int64_t)t.split * p.m + row) * p.n + n0 + c0;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            if (c0 + j >= cols) break;
            float4 v = make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
            if (p.add) {
              const float4 w = *reinterpret_cast<const float4*>(dst + j);
              v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
            }
            *reinterpret_cast<float4*>(dst + j) = v;
          }
        }
      } else {
        // 64 columns at a time through the warp's own two boxes in shared memory
        // and out by TMA: rows' lines leave whole.  (Each thread storing its
        // row's 16-byte pieces, dw of 4 rows, 75,189 x 4584, took 300 us.)
        const int row0 = t.m * kTile + (int)rank * kHalf + q * 32;
#pragma unroll 1
        for (int c0 = 0; c0 < cols && row0 < p.m; c0 += 64, ++boxes) {
          const uint32_t box = out_box + (boxes & 1) * kOutBox;
          if (lane == 0) store_read<1>();  // the box's last store has read it
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            tmem_ld32(acc + c0 + 32 * h, r);
            tmem_wait_ld_r(r);
            if constexpr (EPI == kSlope) {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float e = ex2(fmaf(__uint_as_float(r[j]), p.scale_log2, -z2));
                r[j] = __float_as_uint(c == 0.f ? 0.f : c * ((c0 + 32 * h + j == hit ? 1.f : 0.f) - e));
              }
            }
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              st_shared_v4(box + sw128_offset(lane, 4 * h + j / 8),
                           make_uint4(pack_bf16x2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                      pack_bf16x2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                                      pack_bf16x2(__uint_as_float(r[j + 4]), __uint_as_float(r[j + 5])),
                                      pack_bf16x2(__uint_as_float(r[j + 6]), __uint_as_float(r[j + 7]))));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) store_box(&tmC, box, n0 + c0, row0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(map_to(smem_u32(&bar_free[b]), 0));
    }
    // the stores have left before the CTA does
    if (EPI != kStats && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tbase) : "memory");
  }
}

// dh from its float32 sums: one thread per four elements.
__global__ void __launch_bounds__(256) vocab_sum_kernel(int splits, int64_t n, const float* __restrict__ sums, __nv_bfloat16* __restrict__ out) {
  const int64_t x = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (x >= n) return;
  float4 a = __ldcs(reinterpret_cast<const float4*>(sums + x));
  for (int s = 1; s < splits; ++s) {
    const float4 z = __ldcs(reinterpret_cast<const float4*>(sums + s * n + x));
    a.x += z.x, a.y += z.y, a.z += z.z, a.w += z.w;
  }
  *reinterpret_cast<uint2*>(out + x) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int64_t div_up(int64_t x, int64_t a) { return (x + a - 1) / a; }

// K-major operand [rows][cols]: boxes of 128 rows x 64 columns.
bool k_major(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride) {
  return encode_matrix_map(m, p, rows, cols, stride, kHalf, 1);
}
// MN-major operand [inner rows][cols]: one box of 64 rows x (2 x 64) columns
// where the columns are whole blocks of 64, else boxes of 64 x 64.
bool mn_major(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride, int32_t* boxes) {
  *boxes = cols % 64 == 0 ? 1 : 2;
  return encode_matrix_map(m, p, rows, cols, stride, kBK, *boxes == 1 ? 2 : 1);
}

// An output: boxes of 32 rows x 64 columns.
bool output(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride) {
  return encode_matrix_map(m, p, rows, cols, stride, 32, 1);
}

// Pairs of CTAs that the device holds at once.
template <typename K>
int resident_pairs(K kernel) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(device_sms() / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = device_sms() / 2;
  }
  return n < device_sms() / 2 ? n : device_sms() / 2;
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t run_product(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, ProductParams p, cudaStream_t s) {
  auto* kernel = vocab_tc_kernel<EPI, A_MN, B_MN>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  static const int most = resident_pairs(kernel);
  const int64_t units = (int64_t)p.m_tiles * p.n_tiles * p.splits;
  if (units > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  const int pairs = units < most ? (int)units : most;
  LaunchScope ls(kKVocabTc, s);
  kernel<<<2 * pairs, kThreads, kSmem, s>>>(a, b, c, p);
  return cudaGetLastError();
}

// Columns of a piece: its slope within 256 MB, pieces of about one size, whole tiles.
int64_t tc_piece(const ls_vocab_desc& d) {
  const int64_t n = d.n_rows > 0 ? d.n_rows : 1;
  int64_t most = d.piece > 0 ? d.piece : (128ll << 20) / n;
  most = most / kTile * kTile;
  if (most < kTile) most = kTile;
  if (most >= d.vocab) return d.vocab;
  const int64_t pieces = div_up(d.vocab, most);
  return round_up(div_up(d.vocab, pieces), kTile);
}

// Ways to cut dh's inner dimension (the piece): enough tiles for whole rounds
// of the device's pairs, at least 512 columns each, sums within 256 MB.
int dh_splits(const ls_vocab_desc& d) {
  const int64_t tiles = div_up(d.n_rows, kTile) * div_up(d.hidden, kTile), blocks = div_up(tc_piece(d), kBK);
  const int64_t pairs = device_sms() / 2;
  const bool pieces = tc_piece(d) < d.vocab;
  int best = 1;
  double best_cost = 1e300;
  for (int s = 1; s <= 64; ++s) {
    if (s > 1 && (blocks / s < 8 || s * d.n_rows * d.hidden * 4 > (256ll << 20))) break;
    const int64_t per = div_up(blocks, s);
    // in blocks of a tile's products (about 0.25 us): rounds, an epilogue each, and the sums written and read
    const double rounds = (double)div_up(tiles * s, pairs);
    const double cost = rounds * (per + 3.0) + (s > 1 || pieces ? s * 8.0 * d.n_rows * d.hidden / 6.0e12 / 0.25e-6 : 0.0);
    if (cost < best_cost * 0.98) best_cost = cost, best = s;
  }
  return best;
}

}  // namespace

size_t vocab_tc_scratch(const ls_vocab_desc& d, bool with_grad) {
  const size_t n = (size_t)d.n_rows, nf = (size_t)(d.n_rows < kVocabRows ? d.n_rows : kVocabRows);
  size_t need = (size_t)div_up(d.vocab, kTile) * nf * sizeof(float2) + nf * sizeof(float);
  if (with_grad) {
    const int64_t piece = tc_piece(d);
    const int splits = dh_splits(d);
    size_t g = round_up(n * round_up(piece, 64) * 2, 256);
    if (splits > 1 || piece < d.vocab) g += (size_t)splits * n * d.hidden * sizeof(float);
    need = g > need ? g : need;
  }
  return round_up(need, 256);
}

cudaError_t launch_vocab_tc_fwd(const VocabParams& v, cudaStream_t s) {
  const ls_vocab_desc& d = v.d;
  CUtensorMap a, b;
  if (!k_major(&a, v.h, d.n_rows, d.hidden, d.h_stride) || !k_major(&b, v.w, d.vocab, d.hidden, d.w_stride))
    return cudaErrorInvalidValue;
  ProductParams p{};
  p.m = (int32_t)d.n_rows, p.n = d.vocab, p.k = d.hidden;
  p.m_tiles = (int32_t)div_up(p.m, kTile), p.n_tiles = (int32_t)div_up(p.n, kTile);
  p.splits = 1, p.k_blocks = (int32_t)div_up(p.k, kBK);
  p.m_fast = 1;  // the weight passes once, h stays in L2
  p.vocab = d.vocab;
  p.scale = d.logit_scale, p.scale_log2 = d.logit_scale * kLog2e;
  p.targets = v.targets;
  p.parts = static_cast<float2*>(v.scratch);
  p.hit = reinterpret_cast<float*>(p.parts + (int64_t)p.n_tiles * p.m);
  p.status = v.status;
  const cudaError_t e = run_product<kStats, false, false>(a, b, a, p, s);
  if (e != cudaSuccess) return e;
  return launch_vocab_join(p.n_tiles, v, p.parts, p.hit, s);
}

cudaError_t launch_vocab_tc_bwd(const VocabParams& v, cudaStream_t s) {
  const ls_vocab_desc& d = v.d;
  const int64_t piece = tc_piece(d), ld = round_up(piece, 64);
  const int splits = dh_splits(d);
  const bool direct = splits == 1 && piece == d.vocab;
  __nv_bfloat16* slope = static_cast<__nv_bfloat16*>(v.scratch);
  float* sums = reinterpret_cast<float*>(static_cast<char*>(v.scratch) + round_up((size_t)d.n_rows * ld * 2, 256));
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(v.w);
  CUtensorMap hk, hm;
  int32_t h_boxes = 1;
  if (!k_major(&hk, v.h, d.n_rows, d.hidden, d.h_stride) || !mn_major(&hm, v.h, d.n_rows, d.hidden, d.h_stride, &h_boxes))
    return cudaErrorInvalidValue;
  for (int64_t v0 = 0; v0 < d.vocab; v0 += piece) {
    const int64_t np = d.vocab - v0 < piece ? d.vocab - v0 : piece;
    CUtensorMap wk, wm, sk, sm, so, dho, dwo;
    memset(&dho, 0, sizeof(dho));
    memset(&dwo, 0, sizeof(dwo));
    int32_t w_boxes = 1, s_boxes = 1;
    if (!k_major(&wk, w + v0 * d.w_stride, np, d.hidden, d.w_stride) ||
        !mn_major(&wm, w + v0 * d.w_stride, np, d.hidden, d.w_stride, &w_boxes) ||
        !k_major(&sk, slope, d.n_rows, np, ld) || !mn_major(&sm, slope, d.n_rows, ld, ld, &s_boxes) ||
        !output(&so, slope, d.n_rows, np, ld) || (v.dh && !output(&dho, v.dh, d.n_rows, d.hidden, d.hidden)) ||
        (v.dw && !output(&dwo, static_cast<__nv_bfloat16*>(v.dw) + v0 * d.hidden, np, d.hidden, d.hidden)))
      return cudaErrorInvalidValue;
    ProductParams p{};
    p.m = (int32_t)d.n_rows, p.n = (int32_t)np, p.k = d.hidden;
    p.m_tiles = (int32_t)div_up(p.m, kTile), p.n_tiles = (int32_t)div_up(p.n, kTile);
    p.splits = 1, p.k_blocks = (int32_t)div_up(p.k, kBK);
    p.m_fast = 1;
    p.v0 = (int32_t)v0, p.vocab = d.vocab;
    p.scale = d.logit_scale, p.scale_log2 = d.logit_scale * kLog2e;
    p.targets = v.targets;
    p.lse = v.lse_in;
    p.d_logp = v.d_logp;
    p.status = v.status;
    cudaError_t e = run_product<kSlope, false, false>(hk, wk, so, p, s);
    if (e != cudaSuccess) return e;
    if (v.dh) {
      ProductParams g{};
      g.m = (int32_t)d.n_rows, g.n = d.hidden, g.k = (int32_t)np;
      g.m_tiles = (int32_t)div_up(g.m, kTile), g.n_tiles = (int32_t)div_up(g.n, kTile);
      // the last piece may be shorter: splits past its end have no blocks and are left out
      g.k_blocks = (int32_t)div_up(div_up(piece, kBK), splits);
      g.splits = (int32_t)div_up(div_up(np, kBK), g.k_blocks);
      g.m_fast = 1;
      g.b_boxes = w_boxes;
      g.sums = direct ? nullptr : sums;
      g.add = v0 > 0;
      g.status = v.status;
      e = run_product<kOut, false, true>(sk, wm, dho, g, s);
      if (e != cudaSuccess) return e;
    }
    if (v.dw) {
      ProductParams g{};
      g.m = (int32_t)np, g.n = d.hidden, g.k = (int32_t)d.n_rows;
      g.m_tiles = (int32_t)div_up(g.m, kTile), g.n_tiles = (int32_t)div_up(g.n, kTile);
      g.splits = 1, g.k_blocks = (int32_t)div_up(g.k, kBK);
      g.m_fast = 0;  // a strip of D serves all columns, h stays in L2
      g.a_boxes = s_boxes, g.b_boxes = h_boxes;
      g.status = v.status;
      e = run_product<kOut, true, true>(sm, hm, dwo, g, s);
      if (e != cudaSuccess) return e;
    }
  }
  if (v.dh && !direct) {
    const int64_t n = d.n_rows * d.hidden;
    const int64_t used = div_up(div_up(piece, kBK), div_up(div_up(piece, kBK), splits));
    LaunchScope ls(kKVocabReduce, s);
    vocab_sum_kernel<<<(unsigned)div_up(n, 1024), 256, 0, s>>>((int)used, n, sums, static_cast<__nv_bfloat16*>(v.dh));
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace ls
