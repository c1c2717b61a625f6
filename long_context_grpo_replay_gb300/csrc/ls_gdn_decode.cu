// Recurrent step of the gated-DeltaNet state: one or a few new tokens of each
// sequence move its state S [dv][dk] on (the recurrence of ls_gdn.cu),
//   u = S k,  w = v - a u,  S <- a S + b w k^T,  o = S q,  a = exp(g).
//
// A token does 7 operations an element of a state that has to come from memory
// and go back, so for a token or two the states' bytes bound it.  A row of S needs k,
// q and its own element of v alone: the unit of work is half a head, 64 rows or 32 KB,
// for all of a sequence's tokens, and a block of the launch.  Three blocks an SM begin;
// a block that is through with its unit takes that of one that has not begun (they
// differ by their tokens; dealt out in turn the last SMs end a tenth later).  A
// producer warp brings the coming units into a ring of two stages by bulk copies
// (state, and the tokens' k, q and v as they lie; the gates by 4-byte copies), so that
// some 190 KB an SM are on their way whatever the others do.  Four warps hold the rows
// in registers, eight lanes four rows with sixteen columns each, on packed pairs of
// floats; the four row sums are four shuffles.  The results leave by plain stores, the
// states' in whole lines, a token's in runs of four elements.
//   Measured: 96 sequences x 32 heads, one token, 405 MB in 63.7 us (6.4 TB/s, 94 % of
// a copy's rate; with units dealt out 69.5, without the ring 92).  From four tokens on the
// arithmetic counts, 6 to 7 us a token for 64 x 32 heads: 1 to 6 drafted tokens of 64
// sequences 39.0 us (dealt out 43), where the states' bytes would take 22; 16 tokens 128
// us.  Units dealt out, two rows to eight lanes in twice the warps took 144 us for
// those, four rows to sixteen lanes 180; a token's operands loaded, and its sums taken,
// beside the one before it were no faster.
#include <atomic>

#include "ls_internal.h"
#include "ls_tc.cuh"

namespace ls {
namespace {

constexpr int kD = 128;                 // dk = dv
constexpr int kRows = 64;               // rows of a unit
constexpr int kWarps = 4;               // that compute
constexpr int kGroupRows = 4;           // rows of eight lanes: group, group + 16, + 32, + 48
constexpr int kThreads = kWarps * 32 + 32;
constexpr int kStages = 2;
constexpr int kBlocks = 3;               // an SM's

template <typename T>
struct Stage {
  static constexpr int kTokens = 16 / (int)sizeof(T);  // a stage's
  alignas(16) float s[kRows][kD];
  alignas(16) T k[kTokens][kD], q[kTokens][kD], v[kTokens][kRows];
  float g[kTokens], b[kTokens];
  int64_t tok, from;                    // first token; element where the unit's rows begin in `states`, or -1
  int32_t nt, head, row;                // tokens (-1: no more units)
  int32_t first, last;                  // the unit begins, ends here
};
template <typename T>
struct Shared {
  Stage<T> stage[kStages];
  alignas(16) uint4 answer;              // which unit comes next
  alignas(8) uint64_t full[kStages], empty[kStages], answered;
  uint32_t abort;
};

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

// Four elements as two pairs of floats.
__device__ __forceinline__ void pairs4(const float* p, uint64_t (&x)[2]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p);
  x[0] = a.x, x[1] = a.y;
}
__device__ __forceinline__ void pairs4(const __nv_bfloat16* p, uint64_t (&x)[2]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  x[0] = tc::f2(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u));
  x[1] = tc::f2(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
}
__device__ __forceinline__ float both(uint64_t x) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
  return lo + hi;
}
// This lane's sixteen columns of a token's k or q, or of a row of the state: 4 (l + 8 j) + 0..3.
template <typename T>
__device__ __forceinline__ void columns(const T* p, int l, uint64_t (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t y[2];
    pairs4(p + 4 * (l + 8 * j), y);
    x[2 * j] = y[0], x[2 * j + 1] = y[1];
  }
}
// The four rows' products with x, summed over eight lanes in four shuffles: lane l gets row l / 2's.
__device__ __forceinline__ float row_sums(const uint64_t (&s)[kGroupRows][8], const uint64_t (&x)[8], int l) {
  uint64_t y[kGroupRows] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int r = 0; r < kGroupRows; ++r) y[r] = tc::f2_fma(s[r][j], x[j], y[r]);
  const float z[kGroupRows] = {both(y[0]), both(y[1]), both(y[2]), both(y[3])};
  const bool four = l & 4, two = l & 2;
  float a = four ? z[2] : z[0], b = four ? z[3] : z[1];
  a += __shfl_xor_sync(0xffffffffu, four ? z[0] : z[2], 4);
  b += __shfl_xor_sync(0xffffffffu, four ? z[1] : z[3], 4);
  float c = two ? b : a;
  c += __shfl_xor_sync(0xffffffffu, two ? a : b, 2);
  c += __shfl_xor_sync(0xffffffffu, c, 1);
  return c;
}
// All four in every lane, from what row_sums gave.
__device__ __forceinline__ void share(float y, int l, float (&x)[kGroupRows]) {
  const bool four = l & 4, two = l & 2;
  const float z = __shfl_xor_sync(0xffffffffu, y, 2);
  const float a = two ? z : y, b = two ? y : z;
  const float c = __shfl_xor_sync(0xffffffffu, a, 4), d = __shfl_xor_sync(0xffffffffu, b, 4);
  x[0] = four ? c : a, x[1] = four ? d : b, x[2] = four ? a : c, x[3] = four ? b : d;
}

// A float to shared memory; the barrier hears from the lane when all it asked for has come.
__device__ __forceinline__ void fetch4(float* to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void arrive_fetched(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A block that has units left to start takes the place of one that has not begun, by
// asking the launch for it: the answer is that block's number, or that there is none.
__device__ __forceinline__ void ask(void* answer, uint32_t bar) {
  tc::mbar_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   tc::smem_u32(answer)),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ int asked(const uint4* answer) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(answer);
  int x;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "mov.b128 a, {%1, %2};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
      : "=r"(x)
      : "l"(a.x), "l"(a.y));
  return x;
}

// A sequence's place in the call, as loaded.
struct Place {
  int32_t first, end, use, in, out;
};
__device__ __forceinline__ Place place_of(const GdnDecodeParams& p, int b) {
  Place x;
  x.first = p.q_start[b], x.end = p.q_start[b + 1];
  x.use = p.n_use ? p.n_use[b] : INT32_MIN;
  x.in = p.state_in[b], x.out = p.state_out ? p.state_out[b] : -1;
  return x;
}

// The producer asks for everything and waits for nothing but room: no load's value is
// used here but a unit's number and place, two units before the one that is worked on.
template <typename T>
__device__ __forceinline__ void produce(const GdnDecodeParams& p, Shared<T>& sh) {
  constexpr int K = Stage<T>::kTokens;
  const int lane = threadIdx.x & 31;
  int it = 0, turn = 0;
  // The next stage, once the warps that compute have left it.
  auto take = [&]() -> Stage<T>* {
    const int s = it % kStages;
    if (!__all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&sh.empty[s]), (it / kStages & 1) ^ 1, &sh.abort))) {
      if (lane == 0) sh.abort = 1;
      return nullptr;
    }
    return &sh.stage[s];
  };
  const uint32_t per_seq = 2u * p.d.heads;
  const uint32_t answered = tc::smem_u32(&sh.answered);
  if (lane == 0) ask(&sh.answer, answered);
  for (int unit = (int)blockIdx.x; unit >= 0; ++turn) {
    const uint32_t b = (uint32_t)unit / per_seq, in_seq = (uint32_t)unit - b * per_seq;
    const int half = (int)(in_seq & 1), h = (int)(in_seq >> 1);
    const Place at = place_of(p, (int)b);
    const int64_t first = at.first, n_all = (int64_t)at.end - first, n = p.n_use ? at.use : n_all, in = at.in;
    int64_t out = at.out;
    const bool bad = first < 0 || n_all < 0 || first + n_all > p.d.total_q || n_all > p.d.max_q || n < 0 || n > n_all || in < -1 ||
                     in >= p.d.n_states;
    if ((bad || out >= p.d.n_states) && in_seq == 0 && lane == 0 && p.status) atomicOr(p.status, kStatusBadIndex);
    if (out >= p.d.n_states) out = -1;
    const bool idle = bad || ((n == 0 || !p.o) && (out < 0 || (n == 0 && out == in)));
    const int64_t rows = ((int64_t)h * kD + half * kRows) * kD, state = (int64_t)p.d.heads * kD * kD;
    const int kh = h / (p.d.heads / p.d.key_heads);
    for (int64_t t0 = 0; !idle && (t0 == 0 || t0 < n); t0 += K, ++it) {
      Stage<T>* st = take();
      if (!st) return;
      const uint32_t full = tc::smem_u32(&sh.full[it % kStages]);
      const int nt = n - t0 < K ? (int)(n - t0) : K;
      const bool load = t0 == 0 && in >= 0;
      if (lane == 0) {
        st->tok = first + t0, st->from = out >= 0 ? out * state + rows : -1;
        st->nt = nt, st->head = h, st->row = half * kRows;
        st->first = t0 == 0 ? (in >= 0 ? 1 : 2) : 0, st->last = t0 + K >= n;
        tc::mbar_expect_tx(full, (load ? kRows * kD * 4 : 0) + nt * (2 * kD + kRows) * (int)sizeof(T));
        if (load) tc::bulk_load(tc::smem_u32(st->s), p.states + in * state + rows, kRows * kD * 4, full);
      }
      __syncwarp();
      if (lane < nt) {
        const int64_t tok = first + t0 + lane;
        tc::bulk_load(tc::smem_u32(st->k[lane]), static_cast<const T*>(p.k) + tok * p.d.k_stride + kh * kD, kD * sizeof(T), full);
        tc::bulk_load(tc::smem_u32(st->q[lane]), static_cast<const T*>(p.q) + tok * p.d.q_stride + kh * kD, kD * sizeof(T), full);
        tc::bulk_load(tc::smem_u32(st->v[lane]), static_cast<const T*>(p.v) + tok * p.d.v_stride + h * kD + half * kRows,
                      kRows * sizeof(T), full);
        fetch4(&st->g[lane], p.g + tok * p.d.heads + h);
        fetch4(&st->b[lane], p.beta + tok * p.d.heads + h);
      }
      arrive_fetched(full);
    }
    if (!__all_sync(0xffffffffu, tc::mbar_wait(answered, turn & 1, &sh.abort))) {
      if (lane == 0) sh.abort = 1;
      return;
    }
    unit = asked(&sh.answer);
    __syncwarp();
    if (lane == 0 && unit >= 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read before it is written again
      ask(&sh.answer, answered);
    }
  }
  Stage<T>* st = take();
  if (!st) return;
  if (lane == 0) {
    st->nt = -1;
    tc::mbar_arrive(tc::smem_u32(&sh.full[it % kStages]));
  }
  tc::mbar_arrive(tc::smem_u32(&sh.full[it % kStages]));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocks) gdn_decode_kernel(const GdnDecodeParams p) {
  extern __shared__ __align__(16) char raw[];
  Shared<T>& sh = *reinterpret_cast<Shared<T>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(tc::smem_u32(&sh.full[s]), 33);  // each lane, and the first's word of what it asked for
      tc::mbar_init(tc::smem_u32(&sh.empty[s]), kWarps);
    }
    tc::mbar_init(tc::smem_u32(&sh.answered), 1);
    sh.abort = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  if (warp == kWarps) {
    produce<T>(p, sh);
    if (*(volatile uint32_t*)&sh.abort) {  // a wait gave up: what is on its way lands before the block ends
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane <= kStages) {
        const uint32_t bar = tc::smem_u32(lane < kStages ? &sh.full[lane] : &sh.answered);
        tc::mbar_wait_short(bar, 0), tc::mbar_wait_short(bar, 1);
      }
      if (lane == 0 && p.status) {
        if (!(atomicOr(p.status, kStatusTimeout) & kStatusTimeout)) p.status[1] = (uint32_t)kKGdnDecode << 16 | __LINE__;
      }
    }
    return;
  }
  const int group = tid / 8, l = tid % 8;
  uint64_t s[kGroupRows][8];
  for (int it = 0;; ++it) {
    const int at = it % kStages;
    if (!tc::mbar_wait(tc::smem_u32(&sh.full[at]), it / kStages & 1, &sh.abort)) {
      sh.abort = 1;
      return;
    }
    const Stage<T>& st = sh.stage[at];
    const int nt = st.nt;
    if (nt < 0) return;
    if (st.first == 1) {
#pragma unroll
      for (int r = 0; r < kGroupRows; ++r) columns(st.s[group + 16 * r], l, s[r]);
    } else if (st.first == 2) {
#pragma unroll
      for (int r = 0; r < kGroupRows; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[r][j] = 0;
    }
    const float decay = lane < nt ? expf(st.g[lane]) : 0.f;  // a lane a token
    T* o = p.o ? static_cast<T*>(p.o) + (st.tok * p.d.heads + st.head) * kD + st.row + group + 16 * (l / 2) : nullptr;
    for (int t = 0; t < nt; ++t) {
      uint64_t k[8];
      columns(st.k[t], l, k);
      const float a = __shfl_sync(0xffffffffu, decay, t), b = st.b[t];
      float u[kGroupRows];
      share(row_sums(s, k, l), l, u);
      const uint64_t a2 = tc::f2(a, a);
#pragma unroll
      for (int r = 0; r < kGroupRows; ++r) {
        const float w = b * (value(st.v[t][group + 16 * r]) - a * u[r]);
        const uint64_t w2 = tc::f2(w, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[r][j] = tc::f2_fma(w2, k[j], tc::f2_mul(a2, s[r][j]));
      }
      if (o) {
        columns(st.q[t], l, k);
        const float x = row_sums(s, k, l);
        if ((l & 1) == 0) put(o, x);
        o += (int64_t)p.d.heads * kD;
      }
    }
    const int64_t to = st.last ? st.from : -1;
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.empty[at]));
    if (to >= 0) {
#pragma unroll
      for (int r = 0; r < kGroupRows; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<ulonglong2*>(p.states + to + (group + 16 * r) * kD + 4 * (l + 8 * j)) =
              make_ulonglong2(s[r][2 * j], s[r][2 * j + 1]);
    }
  }
}

template <typename T>
cudaError_t launch(const GdnDecodeParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed;  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(gdn_decode_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared<T>));
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  const int64_t units = (int64_t)p.d.batch * p.d.heads * 2;
  if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
  gdn_decode_kernel<T><<<(unsigned)units, kThreads, sizeof(Shared<T>), s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdn_decode(const GdnDecodeParams& p, cudaStream_t s) {
  LaunchScope ls(kKGdnDecode, s);
  return p.d.dtype == LS_DTYPE_F32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}

}  // namespace ls
