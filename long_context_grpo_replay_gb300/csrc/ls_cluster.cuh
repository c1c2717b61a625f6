// A cluster of C blocks as one team of threads (C = 1: a block alone; C = 0: the launch says how many).
#pragma once

#include <stdint.h>

namespace ls {

template <int C>
struct Cluster {
  static __device__ __forceinline__ uint32_t rank() {
    if constexpr (C == 1) return 0;
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
  }
  static __device__ __forceinline__ uint32_t size() {
    if constexpr (C != 0) return C;
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
  }
  // Every thread of the cluster arrives; what each wrote before, to shared or
  // global memory, all may read after.
  static __device__ __forceinline__ void sync() {
    if constexpr (C == 1)
      __syncthreads();
    else
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // The same in two halves: arrive, and wait for all the others' arrival.
  static __device__ __forceinline__ void arrive() {
    if constexpr (C != 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  static __device__ __forceinline__ void wait() {
    if constexpr (C != 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // The word that block `r` holds in the place of `p` in this block's shared memory.
  template <typename T>
  static __device__ __forceinline__ T at(const T* p, uint32_t r) {
    static_assert(sizeof(T) == 4 || sizeof(T) == 8, "words");
    if constexpr (C == 1) return *p;
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(r));
    union { T t; uint32_t w; uint64_t d; } u;
    if constexpr (sizeof(T) == 4)
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(u.w) : "r"(b) : "memory");
    else
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(u.d) : "r"(b) : "memory");
    return u.t;
  }
};

}  // namespace ls
