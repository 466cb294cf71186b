// nq_paged_cluster.cuh -- blocks of a thread-block cluster: who they are, their barrier, and writes into another's shared memory.
#pragma once

#include <cstdint>

namespace nq {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Eight bytes to the same place in block `rank`'s shared memory.
__device__ __forceinline__ void store_remote(void* place, uint32_t rank, uint64_t v) {
    uint32_t addr = uint32_t(__cvta_generic_to_shared(place));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

}  // namespace nq
