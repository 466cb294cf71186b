// nq_paged_device.cuh -- device building blocks of the paged attention kernels: bounded barrier waits, TMA tile
// loads, 16-bit type conversion, and what a request's lengths mean.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "nq_paged.h"

namespace nq {

constexpr int kKeyTile = 128;   // keys per tile, in both kernels
constexpr int kHalfBytes = kKeyTile * 128;  // a tile's 64 columns: 128 rows of 128 bytes, 128-byte swizzle

// ------------------------------------------------------------------ barriers

__device__ __forceinline__ uint32_t smem_ptr(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Suspended for as long as the hardware allows (it is asked for a millisecond and comes back after 4 us): a waiting warp that
// comes back to look takes issue slots from the ones that compute (with the default limit the large kernel took 3 to 7% longer).
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// A wait gives up after this long (a tile takes microseconds), so that a mistake ends as an error and not as a hang.
constexpr uint64_t kWaitNs = 2000000000ull;

// Waits for the phase of `parity` to end.  Returns false when it does not within kWaitNs, or, after 17 tries (65 us), when another
// thread of the block has given up (*gave_up); the caller goes on without its data, so that all barriers of the block are still
// passed, each within that time.  (Looking at the flag after every try, and leaving the tile loops, made the large kernel 1 to 6% slower.)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
    if (mbar_try(bar, parity)) return true;
    uint64_t since = 0;
    for (int i = 0;; ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 15) != 15) continue;
        if (*gave_up) return false;
        const uint64_t now = global_ns();
        if (since == 0) since = now;
        if (now - since > kWaitNs) {
            *gave_up = 1;
            return false;
        }
    }
}

template <int ID, int THREADS>
__device__ __forceinline__ void named_barrier() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// ------------------------------------------------- programmatic dependent launch

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Returns when the kernels before this one have ended and their writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ----------------------------------------------------------------------- TMA

// Box [1 page][1 head][rows][64 columns] of a pool -> swizzled shared memory.  x is 0 or 64: 16-byte aligned.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int slot, int head,
                                             int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(slot), "r"(head), "r"(page)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// --------------------------------------------------------------------- types

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// The two values of a packed pair of bf16.
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// exp(s - m) goes to the tensor cores in 16 bits.  fp16 loses digits below 2^-14 and everything below 2^-25, and a long context
// has that many small weights that their sum counts.  So there they go in 2^LIFT times as large, up to 2^15: 14 in the small
// kernel, whose largest is 1, and 7 in the large one, whose largest is 2^8 (weights below 2^-39 and 2^-32 are lost, 2^-15 of a result over
// 131072 keys at most).  bf16 has fp32's range and needs none.
template <bool BF16, int LIFT>
constexpr float kLift = BF16 ? 0.0f : float(LIFT);
template <bool BF16, int LIFT>
constexpr float kLifted = BF16 ? 1.0f : float(1 << LIFT);

// -------------------------------------------------------------------- shares

// `total` tiles over the first min(total, kAttnGrid) blocks, sizes differing by one: block b's begin at
// floor(total b / parts).
struct Shares {
    long long total, each;
    uint32_t parts, more;  // total = each * parts + more
    __host__ __device__ __forceinline__ explicit Shares(long long t) : total(t) {
        parts = uint32_t(min(max(t, 1LL), (long long)kAttnGrid));
        each = t / parts;
        more = uint32_t(t - each * parts);
    }
    __host__ __device__ __forceinline__ long long begin(uint32_t b) const {
        return b >= parts ? total : each * b + more * b / parts;
    }
};
// The block whose share holds tile `at` (< total): the last b with total b / parts < at + 1.  Never past the grid, whatever
// `at` is: the join takes the workspace's slots from it.
__host__ __device__ __forceinline__ int share_holding(long long total, long long at) {
    const long long parts = min(total, (long long)kAttnGrid);
    return int(min(((at + 1) * parts - 1) / total, (long long)kAttnGrid - 1));
}

// ------------------------------------------------------------------- lengths

// A request's rows [begin, begin + n) of q and its cached length, with the device's values clamped to the buffers.
struct Request {
    int begin, n, kv;
};

__host__ __device__ __forceinline__ int load_kv(const AttnArgs& a, int r) {
    return int(min(int64_t(max(a.kv_lens[r], 0)), int64_t(a.table_cols) << a.page_shift));
}
__host__ __device__ __forceinline__ Request load_request(const AttnArgs& a, int r) {
    Request q;
    q.begin = min(max(a.q_start[r], 0), a.tokens);
    q.n = max(min(max(a.q_start[r + 1], 0), a.tokens) - q.begin, 0);
    q.kv = load_kv(a, r);
    return q;
}

// First key that a row at position p sees, and the end of its keys.
__host__ __device__ __forceinline__ int keys_from(const AttnArgs& a, int p) {
    return a.window > 0 ? int(max(int64_t(p) - a.window + 1, int64_t(0))) : 0;
}
__host__ __device__ __forceinline__ int keys_to(const AttnArgs& a, int kv, int p) {
    return a.causal ? max(min(kv, p + 1), 0) : kv;
}

}  // namespace nq
