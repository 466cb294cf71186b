// nq_page_release.cu -- pages past the tokens that requests keep, back to the free list.
//
// The k-th released page (requests in order, columns in order) goes to free_pages[top - 1 - k]: the free list is a stack whose
// top is at the front of what is free, where the page map takes from.  Which columns are released is a running sum over the requests'
// lengths; a page's k also depends on the table, since columns that never got a page (the list had run out) give none back.  So one
// cluster of blocks takes a call: each block forms the sums itself, 512 requests at a time, each warp reads an equal part of the columns
// into shared memory and counts its pages, the blocks tell each other their counts, and then each warp knows its first page's k.
// Measured (median of graph replays): 64 requests that give back a page or none 4.6 to 4.9 us, 512 that give back 129362 pages 8.5 to
// 8.8 us: the launch, two chains of dependent loads, the scan's barriers, and 16 multiprocessors that take 32 columns in 30 cycles each.
// (Clusters of 8 blocks 4.5 and 14.4, blocks of 256 threads 4.2 and 16.1, of 1024 6.4 and 9.8; columns loaded into registers by an unrolled
// loop 6.1 and 9.3, the code being fetched anew for every call.  As many blocks as fit, none of which knows of columns without pages
// elsewhere, took 2.6 and 4.7.)
#include "nq_paged.h"
#include "nq_paged_cluster.cuh"

#include <algorithm>

namespace nq {
namespace {

constexpr int kReleaseThreads = 512, kReleaseWarps = kReleaseThreads / 32;
constexpr int kReleaseBlocks = 16;  // of the cluster, at most
constexpr int kGroups = 16;         // of 32 columns, of a warp in a round

// Four bytes into this thread's place.
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Sum of x over the lanes up to this one.
template <typename T>
__device__ __forceinline__ T sum_upto(T x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T v = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += v;
    }
    return x;
}

// CLEAR: -1 into the columns whose pages went on the list.
template <bool CLEAR>
__global__ void __launch_bounds__(kReleaseThreads)
    page_release_kernel(int32_t* table, int64_t table_stride, int table_cols,
                        const int32_t* __restrict__ kv_lens, const int32_t* __restrict__ keep_lens, int requests, int page_shift,
                        int32_t* free_pages, int top, int32_t* counts) {
    __shared__ long long s_upto[kReleaseThreads];  // columns released by the chunk's requests up to this one's end
    __shared__ int s_end[kReleaseThreads];         // the request's last column + 1
    __shared__ long long s_warp[kReleaseWarps];    // columns of a warp's requests
    __shared__ int s_pages[kReleaseWarps];         // pages of a warp's columns
    __shared__ int s_page[kReleaseWarps][kGroups][32];  // a warp's columns of a round
    __shared__ uint64_t s_block[2][kReleaseBlocks];  // by turns, of each block: twice the pages of its columns, and 1 when it has more
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    cluster_arrive();  // the blocks' shared memory exists
    const long long cols = table_cols, P = 1ll << page_shift;
    long long before = 0;  // pages of the earlier chunks
    int turn = 0;
    for (long long r0 = 0; r0 < requests; r0 += kReleaseThreads) {
        const long long r = r0 + threadIdx.x;
        long long end = 0, need = 0;
        if (r < requests) {
            const long long len = max(kv_lens[r], 0), keep = max(keep_lens[r], 0);
            end = min((len + P - 1) >> page_shift, cols);
            need = max(end - ((keep + P - 1) >> page_shift), 0ll);
        }
        long long x = sum_upto(need, lane);
        __syncthreads();  // the previous chunk is read
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        const long long warps_upto = sum_upto(lane < kReleaseWarps ? s_warp[lane] : 0ll, lane), total = __shfl_sync(0xffffffffu, warps_upto, 31);
        const long long warps_before = __shfl_sync(0xffffffffu, warps_upto, max(warp - 1, 0));
        if (warp > 0) x += warps_before;
        s_upto[threadIdx.x] = x;
        s_end[threadIdx.x] = int(end);
        __syncthreads();

        // Rounds of equal parts for all warps, whole groups of 32 columns, until every block has seen its last: what a block tells the
        // others is its pages and whether it has more columns, so that lengths that change meanwhile, by mistake, cannot part them.
        const long long warps = (long long)blocks * kReleaseWarps;
        const long long part = min(((total + warps - 1) / warps + 31) & ~31ll, 32ll * kGroups);
        long long begin = 0;
        for (bool more = true; more; begin += part * warps, turn ^= 1) {
            const long long from = min(begin + part * ((long long)rank * kReleaseWarps + warp), total), to = min(from + part, total);
            const int groups = int((to - from + 31) >> 5);
            // f(group, this lane's entry, whether it has one) for the groups in order.
            auto each = [&](auto f) {
                int at = 0;              // a group's first column is this request's (the first whose columns end past it) or a later one's
                long long ends = 0;      // the columns up to its end
                int32_t* row = nullptr;  // row[i] is its column i's entry
                auto go_to = [&](int request) {
                    at = request;
                    ends = s_upto[at];
                    row = table + (r0 + at) * table_stride + (s_end[at] - ends);
                };
                if (from < to) {
                    const int of_32 = 32 * (__ffs(__ballot_sync(0xffffffffu, lane < kReleaseWarps && s_upto[32 * lane + 31] > from)) - 1);
                    go_to(of_32 + __ffs(__ballot_sync(0xffffffffu, s_upto[of_32 + lane] > from)) - 1);
                }
#pragma unroll 1
                for (int u = 0; u < groups; ++u) {
                    const long long first = from + 32 * u, mine = first + lane;
                    int32_t* entry = row + mine;
                    if (min(first + 32, to) > ends) {  // columns of several requests
                        int lo = at;
                        for (int hi = kReleaseThreads - 1; lo < hi;) {
                            const int mid = (lo + hi) >> 1;
                            if (s_upto[mid] > min(mine, to - 1))
                                hi = mid;
                            else
                                lo = mid + 1;
                        }
                        __syncwarp();
                        entry = table + (r0 + lo) * table_stride + (s_end[lo] - s_upto[lo]) + mine;
                        go_to(__shfl_sync(0xffffffffu, lo, 31));
                    }
                    f(u, entry, mine < to);
                }
            };
            each([&](int u, const int32_t* entry, bool there) {
                if (there)
                    copy_async(&s_page[warp][u][lane], entry);
                else
                    s_page[warp][u][lane] = -1;
            });
            copies_wait();  // a lane reads what it copied
            int pages = 0;
            for (int u = 0; u < groups; ++u) pages += __popc(__ballot_sync(0xffffffffu, s_page[warp][u][lane] >= 0));
            if (lane == 0) s_pages[warp] = pages;
            __syncthreads();
            const int pages_upto = sum_upto(lane < kReleaseWarps ? s_pages[lane] : 0, lane);
            if (r0 == 0 && begin == 0) cluster_wait();
            if (warp == 0) {
                const uint64_t told = uint64_t(__shfl_sync(0xffffffffu, pages_upto, 31)) << 1 | (begin + part * warps < total ? 1 : 0);
                if (lane < int(blocks)) store_remote(&s_block[turn][rank], lane, told);
            }
            __syncwarp();
            cluster_arrive();
            const int warps_pages = __shfl_sync(0xffffffffu, pages_upto, max(warp - 1, 0));
            long long k = before + (warp > 0 ? warps_pages : 0);  // of this warp's first page
            cluster_wait();
            more = false;
#pragma unroll
            for (uint32_t b = 0; b < kReleaseBlocks; ++b) {
                const uint64_t told = b < blocks ? s_block[turn][b] : 0;
                if (b < rank) k += told >> 1;
                before += told >> 1;
                more = more || (told & 1);
            }
            int left = int(max(top - k, 0ll));  // places on the list in front of this warp's
            auto put = [&](int u) {
                const int page = s_page[warp][u][lane];
                const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
                const int to_list = left - 1 - __popc(have & ((1u << lane) - 1));
                left -= __popc(have);
                if (page < 0 || to_list < 0) return false;
                free_pages[to_list] = page;
                return true;
            };
            if constexpr (CLEAR) {
                each([&](int u, int32_t* entry, bool) {
                    if (put(u)) *entry = -1;
                    __syncwarp();
                });
            } else {
                for (int u = 0; u < groups; ++u) put(u);
            }
        }
    }
    if (requests == 0) cluster_wait();
    if (rank == 0 && threadIdx.x == 0) {
        counts[0] = int(min(before, (long long)INT32_MAX));
        counts[1] = int(min(max(before - top, 0ll), (long long)INT32_MAX));
    }
}

// Blocks for a call: what takes all columns that there may be in one round, 16 at most and 8 where a cluster cannot be larger.
template <bool CLEAR>
unsigned cluster_blocks(int requests, int table_cols) {
    static std::mutex mu;
    static std::map<int, unsigned> most;  // per device
    const int64_t most_columns = int64_t(requests) * table_cols;
    unsigned blocks = 1;
    while (blocks < kReleaseBlocks && most_columns > int64_t(blocks) * kReleaseThreads * kGroups) blocks *= 2;
    int device = 0;
    if (blocks <= 8 || cudaGetDevice(&device) != cudaSuccess) return std::min(blocks, 8u);
    std::lock_guard<std::mutex> lock(mu);
    auto& known = most[device];
    if (known == 0) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = kReleaseBlocks;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kReleaseBlocks);
        cfg.blockDim = dim3(kReleaseThreads);
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        const auto kernel = page_release_kernel<CLEAR>;
        known = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0
                    ? kReleaseBlocks
                    : 8;
    }
    return known;
}

template <bool CLEAR>
int release(int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* kv_lens, const int32_t* keep_lens,
            int32_t requests, int32_t page_size, int32_t* free_pages, int32_t top, int32_t* counts, void* stream) {
    if (requests < 0 || table_cols < 0 || top < 0) return NQ_ERR_ARG;
    if (!paged_page_size_ok(page_size)) return NQ_ERR_UNSUPPORTED;
    if (!counts) return NQ_ERR_ARG;
    if (requests > 0 && (!kv_lens || !keep_lens)) return NQ_ERR_ARG;
    if (requests > 0 && table_cols > 0 && !block_table) return NQ_ERR_ARG;
    if (requests > 1 && table_stride < table_cols) return NQ_ERR_ARG;
    if (top > 0 && !free_pages) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(kv_lens),
                          static_cast<const void*>(keep_lens), static_cast<const void*>(free_pages),
                          static_cast<const void*>(counts)})
        if (!paged_aligned(p, 4)) return NQ_ERR_ARG;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster_blocks<CLEAR>(requests, table_cols);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(attr.val.clusterDim.x);
    cfg.blockDim = dim3(kReleaseThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, page_release_kernel<CLEAR>, block_table, table_stride, table_cols, kv_lens, keep_lens,
                                             requests, paged_page_shift(page_size), free_pages, top, counts);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace
}  // namespace nq

extern "C" int nq_page_release(const int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* kv_lens,
                               const int32_t* keep_lens, int32_t requests, int32_t page_size, int32_t* free_pages, int32_t top,
                               int32_t* counts, void* stream) {
    return nq::release<false>(const_cast<int32_t*>(block_table), table_stride, table_cols, kv_lens, keep_lens, requests, page_size,
                              free_pages, top, counts, stream);
}

extern "C" int nq_page_release_clear(int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* kv_lens,
                                     const int32_t* keep_lens, int32_t requests, int32_t page_size, int32_t* free_pages, int32_t top,
                                     int32_t* counts, void* stream) {
    return nq::release<true>(block_table, table_stride, table_cols, kv_lens, keep_lens, requests, page_size, free_pages, top, counts,
                             stream);
}
