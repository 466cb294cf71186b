// nq_page_map.cu -- block table and slot map of a serving step from the
// requests' lengths.
//
// Two running sums over the requests fix everything: the row where a
// request's new tokens begin, and the place in the free list where its new pages
// begin.  Column col of request r is new when col >= a = ceil(ctx / P), and its
// page is free[base + col - a]; a token finds its page from these two numbers alone, and
// only tokens in the page that the request had begun before (col < a, never written here)
// read the table.  A new page's first token (offset 0) writes its table entry.
//
// Measured: 8.7 us on the GPU (in a graph) for 311697 tokens of 16 requests and 4.0 us for 64 single tokens, 10 to 12 us a call from Python.
// One launch, because the work is a few microseconds and a second launch would
// double it: every block forms the sums itself, 512 requests at a time, and takes
// the tiles of 512 rows that are its own (tile index modulo the grid).
#include "nq_paged.h"

#include <algorithm>
#include <climits>

namespace nq {
namespace {

constexpr int kMapThreads = 512;

// Inclusive sums of two 64-bit values over the block; `tot_*` the totals.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long& tot_x, long long& tot_y) {
    __shared__ long long wx[kMapThreads / 32], wy[kMapThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x, d), b = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) {
            x += a;
            y += b;
        }
    }
    __syncthreads();  // the previous use of wx, wy is over
    if (lane == 31) {
        wx[warp] = x;
        wy[warp] = y;
    }
    __syncthreads();
    long long bx = 0, by = 0, sx = 0, sy = 0;
#pragma unroll
    for (int w = 0; w < kMapThreads / 32; ++w) {
        if (w < warp) {
            bx += wx[w];
            by += wy[w];
        }
        sx += wx[w];
        sy += wy[w];
    }
    x += bx;
    y += by;
    tot_x = sx;
    tot_y = sy;
}

__device__ __forceinline__ int sat32(long long v) { return v > INT_MAX ? INT_MAX : int(v); }

__global__ void __launch_bounds__(kMapThreads)
    page_map_kernel(const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int requests,
                    const int32_t* __restrict__ free_pages, int n_free, int32_t* table, int64_t table_stride,
                    int table_cols, int page_shift, int tokens, int32_t* __restrict__ q_start,
                    int32_t* __restrict__ kv_lens, int64_t* __restrict__ slots, int32_t* __restrict__ positions,
                    int32_t* __restrict__ counts) {
    __shared__ long long s_start[kMapThreads + 1];  // row of the request's first token; the chunk's end last
    __shared__ long long s_page[kMapThreads];       // base - a: page of new column col is free[this + col]
    __shared__ int s_ctx[kMapThreads], s_held[kMapThreads];
    const int P = 1 << page_shift;
    const long long cols = table_cols;
    long long row0 = 0, page0 = 0, past = 0;  // sums of the earlier chunks
    for (int r0 = 0; r0 < requests; r0 += kMapThreads) {
        const int r = r0 + threadIdx.x;
        long long c = 0, n = 0;
        if (r < requests) {
            c = max(ctx_lens[r], 0);
            n = max(new_lens[r], 0);
        }
        const long long total = c + n;
        const long long held = min((c + P - 1) >> page_shift, cols);
        const long long need = min((total + P - 1) >> page_shift, cols) - held;
        long long x = n, y = need, tx, ty;
        block_scan2(x, y, tx, ty);  // its barriers also end the previous chunk's reads of s_*
        s_start[threadIdx.x] = row0 + x - n;
        s_page[threadIdx.x] = page0 + y - need - held;
        s_ctx[threadIdx.x] = int(c);
        s_held[threadIdx.x] = int(held);
        if (threadIdx.x == 0) s_start[kMapThreads] = row0 + tx;
        const int is_past = __syncthreads_count(r < requests && total > cols << page_shift);
        past += is_past;
        const int chunk = r0 / kMapThreads;
        if (chunk % int(gridDim.x) == int(blockIdx.x) && r < requests) {
            q_start[r] = sat32(row0 + x - n);
            kv_lens[r] = sat32(total);
        }
        // this block's tiles of rows [row0, row0 + tx)
        const long long end = min(row0 + tx, (long long)tokens);
        long long tile = row0 / kMapThreads;
        tile += (long long)((int(blockIdx.x) - int(tile % gridDim.x) + int(gridDim.x)) % int(gridDim.x));
        for (; tile * kMapThreads < end; tile += gridDim.x) {
            const long long i = tile * kMapThreads + threadIdx.x;
            // the last request that starts at or before a row; the tile's first row's is every row's in a long prompt
            const int n = min(kMapThreads, requests - r0);
            auto request_of = [&](long long row, int lo) {
                for (int hi = n; hi - lo > 1;) {
                    const int mid = (lo + hi) >> 1;
                    if (s_start[mid] <= row)
                        lo = mid;
                    else
                        hi = mid;
                }
                return lo;
            };
            int lo = request_of(max(tile * kMapThreads, row0), 0);
            if (i < row0 || i >= end) continue;
            if (lo + 1 < n && s_start[lo + 1] <= i) lo = request_of(i, lo);
            const long long pos = s_ctx[lo] + (i - s_start[lo]);
            const long long col = pos >> page_shift;
            const int off = int(pos) & (P - 1);
            long long page = -1;
            if (col < cols) {
                int32_t* entry = table + int64_t(r0 + lo) * table_stride + col;
                if (col < s_held[lo]) {
                    page = *entry;
                } else {
                    const long long at = s_page[lo] + col;
                    page = at < n_free ? free_pages[at] : -1;
                    if (off == 0) *entry = int(page);
                }
            }
            slots[i] = page >= 0 ? (page << page_shift) + off : -1;
            positions[i] = sat32(pos);
        }
        row0 += tx;
        page0 += ty;
    }
    for (long long i = max(row0, 0LL) + (long long)blockIdx.x * kMapThreads + threadIdx.x; i < tokens;
         i += (long long)gridDim.x * kMapThreads) {
        slots[i] = -1;
        positions[i] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        q_start[requests] = sat32(row0);
        counts[0] = sat32(row0);
        counts[1] = sat32(page0);
        counts[2] = sat32(max(page0 - n_free, 0LL));
        counts[3] = int(past);
    }
}

}  // namespace

int paged_sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

}  // namespace nq

extern "C" int nq_page_map(const int32_t* ctx_lens, const int32_t* new_lens, int32_t requests,
                           const int32_t* free_pages, int32_t n_free, int32_t* block_table, int64_t table_stride,
                           int32_t table_cols, int32_t page_size, int32_t tokens, int32_t* q_start,
                           int32_t* kv_lens, int64_t* slots, int32_t* positions, int32_t* counts, void* stream) {
    if (requests < 0 || n_free < 0 || table_cols < 0 || tokens < 0) return NQ_ERR_ARG;
    if (!nq::paged_page_size_ok(page_size)) return NQ_ERR_UNSUPPORTED;
    if (!q_start || !counts) return NQ_ERR_ARG;
    if (requests > 0 && (!ctx_lens || !new_lens || !kv_lens)) return NQ_ERR_ARG;
    if (requests > 0 && table_cols > 0 && !block_table) return NQ_ERR_ARG;
    if (requests > 1 && table_stride < table_cols) return NQ_ERR_ARG;
    if (n_free > 0 && !free_pages) return NQ_ERR_ARG;
    if (tokens > 0 && (!slots || !positions)) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                          static_cast<const void*>(free_pages), static_cast<const void*>(block_table),
                          static_cast<const void*>(q_start), static_cast<const void*>(kv_lens),
                          static_cast<const void*>(positions), static_cast<const void*>(counts)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    if (!nq::paged_aligned(slots, 8)) return NQ_ERR_ARG;
    const int sms = nq::paged_sm_count();
    if (sms <= 0) return NQ_ERR_CUDA;
    const int64_t tiles = (int64_t(tokens) + nq::kMapThreads - 1) / nq::kMapThreads;
    const int grid = int(std::max<int64_t>(1, std::min<int64_t>(tiles, int64_t(sms) * 4)));
    nq::page_map_kernel<<<grid, nq::kMapThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        ctx_lens, new_lens, requests, free_pages, n_free, block_table, table_stride, table_cols,
        nq::paged_page_shift(page_size), tokens, q_start, kv_lens, slots, positions, counts);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
