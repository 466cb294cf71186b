// nq_paged_compact.cu -- accepted rows of drafted tokens to the front of the request's drafted rows, in every layer.
//
// Entry k of a request's path names the drafted row that becomes row k.  Paths increase, so a row's source is never a place that an
// earlier move has written, nor one that a move before it still has to read: each 16-byte piece of a row is moved by one thread
// along the whole path, and no other thread touches it.
#include "nq_paged.h"

#include <algorithm>

namespace nq {
namespace {

constexpr int kCompactThreads = 128;

struct CompactArgs {
    const int32_t *table, *q_start, *kv_lens, *path;
    uint16_t *k_pages, *v_pages;
    int64_t table_stride, layer_stride, page_stride, head_stride, slot_stride;
    int tokens, table_cols, page_shift, pages, vecs, row_vecs;  // vecs: 16-byte pieces of a head's row; row_vecs: of a token's
};

// Block (request, layer, K or V).
__global__ void __launch_bounds__(kCompactThreads) paged_compact_kernel(const CompactArgs a) {
    __shared__ int64_t s_src[32], s_dst[32];  // element offsets of a move's rows, -1: not moved
    __shared__ int s_count;
    const int r = blockIdx.x, lane = threadIdx.x & 31;
    uint16_t* pool = (blockIdx.z ? a.v_pages : a.k_pages) + blockIdx.y * a.layer_stride;
    const int begin = min(max(a.q_start[r], 0), a.tokens), n = min(max(a.q_start[r + 1], 0), a.tokens) - begin;
    const int64_t ctx = min(int64_t(max(a.kv_lens[r], 0)), int64_t(a.table_cols) << a.page_shift) - n;
    auto row_at = [&](int64_t pos) -> int64_t {
        if (pos < 0) return -1;
        const int page = a.table[r * a.table_stride + (pos >> a.page_shift)];
        if (page < 0 || page >= a.pages) return -1;
        return page * a.page_stride + (pos & ((1 << a.page_shift) - 1)) * a.slot_stride;
    };
    for (int k0 = 0; k0 < n; k0 += 32) {
        __syncthreads();  // the last moves are read
        if (threadIdx.x < 32) {
            const int k = k0 + lane;
            const int from = k < n ? a.path[begin + k] : -1, before = k > 0 && k < n ? a.path[begin + k - 1] : -1;
            const bool ok = from > before && from < n;
            const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
            const int count = bad ? __ffs(bad) - 1 : 32;
            const bool moves = lane < count && from != k;
            const int64_t src = moves ? row_at(ctx + from) : -1, dst = moves ? row_at(ctx + k) : -1;
            s_src[lane] = dst < 0 ? -1 : src;
            s_dst[lane] = dst;
            if (lane == 0) s_count = count;
        }
        __syncthreads();
        const int count = s_count;
        for (int x = threadIdx.x; x < a.row_vecs; x += kCompactThreads) {
            const int h = x / a.vecs, c = x - h * a.vecs;
            uint16_t* at = pool + h * a.head_stride + 8 * c;
            for (int k = 0; k < count; ++k)
                if (s_src[k] >= 0)
                    *reinterpret_cast<uint4*>(at + s_dst[k]) = *reinterpret_cast<const uint4*>(at + s_src[k]);
        }
        if (count < 32) break;
    }
}

}  // namespace
}  // namespace nq

extern "C" int nq_paged_compact(const nq_pool* pool, int32_t layers, int64_t layer_stride, void* k_pages, void* v_pages,
                                const int32_t* block_table, int64_t table_stride, int32_t table_cols,
                                const int32_t* q_start, const int32_t* kv_lens, int32_t requests, const int32_t* path,
                                int32_t tokens, void* stream) {
    const int st = nq::check_pool(pool);
    if (st != NQ_OK) return st;
    if (layers < 0 || layers > 65535 || requests < 0 || table_cols < 0 || tokens < 0) return NQ_ERR_ARG;
    if (!nq::paged_stride_ok(layer_stride, layers, pool->head_dim)) return NQ_ERR_ARG;
    if (int64_t(table_cols) * pool->page_size > INT32_MAX - 65536) return NQ_ERR_ARG;
    if (requests > 1 && table_stride < table_cols) return NQ_ERR_ARG;
    if (tokens == 0 || requests == 0 || layers == 0 || table_cols == 0) return NQ_OK;
    if (!k_pages || !v_pages || !block_table || !q_start || !kv_lens || !path) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(k_pages), static_cast<const void*>(v_pages)})
        if (!nq::paged_aligned(p, 16)) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(q_start),
                          static_cast<const void*>(kv_lens), static_cast<const void*>(path)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    nq::CompactArgs a;
    a.table = block_table;
    a.q_start = q_start;
    a.kv_lens = kv_lens;
    a.path = path;
    a.k_pages = static_cast<uint16_t*>(k_pages);
    a.v_pages = static_cast<uint16_t*>(v_pages);
    a.table_stride = table_stride;
    a.layer_stride = layers > 1 ? layer_stride : 0;
    a.page_stride = pool->page_stride;
    a.head_stride = pool->head_stride;
    a.slot_stride = pool->slot_stride;
    a.tokens = tokens;
    a.table_cols = table_cols;
    a.page_shift = nq::paged_page_shift(pool->page_size);
    a.pages = pool->pages;
    a.vecs = pool->head_dim / 8;
    a.row_vecs = pool->kv_heads * a.vecs;
    nq::paged_compact_kernel<<<dim3(requests, layers, 2), nq::kCompactThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
