// nq_paged_compact.cu -- accepted rows of drafted tokens to the front of the request's drafted rows, in every layer.
//
// Entry k of a request's path names the drafted row that becomes row k.  Paths increase, so place k is a source only for moves
// before k: a thread may read the sources of several moves before it writes the first.  Each 16-byte piece of a row is moved by one
// thread along the whole path, and no other thread touches it.
//
// Bytes are few (a handful of rows for each request and layer); what takes time is the chain from row starts through path and
// table to the rows.  So a block finds the places once, for two layers where there are enough blocks, and a thread has the
// pieces of kMoves moves in flight.
// Measured (median of graph replays, other pools each time): 64 requests, 48 layers of 8 heads of 128, 62 moved rows in each, 24 MB
// read and written, 7.0 us, 3.5 TB/s (one layer a block 8.0, four 7.2, blocks of 512 threads 10.4); one request, 32 layers 2.5 us, the
// launch and the chain.
#include "nq_paged.h"

namespace nq {
namespace {

constexpr int kCompactThreads = 128, kMoves = 4;

struct CompactArgs {
    const int32_t *table, *q_start, *kv_lens, *path;
    uint16_t *k_pages, *v_pages;
    int64_t table_stride, layer_stride, page_stride, head_stride, slot_stride;
    int tokens, table_cols, page_shift, pages, layers, vecs, row_vecs;  // vecs: 16-byte pieces of a head's row; row_vecs: of a token's
};

// Block (request, `each` layers, K or V).
__global__ void __launch_bounds__(kCompactThreads) paged_compact_kernel(const CompactArgs a, int each) {
    __shared__ int64_t s_src[32], s_dst[32];  // element offsets of the moves' rows
    __shared__ int s_moves, s_count;
    const int r = blockIdx.x, lane = threadIdx.x & 31;
    const int layer0 = int(blockIdx.y) * each, layers = min(each, a.layers - layer0);
    uint16_t* pool = (blockIdx.z ? a.v_pages : a.k_pages) + layer0 * a.layer_stride;
    const int begin = min(max(a.q_start[r], 0), a.tokens), n = min(max(a.q_start[r + 1], 0), a.tokens) - begin;
    const int64_t ctx = min(int64_t(max(a.kv_lens[r], 0)), int64_t(a.table_cols) << a.page_shift) - n;
    auto row_at = [&](int64_t pos) -> int64_t {
        if (pos < 0) return -1;
        const int page = a.table[r * a.table_stride + (pos >> a.page_shift)];
        if (page < 0 || page >= a.pages) return -1;
        return page * a.page_stride + (pos & ((1 << a.page_shift) - 1)) * a.slot_stride;
    };
    for (int k0 = 0; k0 < n; k0 += 32) {
        if (k0 > 0) __syncthreads();  // the last moves are read
        if (threadIdx.x < 32) {
            const int k = k0 + lane;
            const int from = k < n ? a.path[begin + k] : -1;
            int before = __shfl_up_sync(0xffffffffu, from, 1);
            if (lane == 0) before = k0 > 0 ? a.path[begin + k0 - 1] : -1;
            const uint32_t bad = __ballot_sync(0xffffffffu, !(from > before && from < n));
            const int count = bad ? __ffs(bad) - 1 : 32;
            int64_t src = -1, dst = -1;
            if (lane < count && from != k) {
                src = row_at(ctx + from);
                dst = row_at(ctx + k);
            }
            const uint32_t moves = __ballot_sync(0xffffffffu, src >= 0 && dst >= 0);
            if (moves >> lane & 1u) {
                const int at = __popc(moves & ((1u << lane) - 1));
                s_src[at] = src;
                s_dst[at] = dst;
            }
            if (lane == 0) {
                s_moves = __popc(moves);
                s_count = count;
            }
        }
        __syncthreads();
        const int moves = s_moves;
        for (int x = threadIdx.x; moves > 0 && x < a.row_vecs; x += kCompactThreads) {
            const int h = x / a.vecs, c = x - h * a.vecs;
            for (int layer = 0; layer < layers; ++layer) {
                uint16_t* at = pool + layer * a.layer_stride + h * a.head_stride + 8 * c;
                for (int m0 = 0; m0 < moves; m0 += kMoves) {
                    uint4 w[kMoves];
#pragma unroll
                    for (int i = 0; i < kMoves; ++i)
                        if (m0 + i < moves) w[i] = *reinterpret_cast<const uint4*>(at + s_src[m0 + i]);
#pragma unroll
                    for (int i = 0; i < kMoves; ++i)
                        if (m0 + i < moves) *reinterpret_cast<uint4*>(at + s_dst[m0 + i]) = w[i];
                }
            }
        }
        if (s_count < 32) break;
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
    if (k_pages == v_pages) return NQ_ERR_ARG;  // rows of one would move twice
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
    a.layers = layers;
    a.vecs = pool->head_dim / 8;
    a.row_vecs = pool->kv_heads * a.vecs;
    // two layers a block when that leaves sixteen blocks for each of 152 multiprocessors, as many as run at once
    const int each = int64_t(requests) * layers >= 152 * 16 ? 2 : 1;
    nq::paged_compact_kernel<<<dim3(requests, (layers + each - 1) / each, 2), nq::kCompactThreads, 0,
                               static_cast<cudaStream_t>(stream)>>>(a, each);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
