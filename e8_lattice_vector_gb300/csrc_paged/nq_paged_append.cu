// nq_paged_append.cu -- a step's K and V rows into the page pools.
//
// A pure copy: every row is read once and written once, 16 bytes a thread.
// Both types are 16 bits wide, so the kernel moves bits and knows no type.
#include "nq_paged.h"

#include <algorithm>

namespace nq {
namespace {

constexpr int kAppendThreads = 256;

struct AppendArgs {
    const uint16_t *k, *v;
    uint16_t *k_pages, *v_pages;
    const int64_t* slots;
    int64_t k_token, k_head, v_token, v_head, page_stride, head_stride, slot_stride, n_slots;
    int tokens, vecs, row_vecs, page_shift;  // vecs: 16-byte pieces of a head's row; row_vecs: of a token's
};

// blockIdx.y: 0 = K, 1 = V.
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a) {
    const bool is_v = blockIdx.y != 0;
    const uint16_t* src = is_v ? a.v : a.k;
    uint16_t* dst = is_v ? a.v_pages : a.k_pages;
    const int64_t ts = is_v ? a.v_token : a.k_token, hs = is_v ? a.v_head : a.k_head;
    const int64_t n = int64_t(a.tokens) * a.row_vecs;
    for (int64_t i = int64_t(blockIdx.x) * kAppendThreads + threadIdx.x; i < n;
         i += int64_t(gridDim.x) * kAppendThreads) {
        const int64_t t = i / a.row_vecs;
        const int x = int(i - t * a.row_vecs), h = x / a.vecs, c = x - h * a.vecs;
        const int64_t slot = __ldg(a.slots + t);
        if (slot < 0 || slot >= a.n_slots) continue;
        const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + t * ts + h * hs + 8 * c));
        *reinterpret_cast<uint4*>(dst + page * a.page_stride + h * a.head_stride + off * a.slot_stride + 8 * c) = w;
    }
}

}  // namespace
}  // namespace nq

extern "C" int nq_paged_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                               int64_t v_token_stride, int64_t v_head_stride, int32_t tokens, const int64_t* slots,
                               const nq_pool* pool, void* k_pages, void* v_pages, void* stream) {
    const int st = nq::check_pool(pool);
    if (st != NQ_OK) return st;
    if (tokens < 0) return NQ_ERR_ARG;
    if (tokens == 0) return NQ_OK;
    if (!k || !v || !slots || !k_pages || !v_pages) return NQ_ERR_ARG;
    for (const void* p : {k, v, static_cast<const void*>(k_pages), static_cast<const void*>(v_pages)})
        if (!nq::paged_aligned(p, 16)) return NQ_ERR_ARG;
    if (!nq::paged_aligned(slots, 8)) return NQ_ERR_ARG;
    for (int64_t s : {k_token_stride, v_token_stride})
        if (!nq::paged_stride_ok(s, tokens, 0)) return NQ_ERR_ARG;
    for (int64_t s : {k_head_stride, v_head_stride})
        if (!nq::paged_stride_ok(s, pool->kv_heads, 0)) return NQ_ERR_ARG;
    const int sms = nq::paged_sm_count();
    if (sms <= 0) return NQ_ERR_CUDA;
    nq::AppendArgs a;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.k_pages = static_cast<uint16_t*>(k_pages);
    a.v_pages = static_cast<uint16_t*>(v_pages);
    a.slots = slots;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.page_stride = pool->page_stride;
    a.head_stride = pool->head_stride;
    a.slot_stride = pool->slot_stride;
    a.n_slots = int64_t(pool->pages) * pool->page_size;
    a.tokens = tokens;
    a.vecs = pool->head_dim / 8;
    a.row_vecs = pool->kv_heads * a.vecs;
    a.page_shift = nq::paged_page_shift(pool->page_size);
    const int64_t want = (int64_t(tokens) * a.row_vecs + nq::kAppendThreads - 1) / nq::kAppendThreads;
    const int grid = int(std::min<int64_t>(want, int64_t(sms) * 64));
    nq::paged_append_kernel<<<dim3(grid, 2), nq::kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
