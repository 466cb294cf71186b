// nq_paged_append.cu -- a step's K and V rows into the page pools.
//
// A pure copy: every row is read once and written once, 16 bytes a thread, a token's row_vecs pieces on neighbouring
// threads.  Both types are 16 bits wide, so the kernel moves bits and knows no type.  Memory-bound: a thread takes PASS tokens
// so that as many loads are in flight before the first store.
// Measured: a 131072-token cache of 8 heads of 128, head-major as the codec leaves it, 164 us, 6.56 TB/s read and written, 98% of
// the measured copy rate (one vector a thread in a strided loop: 185 us); 64 tokens 8 us a call, the launch.
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

// blockIdx.y: 0 = K, 1 = V.  A block takes PASS times `together` tokens, as many as its threads hold rows of (at least one).
template <int PASS>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a, int together) {
    const bool is_v = blockIdx.y != 0;
    const uint16_t* src = is_v ? a.v : a.k;
    uint16_t* dst = is_v ? a.v_pages : a.k_pages;
    const int64_t ts = is_v ? a.v_token : a.k_token, hs = is_v ? a.v_head : a.k_head;
    const int mine = int(threadIdx.x) / a.row_vecs;  // of the tokens taken together
    if (mine >= together) return;
    const int64_t t0 = int64_t(blockIdx.x) * PASS * together + mine;
    for (int x = threadIdx.x - mine * a.row_vecs; x < a.row_vecs; x += kAppendThreads) {
        const int h = x / a.vecs, c = x - h * a.vecs;
        int64_t slot[PASS];
        uint4 w[PASS];
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int64_t t = t0 + i * together;
            slot[i] = t < a.tokens ? __ldg(a.slots + t) : -1;
        }
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int64_t t = min(t0 + i * together, int64_t(a.tokens) - 1);
            w[i] = __ldg(reinterpret_cast<const uint4*>(src + t * ts + h * hs + 8 * c));
        }
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            if (slot[i] < 0 || slot[i] >= a.n_slots) continue;
            const int64_t page = slot[i] >> a.page_shift, off = slot[i] & ((1 << a.page_shift) - 1);
            *reinterpret_cast<uint4*>(dst + page * a.page_stride + h * a.head_stride + off * a.slot_stride + 8 * c) = w[i];
        }
    }
}

template <int PASS>
int launch_append(const AppendArgs& a, int together, cudaStream_t stream) {
    const int64_t blocks = (int64_t(a.tokens) + PASS * together - 1) / (PASS * together);
    paged_append_kernel<PASS><<<dim3(unsigned(blocks), 2), kAppendThreads, 0, stream>>>(a, together);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
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
    const int together = std::max(nq::kAppendThreads / a.row_vecs, 1);
    // one pass while that does not fill the GPU (152 multiprocessors of eight blocks): then latency counts
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return 2 * (int64_t(tokens) / together) < 152 * 8 ? nq::launch_append<1>(a, together, s)
                                                      : nq::launch_append<4>(a, together, s);
}
