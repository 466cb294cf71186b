// nq_paged.h -- declarations shared by the paged-cache translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/nq.h"

namespace nq {

inline bool paged_aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool paged_page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

// log2 of a page size.
inline int paged_page_shift(int p) {
    int s = 4;
    while ((1 << s) < p) ++s;
    return s;
}

// A stride in elements of an axis of `extent` rows; the stride of a single row is never used.
inline bool paged_stride_ok(int64_t stride, int64_t extent, int64_t least) {
    return extent <= 1 || (stride >= least && stride % 8 == 0 && stride < (int64_t(1) << 39));
}

inline int check_pool(const nq_pool* p) {
    if (!p) return NQ_ERR_ARG;
    if (p->dtype != NQ_F16 && p->dtype != NQ_BF16) return NQ_ERR_UNSUPPORTED;
    if (p->head_dim != 64 && p->head_dim != 96 && p->head_dim != 128) return NQ_ERR_UNSUPPORTED;
    if (!paged_page_size_ok(p->page_size)) return NQ_ERR_UNSUPPORTED;
    if (p->pages < 1 || p->kv_heads < 1) return NQ_ERR_ARG;
    if (!paged_stride_ok(p->page_stride, p->pages, p->head_dim) ||
        !paged_stride_ok(p->head_stride, p->kv_heads, p->head_dim) ||
        !paged_stride_ok(p->slot_stride, p->page_size, p->head_dim))
        return NQ_ERR_ARG;
    return NQ_OK;
}

// Streaming multiprocessors of the current device, 0 when it cannot be queried.
int paged_sm_count();

// What the attention kernels know of a call.
struct AttnArgs {
    const void* q;
    void* out;
    float* lse;
    const int32_t* table;
    const int32_t* q_start;
    const int32_t* kv_lens;
    const void* k_pages;
    const void* v_pages;
    void* workspace;
    int64_t table_stride, q_token_stride, q_head_stride, out_token_stride, out_head_stride;
    int64_t page_stride, head_stride, slot_stride;
    int tokens, q_heads, kv_heads, group, requests, table_cols, page_shift, pages, head_dim, causal, window;
    int bf16;
    float scale;
    cudaStream_t stream;
};

}  // namespace nq
