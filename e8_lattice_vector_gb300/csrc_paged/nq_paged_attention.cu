// nq_paged_attention.cu -- attention of a step's new tokens over the paged cache.
//
// One warp for each (row, query head): it walks the visible keys one by one with a
// running maximum and sum, each lane holding head_dim / 32 elements.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "nq_paged.h"

namespace nq {
namespace {

constexpr int kRowThreads = 128;

template <bool BF16>
__device__ __forceinline__ float2 to_float2(uint32_t w) {
    if constexpr (BF16)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ uint32_t from_float2(float x, float y) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) attention_rows_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
    if (item >= int64_t(a.tokens) * a.q_heads) return;
    const int t = int(item / a.q_heads), head = int(item - int64_t(t) * a.q_heads), kvh = head / a.group;
    int r = 0;
    for (; r < a.requests; ++r)
        if (a.q_start[r] <= t && t < a.q_start[r + 1]) break;
    if (r == a.requests) return;  // a row of no request
    const int begin = max(a.q_start[r], 0), end = min(a.q_start[r + 1], a.tokens);
    const int64_t room = int64_t(a.table_cols) << a.page_shift;
    const int kv = int(min(int64_t(max(a.kv_lens[r], 0)), room));
    const int p = kv - (end - begin) + (t - begin);
    const int hi = a.causal ? min(kv, p + 1) : kv;
    const int lo = a.window > 0 ? max(p - a.window + 1, 0) : 0;
    const int pairs = a.head_dim / 2;  // pair lane, lane + 32 of each row
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + t * a.q_token_stride +
                                                          head * a.q_head_stride);
    float2 qv[2], o[2];
    for (int e = 0; e < 2; ++e) {
        o[e] = make_float2(0.0f, 0.0f);
        qv[e] = lane + 32 * e < pairs ? to_float2<BF16>(q[lane + 32 * e]) : make_float2(0.0f, 0.0f);
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = lo; j < hi; ++j) {
        const int page = a.table[r * a.table_stride + (j >> a.page_shift)];
        if (page < 0 || page >= a.pages) continue;
        const int64_t at = page * a.page_stride + kvh * a.head_stride + (j & ((1 << a.page_shift) - 1)) * a.slot_stride;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.k_pages) + at);
        const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v_pages) + at);
        float s = 0.0f;
        for (int e = 0; e < 2; ++e)
            if (lane + 32 * e < pairs) {
                const float2 kk = to_float2<BF16>(k[lane + 32 * e]);
                s = fmaf(qv[e].x, kk.x, fmaf(qv[e].y, kk.y, s));
            }
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        const float mn = fmaxf(m, s), keep = expf(m - mn), w = expf(s - mn);
        l = fmaf(l, keep, w);
        m = mn;
        for (int e = 0; e < 2; ++e)
            if (lane + 32 * e < pairs) {
                const float2 vv = to_float2<BF16>(v[lane + 32 * e]);
                o[e].x = fmaf(o[e].x, keep, w * vv.x);
                o[e].y = fmaf(o[e].y, keep, w * vv.y);
            }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + t * a.out_token_stride +
                                                head * a.out_head_stride);
    for (int e = 0; e < 2; ++e)
        if (lane + 32 * e < pairs) out[lane + 32 * e] = from_float2<BF16>(o[e].x * inv, o[e].y * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[int64_t(t) * a.q_heads + head] = l > 0.0f ? m + logf(l) : -INFINITY;
}

int check_attention(const nq_attention* a, const nq_pool* pool) {
    const int st = check_pool(pool);
    if (st != NQ_OK) return st;
    if (!a) return NQ_ERR_ARG;
    if (a->tokens < 0 || a->requests < 0 || a->table_cols < 0 || a->max_q < 0 || a->window < 0) return NQ_ERR_ARG;
    if (a->causal != 0 && a->causal != 1) return NQ_ERR_ARG;
    if (a->q_heads < 1 || a->q_heads % pool->kv_heads != 0) return NQ_ERR_ARG;
    if (!(a->scale > 0.0f) || !std::isfinite(a->scale)) return NQ_ERR_ARG;
    if (int64_t(a->table_cols) * pool->page_size > INT_MAX) return NQ_ERR_ARG;
    if (a->requests > 1 && a->table_stride < a->table_cols) return NQ_ERR_ARG;
    if (!paged_stride_ok(a->q_token_stride, a->tokens, 0) || !paged_stride_ok(a->q_head_stride, a->q_heads, 0) ||
        !paged_stride_ok(a->out_token_stride, a->tokens, 0) || !paged_stride_ok(a->out_head_stride, a->q_heads, 0))
        return NQ_ERR_ARG;
    return NQ_OK;
}

}  // namespace
}  // namespace nq

extern "C" {

int nq_paged_attention_workspace(const nq_attention* a, const nq_pool* pool, uint64_t* bytes) {
    const int st = nq::check_attention(a, pool);
    if (st != NQ_OK) return st;
    if (!bytes) return NQ_ERR_ARG;
    *bytes = 0;
    return NQ_OK;
}

int nq_paged_attention(const nq_attention* a, const void* q, const nq_pool* pool, const void* k_pages,
                       const void* v_pages, const int32_t* block_table, const int32_t* q_start,
                       const int32_t* kv_lens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream) {
    uint64_t need = 0;
    const int st = nq_paged_attention_workspace(a, pool, &need);
    if (st != NQ_OK) return st;
    if (a->tokens == 0 || a->requests == 0) return NQ_OK;
    if (!q || !k_pages || !v_pages || !q_start || !kv_lens || !out) return NQ_ERR_ARG;
    if (a->table_cols > 0 && !block_table) return NQ_ERR_ARG;
    if (need > 0 && !workspace) return NQ_ERR_ARG;
    for (const void* p : {q, k_pages, v_pages, static_cast<const void*>(out), static_cast<const void*>(workspace)})
        if (!nq::paged_aligned(p, 16)) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(q_start),
                          static_cast<const void*>(kv_lens), static_cast<const void*>(lse)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    if (workspace_bytes < need) return NQ_ERR_SIZE;
    nq::AttnArgs x;
    x.q = q;
    x.out = out;
    x.lse = lse;
    x.table = block_table;
    x.q_start = q_start;
    x.kv_lens = kv_lens;
    x.k_pages = k_pages;
    x.v_pages = v_pages;
    x.workspace = workspace;
    x.table_stride = a->table_stride;
    x.q_token_stride = a->q_token_stride;
    x.q_head_stride = a->q_head_stride;
    x.out_token_stride = a->out_token_stride;
    x.out_head_stride = a->out_head_stride;
    x.page_stride = pool->page_stride;
    x.head_stride = pool->head_stride;
    x.slot_stride = pool->slot_stride;
    x.tokens = a->tokens;
    x.q_heads = a->q_heads;
    x.kv_heads = pool->kv_heads;
    x.group = a->q_heads / pool->kv_heads;
    x.requests = a->requests;
    x.table_cols = a->table_cols;
    x.page_shift = nq::paged_page_shift(pool->page_size);
    x.pages = pool->pages;
    x.head_dim = pool->head_dim;
    x.causal = a->causal;
    x.window = a->window;
    x.bf16 = pool->dtype == NQ_BF16;
    x.scale = a->scale;
    x.stream = static_cast<cudaStream_t>(stream);
    const int64_t items = int64_t(x.tokens) * x.q_heads;
    const int64_t blocks = (items * 32 + nq::kRowThreads - 1) / nq::kRowThreads;
    if (blocks > INT_MAX) return NQ_ERR_ARG;
    if (x.bf16)
        nq::attention_rows_kernel<true><<<int(blocks), nq::kRowThreads, 0, x.stream>>>(x);
    else
        nq::attention_rows_kernel<false><<<int(blocks), nq::kRowThreads, 0, x.stream>>>(x);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // extern "C"
