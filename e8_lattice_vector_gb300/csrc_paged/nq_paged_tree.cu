// nq_paged_tree.cu -- attention of drafted trees over the paged cache.
//
// Simplest form: a block for a request and query head, four warps that take every fourth key, the dimensions on the lanes.
#include "nq_paged_device.cuh"

namespace nq {
namespace {

constexpr int kTreeWarps = 4;

template <bool BF16>
__device__ __forceinline__ float load16(const void* base, int64_t at) {
    if constexpr (BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
    else
        return __half2float(static_cast<const __half*>(base)[at]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kTreeWarps * 32) attention_tree_kernel(const AttnArgs a) {
    constexpr int E = D / 32;
    __shared__ float s_o[kTreeWarps][D], s_m[kTreeWarps], s_l[kTreeWarps];
    const int r = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Request q = load_request(a, r);
    const int ctx = q.kv - q.n;
    for (int i = 0; i < q.n; ++i) {
        const int t = q.begin + i;
        float x[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = load16<BF16>(a.q, t * a.q_token_stride + h * a.q_head_stride + lane + 32 * e);
            o[e] = 0.0f;
        }
        const int from = a.window > 0 ? tree_keys_from(a, q, t, i) : 0;
        for (int j = from + warp; j < min(q.kv, ctx + i + 1); j += kTreeWarps) {
            if (j >= ctx && !tree_sees(a, t, j - ctx)) continue;
            const int page = a.table[r * a.table_stride + (j >> a.page_shift)];
            if (page < 0 || page >= a.pages) continue;
            const int64_t at = page * a.page_stride + (h / a.group) * a.head_stride +
                               (j & ((1 << a.page_shift) - 1)) * a.slot_stride + lane;
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = __fmaf_rn(x[e], load16<BF16>(a.k_pages, at + 32 * e), s);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            s *= a.scale;
            const float m_new = fmaxf(m, s), f = m == -INFINITY ? 0.0f : expf(m - m_new), p = expf(s - m_new);
            l = l * f + p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * load16<BF16>(a.v_pages, at + 32 * e);
            m = m_new;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        __syncthreads();
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < kTreeWarps; ++w) top = fmaxf(top, s_m[w]);
        for (int w = 0; w < kTreeWarps; ++w) sum += s_m[w] == -INFINITY ? 0.0f : s_l[w] * expf(s_m[w] - top);
        for (int d = threadIdx.x; d < D; d += kTreeWarps * 32) {
            float y = 0.0f;
            for (int w = 0; w < kTreeWarps; ++w) y += s_m[w] == -INFINITY ? 0.0f : s_o[w][d] * expf(s_m[w] - top);
            y = sum > 0.0f ? y / sum : 0.0f;
            const int64_t at = t * a.out_token_stride + h * a.out_head_stride + d;
            if constexpr (BF16)
                static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16(y);
            else
                static_cast<__half*>(a.out)[at] = __float2half(y);
        }
        if (threadIdx.x == 0 && a.lse) a.lse[int64_t(t) * a.q_heads + h] = sum > 0.0f ? top + logf(sum) : -INFINITY;
        __syncthreads();
    }
}

template <bool BF16>
int launch_tree(const AttnArgs& a) {
    const dim3 grid(a.requests, a.q_heads);
    if (a.head_dim == 64)
        attention_tree_kernel<64, BF16><<<grid, kTreeWarps * 32, 0, a.stream>>>(a);
    else if (a.head_dim == 96)
        attention_tree_kernel<96, BF16><<<grid, kTreeWarps * 32, 0, a.stream>>>(a);
    else
        attention_tree_kernel<128, BF16><<<grid, kTreeWarps * 32, 0, a.stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace

int launch_attention_tree(const AttnArgs& a) { return a.bf16 ? launch_tree<true>(a) : launch_tree<false>(a); }

}  // namespace nq
