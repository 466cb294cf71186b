// nq_verify_drafts.cu -- drafted tokens against the model's probabilities, from given random numbers.
//
// Simplest form: a block for a request.  Its first thread walks the tree; sums over the vocabulary are formed by the block in 64 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nq_paged.h"

namespace nq {
namespace {

constexpr int kVerifyThreads = 512;

struct VerifyArgs {
    const void *probs, *draft_probs;
    int64_t probs_stride, draft_stride;
    const int32_t *drafts, *parents, *q_start;
    const float* uniform;
    int32_t *accepted, *path, *tokens_out;
    int vocab, tokens;
};

__device__ __forceinline__ float weight_of(float x) { return x > 0.0f ? x : 0.0f; }  // NaN counts as 0
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_drafts_kernel(const VerifyArgs a) {
    __shared__ double s_sum[kVerifyThreads];
    __shared__ int s_cur, s_next;
    __shared__ double s_taken, s_total;
    const int r = blockIdx.x, V = a.vocab;
    const int begin = min(max(a.q_start[r], 0), a.tokens), n = max(min(max(a.q_start[r + 1], 0), a.tokens) - begin, 0);
    if (n == 0) {
        if (threadIdx.x == 0) a.accepted[r] = 0;
        return;
    }
    const bool sampled = a.draft_probs != nullptr;
    auto p_at = [&](int node, int x) {
        return double(weight_of(to_float(static_cast<const T*>(a.probs)[(begin + node) * a.probs_stride + x])));
    };
    auto q_at = [&](int node, int x) {
        return double(weight_of(to_float(static_cast<const T*>(a.draft_probs)[(begin + node) * a.draft_stride + x])));
    };
    // an earlier child of the same node, rejected, that was this token
    auto rejected = [&](int cur, int x, int upto) {
        for (int i = cur + 1; i < upto; ++i)
            if (a.parents[begin + i] == cur && a.drafts[begin + i] == x) return true;
        return false;
    };
    // what is left of the current node's probabilities
    auto left = [&](int cur, double taken, int x) {
        if (sampled) return max(p_at(cur, x) - taken * (taken > 0.0 ? q_at(cur, x) : 0.0), 0.0);
        return taken < 0.0 || !rejected(cur, x, n) ? p_at(cur, x) : 0.0;
    };
    const int each = (V + kVerifyThreads - 1) / kVerifyThreads;
    const int v0 = min(int(threadIdx.x) * each, V), v1 = min(v0 + each, V);
    auto sum = [&](int cur, double taken) {
        double x = 0.0;
        for (int v = v0; v < v1; ++v) x += left(cur, taken, v);
        s_sum[threadIdx.x] = x;
        __syncthreads();
        double total = 0.0;
        if (threadIdx.x == 0) {
            for (int t = 0; t < kVerifyThreads; ++t) total += s_sum[t];
            s_total = total;
        }
        __syncthreads();
    };
    if (threadIdx.x == 0) {
        s_cur = 0;
        s_next = 1;
        s_taken = 0.0;
        s_total = 1.0;
        a.path[begin] = 0;
    }
    __syncthreads();
    int kept = 1;  // the first thread's
    while (true) {
        // the first thread walks up to the first rejected draft whose leftovers have to be summed
        if (threadIdx.x == 0) {
            int i = s_next, cur = s_cur;
            double taken = s_taken, total = s_total;
            for (; i < n; ++i) {
                if (a.parents[begin + i] != cur) continue;
                const int x = a.drafts[begin + i];
                if (x < 0 || x >= V) continue;  // no draft
                const double u = a.uniform[begin + i], q = sampled ? q_at(cur, x) : 1.0;
                const double w = sampled ? max(p_at(cur, x) - taken * q, 0.0) : rejected(cur, x, i) ? 0.0 : p_at(cur, x);
                if (u * (total * q) < w) {
                    a.tokens_out[begin + kept - 1] = x;
                    a.path[begin + kept++] = i;
                    cur = i;
                    taken = 0.0;
                    total = 1.0;
                } else if (sampled) {
                    taken += total;
                    ++i;
                    break;
                } else {
                    total -= w;
                }
            }
            s_cur = cur;
            s_next = i;
            s_taken = taken;
            s_total = total;
        }
        __syncthreads();
        const int next = s_next;
        __syncthreads();
        sum(s_cur, s_taken);
        if (next >= n) break;
    }
    const int cur = s_cur;
    double taken = s_taken;
    if (!(s_total > 0.0)) {
        taken = sampled ? 0.0 : -1.0;  // nothing is left: the node's own probabilities
        __syncthreads();
        sum(cur, taken);
    }
    if (threadIdx.x > 0) return;
    const double u = a.uniform[begin], target = u * s_total;
    int token = -1;
    double upto = 0.0;
    for (int t = 0; t < kVerifyThreads && token < 0; ++t) {
        if (upto + s_sum[t] > target) {
            double x = upto;
            for (int v = t * each; v < min((t + 1) * each, V); ++v) {
                x += left(cur, taken, v);
                if (x > target) {
                    token = v;
                    break;
                }
            }
        }
        upto += s_sum[t];
    }
    for (int v = V - 1; v >= 0 && token < 0; --v)
        if (left(cur, taken, v) > 0.0) token = v;
    a.accepted[r] = kept;
    a.tokens_out[begin + kept - 1] = token;
    for (int k = kept; k < n; ++k) a.path[begin + k] = a.tokens_out[begin + k] = -1;
}

}  // namespace
}  // namespace nq

extern "C" int nq_verify_drafts(const void* probs, int64_t probs_stride, const void* draft_probs, int64_t draft_stride,
                                int32_t dtype, int32_t vocab, const int32_t* drafts, const int32_t* parents,
                                const float* uniform, int32_t tokens, const int32_t* q_start, int32_t requests,
                                int32_t* accepted, int32_t* path, int32_t* tokens_out, void* stream) {
    if (dtype != NQ_F16 && dtype != NQ_BF16 && dtype != NQ_F32) return NQ_ERR_UNSUPPORTED;
    if (tokens < 0 || requests < 0 || vocab < 1 || vocab > INT32_MAX - 65536) return NQ_ERR_ARG;
    if (tokens > 1 && (probs_stride < vocab || (draft_probs && draft_stride < vocab))) return NQ_ERR_ARG;
    if (requests == 0) return NQ_OK;
    if (!q_start || !accepted) return NQ_ERR_ARG;
    if (tokens > 0 && (!probs || !drafts || !parents || !uniform || !path || !tokens_out)) return NQ_ERR_ARG;
    const uintptr_t size = dtype == NQ_F32 ? 4 : 2;
    if (!nq::paged_aligned(probs, size) || !nq::paged_aligned(draft_probs, size)) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(drafts), static_cast<const void*>(parents),
                          static_cast<const void*>(uniform), static_cast<const void*>(q_start),
                          static_cast<const void*>(accepted), static_cast<const void*>(path),
                          static_cast<const void*>(tokens_out)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    nq::VerifyArgs a{probs, draft_probs, probs_stride, draft_stride, drafts, parents, q_start, uniform, accepted, path, tokens_out,
                     vocab, tokens};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == NQ_F32)
        nq::verify_drafts_kernel<float><<<requests, nq::kVerifyThreads, 0, s>>>(a);
    else if (dtype == NQ_F16)
        nq::verify_drafts_kernel<__half><<<requests, nq::kVerifyThreads, 0, s>>>(a);
    else
        nq::verify_drafts_kernel<__nv_bfloat16><<<requests, nq::kVerifyThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
