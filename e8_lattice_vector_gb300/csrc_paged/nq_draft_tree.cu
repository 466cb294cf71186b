// nq_draft_tree.cu -- the map of a step's drafted trees: which drafted tokens each one sees, and its position.
//
// A node's parent stands before it, so its way to the root is a walk of decreasing indices: the bits of a 64-bit word are complete
// when the walk leaves it, and a node needs no more than one word in registers, whatever the tree's size.  A block takes a
// request and reads its parents once, into shared memory, where a level of the walk takes 30 cycles.
// Measured (graph replays): one tree of 8 2.0 to 2.3 us, 256 trees of up to 64 2.5 to 2.8 us: the launch, and two dependent loads.  A node walks
// all its depth, so long chains are slow: one of 256 41 us, of 1024 0.30 ms, of 4096 4.0 ms (calls timed by events), where a star or a
// tree of 4096 whose nodes have three children takes 0.15 ms.
#include "nq_paged.h"

#include <algorithm>

namespace nq {
namespace {

constexpr int kTreeNodes = 2048;  // parents in shared memory; those of a larger request are read where they are

__global__ void draft_tree_kernel(const int32_t* __restrict__ parents, int tokens, const int32_t* __restrict__ q_start,
                                  const int32_t* __restrict__ kv_lens, int window, int words, unsigned long long* ancestors,
                                  int32_t* positions) {
    __shared__ int s_parent[kTreeNodes];
    const int r = blockIdx.x;
    const int begin = min(max(q_start[r], 0), tokens), n = min(max(q_start[r + 1], 0), tokens) - begin;
    const int ctx = max(kv_lens[r], 0) - n;
    const bool shared = n <= kTreeNodes;
    if (shared)
        for (int i = threadIdx.x; i < n; i += blockDim.x) s_parent[i] = parents[begin + i];
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        unsigned long long* row = ancestors + int64_t(begin + i) * words;
        unsigned long long bits = 0;
        int depth = -1, word = i >> 6;
        for (int w = word + 1; w < words; ++w) row[w] = 0;
        for (int j = i; j >= 0;) {
            if (j >> 6 != word) {
                if (word < words) row[word] = bits;
                for (int w = min(word, words) - 1; w > j >> 6; --w) row[w] = 0;
                word = j >> 6;
                bits = 0;
            }
            if (window == 0 || depth + 1 < window) bits |= 1ull << (j & 63);
            ++depth;
            const int up = shared ? s_parent[j] : __ldg(parents + begin + j);
            j = up < j ? max(up, -1) : -1;
        }
        if (word < words) row[word] = bits;
        for (int w = min(word, words) - 1; w >= 0; --w) row[w] = 0;
        positions[begin + i] = ctx + depth;
    }
}

}  // namespace
}  // namespace nq

extern "C" int nq_draft_tree(const int32_t* parents, int32_t tokens, const int32_t* q_start, const int32_t* kv_lens,
                             int32_t requests, int32_t window, int32_t words, int64_t* ancestors, int32_t* positions,
                             void* stream) {
    if (tokens < 0 || requests < 0 || window < 0 || words < 1 || words > NQ_TREE_WORDS) return NQ_ERR_ARG;
    if (tokens == 0 || requests == 0) return NQ_OK;
    if (!parents || !q_start || !kv_lens || !ancestors || !positions) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(q_start),
                          static_cast<const void*>(kv_lens), static_cast<const void*>(positions)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    if (!nq::paged_aligned(ancestors, 8)) return NQ_ERR_ARG;
    nq::draft_tree_kernel<<<requests, std::min(64 * words, 256), 0, static_cast<cudaStream_t>(stream)>>>(
        parents, tokens, q_start, kv_lens, window, words, reinterpret_cast<unsigned long long*>(ancestors), positions);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}
