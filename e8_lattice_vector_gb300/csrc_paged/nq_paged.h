// nq_paged.h -- declarations shared by the paged-cache translation units.
#pragma once

#include <cuda.h>  // CUtensorMap (type only; the encoder is fetched at run time)
#include <cuda_runtime.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <utility>

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
    if (p->pages < 1 || p->kv_heads < 1 || p->kv_heads > 65536) return NQ_ERR_ARG;
    if (!paged_stride_ok(p->page_stride, p->pages, p->head_dim) ||
        !paged_stride_ok(p->head_stride, p->kv_heads, p->head_dim) ||
        !paged_stride_ok(p->slot_stride, p->page_size, p->head_dim))
        return NQ_ERR_ARG;
    return NQ_OK;
}

// Streaming multiprocessors of the current device, 0 when it cannot be queried.
int paged_sm_count();

// Division of n < 2^31 by a number fixed for the call: n / d = (umulhi(n, mul) + n) >> shift with 2^shift >= d and
// mul = floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery's division by invariant integers).
struct FastDiv {
    uint32_t mul, shift;
    static FastDiv by(uint32_t d) {
        FastDiv f;
        f.shift = 0;
        while ((uint64_t(1) << f.shift) < d) ++f.shift;
        f.mul = uint32_t((((uint64_t(1) << f.shift) - d) << 32) / d + 1);
        return f;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int of(int n) const { return int((__umulhi(uint32_t(n), mul) + uint32_t(n)) >> shift); }
#endif
};

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
    int mixed;      // both kernels are launched: the small one takes requests of at most kSmallRows rows, the large one others
    int out_by_32;  // rows of out start on 32-byte boundaries
    FastDiv by_group;
    int half_tokens;  // tokens whose rows fit one half of the large kernel's row tile (0: a group of more than 128 heads)
    float scale;
    cudaStream_t stream;
};

// Both kernels run one block per multiprocessor of a GB300, each with an equal share of the step's (row tile, key
// tile) pairs, in the order request, KV head, row tile, key tile.  A row tile whose keys end up in several
// blocks leaves partial results in the workspace: per block two slots (0: its first piece, which an earlier
// block began; 1: its last, which a later block ends), joined by a second launch.
constexpr int kAttnGrid = 152;

struct AttnSplit {  // per block: the row tile that it began and did not end, or last_block = -1
    int begin;         // row of q where the request's (small kernel) or the row tile's (large kernel) tokens begin
    int row0, n_rows;  // the row tile's rows, counted from there
    int head, last_block;
};

struct AttnWorkspace {
    AttnSplit* split;  // [kAttnGrid]
    float2* ml;        // [kAttnGrid * 2][rows]: running maximum (unscaled score), sum
    float* o;          // [kAttnGrid * 2][rows][head_dim]; the large kernel: [kAttnGrid * 4][head_dim / 8][128][8]
    uint64_t total;
};

// The arrays begin on the first 256-byte boundary at or after `base`: pieces are stored 32 bytes at a time, and a caller's
// scratch need only be 16-byte aligned.  `total` counts from `base` and has room for the bytes that are skipped.
constexpr uintptr_t kWorkspaceAlign = 256;

inline AttnWorkspace attn_workspace(void* base, int rows, int head_dim) {
    char* p = static_cast<char*>(base);
    p += (kWorkspaceAlign - reinterpret_cast<uintptr_t>(p) % kWorkspaceAlign) % kWorkspaceAlign;
    AttnWorkspace w;
    uint64_t off = 0;
    w.split = reinterpret_cast<AttnSplit*>(p);
    off += (kAttnGrid * sizeof(AttnSplit) + 255) / 256 * 256;
    w.ml = reinterpret_cast<float2*>(p + off);
    off += (uint64_t(kAttnGrid) * 2 * rows * sizeof(float2) + 255) / 256 * 256;
    w.o = reinterpret_cast<float*>(p + off);
    off += uint64_t(kAttnGrid) * 2 * rows * head_dim * sizeof(float);
    w.total = off + kWorkspaceAlign - 16;
    return w;
}

// Rows of q (times the heads that share a KV head) per tile of the small kernel.
constexpr int kSmallRows = 16;
// ... and of the large one: two halves of 128, each filled with the rows of whole tokens.
constexpr int kChunkRows = 256;

// TMA maps of the two pools: boxes of 64 columns x min(page_size, 128) slots, 128-byte swizzle.  false on failure.
bool make_pool_maps(const AttnArgs& a, CUtensorMap* k, CUtensorMap* v);
// TMA map of q: boxes of 64 columns x a group's heads x a half's tokens, 128-byte swizzle.
bool make_query_map(const AttnArgs& a, CUtensorMap* q);

int launch_attention_small(const AttnArgs& a);
int launch_attention_chunk(const AttnArgs& a);
uint64_t chunk_workspace(int64_t tokens, int group, int requests, int head_dim);
// Join the pieces of split row tiles, launched after the small or the large kernel as its dependent.
int launch_join_few_rows(const AttnArgs& a, const AttnWorkspace& ws);
int launch_join_many_rows(const AttnArgs& a, const AttnWorkspace& ws);

// Copies of the counts of blocks that gave up a wait, in stream order.
int read_small_gave_up(uint64_t* blocks, cudaStream_t stream);
int read_chunk_gave_up(uint64_t* blocks, cudaStream_t stream);

// What has been reported of these counts, per device.  The counts on the device only grow, so that one that grows while it is
// read, by a kernel on another stream, is reported by the next call.
class GiveUps {
public:
    // Whether either count is past what has been reported; it is reported then.  A copy older than another thread's says nothing.
    bool grew(int device, uint64_t small, uint64_t chunk) {
        std::lock_guard<std::mutex> lock(mu_);
        auto& seen = seen_[device];
        const bool s = small > seen.first, c = chunk > seen.second;
        if (s) seen.first = small;
        if (c) seen.second = chunk;
        return s || c;
    }

private:
    std::mutex mu_;
    std::map<int, std::pair<uint64_t, uint64_t>> seen_;
};

// Allow `kernel` `smem` bytes of dynamic shared memory on the current device (once per device); false on a CUDA error.
bool ensure_smem(const void* kernel, int smem);

}  // namespace nq
