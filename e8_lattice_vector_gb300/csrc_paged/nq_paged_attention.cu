// nq_paged_attention.cu -- attention of a step's new tokens over the paged cache: argument checks, the choice of
// the kernel, and the second launch that joins row tiles whose keys were read by several blocks.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "nq_paged_device.cuh"

namespace nq {
namespace {

constexpr int kJoinWarps = 8;

// A row's pieces: block b's slot 1, then slot 0 of the blocks after it.
__device__ __forceinline__ int piece_slot(int b, int i) { return i == 0 ? 2 * b + 1 : 2 * (b + i); }

template <bool BF16>
__device__ __forceinline__ void join_store(const AttnArgs& a, const AttnSplit& s, int row, int lane, float4 acc, float top,
                                           float sum, bool lse) {
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const int token = a.by_group.of(s.row0 + row), t = s.begin + token;
    const int h = s.head * a.group + s.row0 + row - token * a.group;
    uint2 packed;
    packed.x = pack2<BF16>(acc.x * inv, acc.y * inv);
    packed.y = pack2<BF16>(acc.z * inv, acc.w * inv);
    if (4 * lane < a.head_dim)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + t * a.out_token_stride + h * a.out_head_stride + 4 * lane) =
            packed;
    if (lse && a.lse != nullptr)
        a.lse[int64_t(t) * a.q_heads + h] = sum > 0.0f ? top * a.scale + logf(sum) : -INFINITY;
}

// Few rows with many pieces (up to one from every block): block (b, y) takes row y of the row tile that block b of the
// attention kernel began and did not end.  Each warp takes every eighth piece, and the sums meet in shared memory, in an
// order that depends on the lengths alone.
template <bool BF16>
__global__ void __launch_bounds__(kJoinWarps * 32) join_few_rows_kernel(const AttnArgs a, const AttnWorkspace ws) {
    __shared__ float4 part[kJoinWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x, row = blockIdx.y;
    pdl_wait();
    const AttnSplit s = ws.split[b];
    if (s.last_block < 0 || row >= s.n_rows) return;
    const int pieces = s.last_block - b + 1, D = a.head_dim;
    const float sc = a.scale * kLog2e;
    auto at = [&](int i) { return int64_t(piece_slot(b, i)) * kSmallRows + row; };
    // a lane for each piece, 32 at a time; the first 32 are kept
    const float2 none = make_float2(-INFINITY, 0.0f), ml = lane < pieces ? ws.ml[at(lane)] : none;
    float top = ml.x;
    for (int i = lane + 32; i < pieces; i += 32) top = fmaxf(top, ws.ml[at(i)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < pieces; i0 += 32) {
        const float2 x = i0 == 0 ? ml : i0 + lane < pieces ? ws.ml[at(i0 + lane)] : none;
        const float f = x.x == -INFINITY ? 0.0f : exp2_fast((x.x - top) * sc);
        sum += x.y * f;
        const int n = min(pieces - i0, 32);
#pragma unroll 4
        for (int i = warp; i < n; i += kJoinWarps) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            if (4 * lane < D) {
                const float4 o = *reinterpret_cast<const float4*>(ws.o + at(i0 + i) * D + 4 * lane);
                acc.x = fmaf(o.x, fi, acc.x);
                acc.y = fmaf(o.y, fi, acc.y);
                acc.z = fmaf(o.z, fi, acc.z);
                acc.w = fmaf(o.w, fi, acc.w);
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    part[warp][lane] = acc;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int v = 1; v < kJoinWarps; ++v) {
        const float4 o = part[v][lane];
        acc.x += o.x;
        acc.y += o.y;
        acc.z += o.z;
        acc.w += o.w;
    }
    join_store<BF16>(a, s, row, lane, acc, top, sum, lane == 0);
}

// Many rows with few pieces: a warp for a row.  (Two or four rows a warp, their loads in flight together, were 2 us faster for 152
// row tiles of two pieces each and 3 to 6 us slower for 16 row tiles of ten.)  152 row tiles of 256 rows and two to three
// pieces take 14 us, 4.5 TB/s, nearly all of it out of the L2.
template <bool BF16>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_many_rows_kernel(const AttnArgs a, const AttnWorkspace ws, int half_rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
    pdl_wait();
    const AttnSplit s = ws.split[b];
    const int row = int(blockIdx.y) * kJoinWarps + warp;
    if (s.last_block < 0 || row >= s.n_rows) return;
    const int pieces = s.last_block - b + 1, D = a.head_dim;
    const float sc = a.scale * kLog2e;
    const int place = row >= half_rows ? 128 + row - half_rows : row;  // among the 256 of a slot: the halves begin at 0 and 128
    const float2 none = make_float2(-INFINITY, 0.0f);
    auto ml_at = [&](int i) { return i < pieces ? ws.ml[int64_t(piece_slot(b, i)) * kChunkRows + place] : none; };
    const float2 ml = ml_at(lane);
    float top = ml.x;
    for (int i = lane + 32; i < pieces; i += 32) top = fmaxf(top, ml_at(i).x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    // 8 columns of a half's 128 rows are stored together
    const float* o = ws.o + int64_t(place >> 7) * D * 128 + (lane >> 1) * 1024 + (place & 127) * 8 + 4 * (lane & 1);
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < pieces; i0 += 32) {
        const float2 x = i0 == 0 ? ml : ml_at(i0 + lane);
        const float f = x.x == -INFINITY ? 0.0f : exp2_fast((x.x - top) * sc);
        sum += x.y * f;
        const int n = min(pieces - i0, 32);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            if (4 * lane >= D) continue;
            const float4 y = *reinterpret_cast<const float4*>(o + int64_t(piece_slot(b, i0 + i)) * kChunkRows * D);
            acc.x = fmaf(y.x, fi, acc.x);
            acc.y = fmaf(y.y, fi, acc.y);
            acc.z = fmaf(y.z, fi, acc.z);
            acc.w = fmaf(y.w, fi, acc.w);
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    join_store<BF16>(a, s, row, lane, acc, top, sum, lane == 0);
}

int check_attention(const nq_attention* a, const nq_pool* pool) {
    const int st = check_pool(pool);
    if (st != NQ_OK) return st;
    if (!a) return NQ_ERR_ARG;
    if (a->tokens < 0 || a->requests < 0 || a->table_cols < 0 || a->max_q < 0 || a->window < 0) return NQ_ERR_ARG;
    if (a->causal != 0 && a->causal != 1) return NQ_ERR_ARG;
    if (a->q_heads < 1 || a->q_heads % pool->kv_heads != 0) return NQ_ERR_ARG;
    if (!(a->scale > 0.0f) || !std::isfinite(a->scale)) return NQ_ERR_ARG;
    // positions and tile ends stay within 32 bits
    if (int64_t(a->table_cols) * pool->page_size > INT_MAX - 65536) return NQ_ERR_ARG;
    if (int64_t(a->tokens) * a->q_heads > INT_MAX - 65536) return NQ_ERR_ARG;
    if (a->requests > 1 && a->table_stride < a->table_cols) return NQ_ERR_ARG;
    const int dim = pool->head_dim;
    if (!paged_stride_ok(a->q_token_stride, a->tokens, dim) || !paged_stride_ok(a->q_head_stride, a->q_heads, dim) ||
        !paged_stride_ok(a->out_token_stride, a->tokens, dim) || !paged_stride_ok(a->out_head_stride, a->q_heads, dim))
        return NQ_ERR_ARG;
    return NQ_OK;
}

// Whether most requests have far fewer rows than the longest: then the small kernel takes those that fit its tile and the
// large kernel the others.  The large kernel alone spends tiles of 128 rows on single tokens.  What both take, over what the large
// one alone takes (32 heads on 8): 512 tokens beside 31 single tokens over 8000 cached 0.66 to 0.97 (head_dim 64 and 128, fp16 and
// bf16; 252 against 301 us at 128 in bf16), over 2000 cached 0.83 to 1.14, 128 tokens beside 7 over 2000 1.08 to 1.30, and where the
// small kernel finds nothing to do 1.05 to 1.11 (its two launches: 4 to 5 us).  The contexts, which decide, are not known here; a
// long one gains more than a short one loses.
bool may_mix(const nq_attention* a, int group) {
    return group <= kSmallRows && 4 * int64_t(a->tokens) < int64_t(a->requests) * a->max_q;
}

// The small kernel's calls: a request's rows for one KV head fit its tile, or some need a second one and most do not, or a
// token's rows do not fit a half of the large kernel's row tile.  "Most do not": rows of three quarters of a tile on average, when
// rows are short enough that reading keys twice costs less than the large kernel's tiles of 128 rows, else calls that would be mixed.
// Drafts of 1 to 8 tokens for 32 requests over 2000 and 8000 cached and windows of 4096 (32 heads on 8, fp16 and bf16; what
// the small kernel takes, over the large one or the mixed call): head_dim 64 0.64 to 1.05, 96 0.76 to 1.09, 128 0.78 to 1.01 where the
// call would be mixed, and 0.98 to 1.18 where not.
bool few_rows(const nq_attention* a, int group, int head_dim) {
    const int64_t longest = int64_t(std::min(a->max_q, a->tokens)) * group;
    if (longest <= kSmallRows || group > 128) return true;
    if (longest > 2 * kSmallRows) return false;
    return may_mix(a, group) ||
           (head_dim <= 96 && 4 * int64_t(a->tokens) * group <= 3 * kSmallRows * int64_t(a->requests));
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return encode;
}

bool make_pool_map(const AttnArgs& a, const void* base, CUtensorMap* map) {
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    const int page_size = 1 << a.page_shift;
    const cuuint64_t dims[4] = {cuuint64_t(a.head_dim), cuuint64_t(page_size), cuuint64_t(a.kv_heads), cuuint64_t(a.pages)};
    // the stride of a single head or page is never used, but has to be a valid one
    const cuuint64_t strides[3] = {cuuint64_t(a.slot_stride) * 2,
                                   cuuint64_t(a.kv_heads > 1 ? a.head_stride : a.slot_stride) * 2,
                                   cuuint64_t(a.pages > 1 ? a.page_stride : a.slot_stride) * 2};
    const cuuint32_t box[4] = {64, cuuint32_t(std::min(page_size, kKeyTile)), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode(map, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_pool_maps(const AttnArgs& a, CUtensorMap* k, CUtensorMap* v) {
    return make_pool_map(a, a.k_pages, k) && make_pool_map(a, a.v_pages, v);
}

bool make_query_map(const AttnArgs& a, CUtensorMap* q) {
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {cuuint64_t(a.head_dim), cuuint64_t(a.q_heads), cuuint64_t(a.tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(a.q_heads > 1 ? a.q_head_stride : a.head_dim) * 2,
                                   cuuint64_t(a.tokens > 1 ? a.q_token_stride : a.head_dim) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(a.group), cuuint32_t(a.half_tokens)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(q, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(a.q),
                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {
cudaLaunchConfig_t join_config(const AttnArgs& a, int rows, int rows_per_block, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    rows = int(std::min<int64_t>(int64_t(a.tokens) * a.group, rows));
    cfg.gridDim = dim3(kAttnGrid, unsigned((rows + rows_per_block - 1) / rows_per_block));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}
}  // namespace

int launch_join_few_rows(const AttnArgs& a, const AttnWorkspace& ws) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = join_config(a, kSmallRows, 1, &attr);
    const cudaError_t e = a.bf16 ? cudaLaunchKernelEx(&cfg, join_few_rows_kernel<true>, a, ws)
                                 : cudaLaunchKernelEx(&cfg, join_few_rows_kernel<false>, a, ws);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

int launch_join_many_rows(const AttnArgs& a, const AttnWorkspace& ws) {
    cudaLaunchAttribute attr;
    const int half_rows = a.half_tokens * a.group;
    const cudaLaunchConfig_t cfg = join_config(a, 2 * half_rows, kJoinWarps, &attr);
    const cudaError_t e = a.bf16 ? cudaLaunchKernelEx(&cfg, join_many_rows_kernel<true>, a, ws, half_rows)
                                 : cudaLaunchKernelEx(&cfg, join_many_rows_kernel<false>, a, ws, half_rows);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace nq

extern "C" {

int nq_paged_attention_workspace(const nq_attention* a, const nq_pool* pool, uint64_t* bytes) {
    const int st = nq::check_attention(a, pool);
    if (st != NQ_OK) return st;
    if (!bytes) return NQ_ERR_ARG;
    const int group = a->q_heads / pool->kv_heads;
    // the large kernel's calls may be mixed; their size is the larger one in any case
    *bytes = nq::attn_workspace(nullptr, nq::kSmallRows, pool->head_dim).total;
    if (!nq::few_rows(a, group, pool->head_dim)) *bytes += nq::chunk_workspace(a->tokens, group, a->requests, pool->head_dim);
    return NQ_OK;
}

int nq_paged_status(void* stream) {
    static nq::GiveUps reported;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint64_t small = 0, chunk = 0;
    int device = 0;
    const bool read = nq::read_small_gave_up(&small, s) == NQ_OK && nq::read_chunk_gave_up(&chunk, s) == NQ_OK;
    if (cudaStreamSynchronize(s) != cudaSuccess || !read || cudaGetDevice(&device) != cudaSuccess) return NQ_ERR_CUDA;
    return reported.grew(device, small, chunk) ? NQ_ERR_CUDA : NQ_OK;
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
    x.out_by_32 = nq::paged_aligned(out, 32) && (a->tokens == 1 || a->out_token_stride % 16 == 0) &&
                  (a->q_heads == 1 || a->out_head_stride % 16 == 0);
    x.by_group = nq::FastDiv::by(uint32_t(x.group));
    x.half_tokens = 128 / x.group;
    x.mixed = 0;
    x.scale = a->scale;
    x.stream = static_cast<cudaStream_t>(stream);
    if (nq::few_rows(a, x.group, x.head_dim)) return nq::launch_attention_small(x);
    if (nq::may_mix(a, x.group)) {
        x.mixed = 1;
        const int small = nq::launch_attention_small(x);
        if (small != NQ_OK) return small;
    }
    return nq::launch_attention_chunk(x);
}

}  // extern "C"
