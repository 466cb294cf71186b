// nq_paged_chunk.cu -- attention of many rows per request over the paged cache (prompt chunks, whole prompts).
//
// Rows are tokens times the `group` query heads that share a KV head.  A half is as many whole tokens as fit 128 rows, a row
// tile two halves.  For each tile of 128 keys and each half, on the tensor cores (tcgen05, accumulators in tensor memory):
//   S = Q K^T                    128 x 128, fp32
//   P = exp2((S - m) c)          by a warpgroup, a thread per row: no exchange between threads
//   O = O f + P V                P from tensor memory, where it takes the place of S
// m is a reference that follows the running maximum only when that has grown by more than 2^8 in P (kSlack): O is
// rescaled on those few tiles, and on the others the tensor cores add to it undisturbed.  P stays below 2^8 (times 2^7 in
// fp16, see kLift), and its sum below 2^46 for any length.
//
// The two halves alternate on the tensor cores: while one half's exponentials are taken, the other half's products run.  A
// row tile with rows for one half only is given to both, each taking every other key tile; the two sums meet
// in tensor memory.  One warp loads K and V (TMA, one box per page and 64 columns), one loads Q, one issues the products.
//
// Shares: the row tiles' key tiles, in order, in equal parts over 152 blocks; a launch of one block finds where each part
// begins.  Row tiles that end up in several blocks are joined by a second launch.
//
// Measured (32 query heads on 8 KV heads, head_dim 128, 2000 tokens over 30000 cached, median of graph replays): fp16 706 us, 1438
// TFLOP/s, 77% of the measured cuBLAS rate (the best replay 664; 736 to 768 in long streams of calls, under the power cap); bf16
// 972 us, 1045 TFLOP/s (the best 922).  What bounds it is the chain of one half: its exponentials (about 1200 of 3000
// cycles a tile), its two products (1024, 1536 in bf16) and the hand-overs between them, with the tensor cores busy 68% (bf16: 73%)
// of the time under the profiler.  Taking the exponentials before the maximum is known, or starting the second product with
// half of P, shortened the chain and took as long or longer.
//
// In bf16 P is the sum of two bf16 (hi + lo), each with its own product: one bf16 has 2^-8 of p as its rounding error, as much as
// the output's own, and fp16 tensors, whose P has 2^-11, show that the second product costs 38% of the time.  It is the
// price of an output that is off by its own rounding and nothing else.
#include "nq_paged_walk.cuh"

namespace nq {
namespace {

__device__ unsigned long long g_gave_up;  // blocks that gave up a wait, ever

constexpr int kThreadsChunk = 384;  // two warpgroups for the halves; loads, products, clearing, pieces and Q
constexpr int kPlanThreads = 1024;
constexpr float kSlack = 8.0f;  // in powers of two
constexpr float kExactRef = 1048576.0f;  // references up to 2^20: off by 2^-5 from m sc at most

template <int D>
struct Chunk {
    static constexpr int HALVES = D > 64 ? 2 : 1;  // 64-column halves of a tile
    static constexpr int TILE = HALVES * kHalfBytes;
    static constexpr int Q = 2 * TILE;
    static constexpr int STAGES = (224 * 1024 - Q) / TILE;  // 5, or 12 of half the size
    static constexpr int SMEM = 1024 + Q + STAGES * TILE;
};
constexpr int kLiveRing = 8;  // tiles whose page masks are kept; the loads are at most six tiles ahead of a half

// Block-wide inclusive sum; *total the sum over all threads.
__device__ __forceinline__ long long plan_scan(long long x, long long* total) {
    __shared__ long long warps[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += v;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    long long t = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += v;
    }
    *total = __shfl_sync(0xffffffffu, t, 31);
    const long long before = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
    return x + (warp > 0 ? before : 0);
}

// The largest of the values (none negative) of the threads before; *total over all threads.
__device__ __forceinline__ int plan_top(int x, int* total) {
    __shared__ int warps[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) x = max(x, __shfl_up_sync(0xffffffffu, x, d));  // lanes below d get their own
    int before = __shfl_up_sync(0xffffffffu, x, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    const int w = warps[lane];
    *total = __reduce_max_sync(0xffffffffu, w);
    return max(before, __reduce_max_sync(0xffffffffu, lane < warp ? w : 0));
}

// One block: the requests' rows, the running sum of key tiles over the (request, row tile) pairs, then the beginning of every
// share.  `room`: pairs that the arrays hold, all there are.
//
// The order is request, KV head, row tile: the row tiles that read the same keys come one after the other, in a block and in
// its neighbours, and find them in the L2 (with row tiles outside heads 2000 tokens over 30000 cached took 2% longer).
__global__ void __launch_bounds__(kPlanThreads) attention_plan_kernel(const AttnArgs a, const ChunkPlan plan, long long room) {
    __shared__ int s_pair[kPlanThreads];
    pdl_trigger();
    long long pairs = 0, tiles = 0;
    int top = 0;
    for (int r0 = 0; r0 < a.requests; r0 += kPlanThreads) {
        const int r = r0 + threadIdx.x;
        Request q{0, 0, 0};
        if (r < a.requests) q = load_request(a, r);
        int chunk_top;
        const RowRange rows = row_range(a, q, max(plan_top(rows_end(q), &chunk_top), top));
        top = max(top, chunk_top);
        if (r < a.requests) plan.rows[r] = rows;
        const int n = row_tiles_of(a, Request{rows.begin, rows.n, 0});
        long long chunk_pairs, chunk_tiles;
        const int upto = int(plan_scan(n, &chunk_pairs));
        __syncthreads();  // s_pair of the previous chunk is read
        s_pair[threadIdx.x] = upto - n;
        __syncthreads();
        chunk_pairs = min(chunk_pairs, room - pairs);
        for (int p0 = 0; p0 < int(chunk_pairs); p0 += kPlanThreads) {
            const int p = p0 + threadIdx.x;
            long long mine = 0;
            if (p < int(chunk_pairs)) {
                int lo = 0, hi = kPlanThreads;  // the last request whose first pair is at or before p
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_pair[mid] <= p)
                        lo = mid;
                    else
                        hi = mid;
                }
                const int row_tile = p - s_pair[lo];
                mine = row_tile_of(a, planned_request(a, plan, r0 + lo), row_tile).count;
                plan.pair_request[pairs + p] = r0 + lo;
                plan.pair_row_tile[pairs + p] = row_tile;
            }
            const long long sum = plan_scan(mine, &chunk_tiles);
            if (p < int(chunk_pairs)) plan.unit_sum[pairs + p] = tiles + sum - mine;
            tiles += chunk_tiles;
        }
        pairs += chunk_pairs;
    }
    const int cost = tiles * a.kv_heads >= (long long)kCostFrom * kAttnGrid ? kRowTileCost : 0;
    __syncthreads();  // the tiles' sums are written; the cost joins them
    for (long long p = threadIdx.x; p < pairs; p += kPlanThreads) plan.unit_sum[p] += cost * p;
    if (threadIdx.x == 0) plan.unit_sum[pairs] = tiles + cost * pairs;
    __syncthreads();
    const int b = threadIdx.x;
    if (b < kAttnGrid) plan.start[b] = chunk_start(a, plan, pairs, (tiles + cost * pairs) * a.kv_heads, cost, b);
}

// ------------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// A place in the ring and the parity of its use.
template <int STAGES>
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step() {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void back() {
        if (--stage < 0) {
            stage = STAGES - 1;
            phase ^= 1;
        }
    }
};

// Box [tokens of a half][heads of a group][64 columns] of q -> swizzled shared memory.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int head, int token) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(head), "r"(token)
        : "memory");
}

// Shared-memory operands, 128-byte swizzle: the low word holds the address and the leading offset, the high word the stride
// between groups of eight rows (1024 bytes), the version and the swizzle; both in 16-byte units.
constexpr uint32_t kDescHigh = 64u | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t tc_desc(uint32_t addr, uint32_t lead) { return (addr & 0x3ffffu) >> 4 | lead << 16; }
// Instruction descriptor: fp32 accumulator, both operands bf16 or fp16, 128 x N; B with N innermost when `b_n_major`.
template <bool BF16>
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_n_major) {
    return 1u << 4 | (BF16 ? 1u : 0u) << 7 | (BF16 ? 1u : 0u) << 10 | (b_n_major ? 1u : 0u) << 16 | uint32_t(n >> 3) << 17 |
           uint32_t(128 >> 4) << 24;
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(uint32_t(add)), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(uint32_t(add)), "n"(kDescHigh)
        : "memory");
}

// 32 columns of this thread's row.
__device__ __forceinline__ void tm_load(float* r, uint32_t addr) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr));
}
// Ends the loads into r[0, N): nothing that uses them comes before the wait.
template <int N>
__device__ __forceinline__ void tm_wait(float* r) {
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
// 16 columns: with 128 scores held there is no room for more at a time.
__device__ __forceinline__ void tm_load16(float* r, uint32_t addr) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr));
}
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t* u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
          "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
        : "memory");
}

// The reference is taken as fp32's nearest to LIFT - m sc; this is m sc + that number - LIFT, to the last bits of m sc (the sum's
// rounding error by Knuth's two-sum).
template <bool BF16>
__device__ __forceinline__ float beyond_reference(float m, float sc) {
    const float scaled = m * sc;
    if (fabsf(scaled) > kExactRef) return 0.0f;
    const float rest = __fmaf_rn(m, sc, -scaled);
    if constexpr (BF16) return rest;
    constexpr float lift = kLift<BF16, 7>;
    const float neg = lift - scaled, b = neg - lift;
    return rest - ((lift - (neg - b)) + (-scaled - b));
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void* dst, const uint32_t* u) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
// The lowest n bits, n of any sign and size.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

// Pairs of fp32 in one operation.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// -------------------------------------------------------------------- kernel

constexpr int kPieceRing = 4;

// One piece of a block's share: key tiles [key0 / 128, + take) of one row tile and KV head.
struct __align__(16) Piece {
    int take;           // 0: no more pieces
    int count[2];       // tiles of each half: every other one when shared; else those up to the half's last key
    int shared;         // one half's tokens, for both halves
    int row, n, pos;    // first token's row in q, tokens, position of the first
    int kv, key0, lo, hi;
    int head, request;
    int slot;           // workspace slot for the results, -1: the piece is the whole row tile
    int pad[2];
};

struct ChunkControl {
    // Places of the ring, by use; a tile's barriers, by tile: each is waited for in turn by one role, so that a wait is never
    // two phases from the barrier's own, whatever order the loads end in.
    uint64_t empty[12];
    uint64_t k_full[kLiveRing], v_full[kLiveRing], clean[kLiveRing];  // clean: V has no values that no row sees
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_full[2], drained;
    uint64_t piece_full[kPieceRing], piece_free[kPieceRing];
    uint64_t merge_full, merge_free;
    Piece piece[kPieceRing];
    uint32_t live[kLiveRing];  // per key tile: which of its pages are loaded
    uint32_t tmem;
    int gave_up;
    float m[128], l[128];  // a shared row tile's second half, for the first
};
constexpr int kPieceReaders = 11;  // eight softmax warps, loads, products, clearing

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreadsChunk, 1)
    attention_chunk_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                           const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map,
                           const AttnWorkspace ws, const ChunkPlan plan) {
    using C = Chunk<D>;
    constexpr int HALVES = C::HALVES, STAGES = C::STAGES;
    extern __shared__ char smem_raw[];
    __shared__ ChunkControl c;
    char* q_smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    char* ring = q_smem + C::Q;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_ptr(&c.empty[i]), 1);
        }
        for (int i = 0; i < kLiveRing; ++i) {
            mbar_init(smem_ptr(&c.k_full[i]), 1);
            mbar_init(smem_ptr(&c.v_full[i]), 1);
            mbar_init(smem_ptr(&c.clean[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_ptr(&c.q_full[i]), 1);
            mbar_init(smem_ptr(&c.q_free[i]), 1);
            mbar_init(smem_ptr(&c.s_full[i]), 1);
            mbar_init(smem_ptr(&c.p_full[i]), 4);
            mbar_init(smem_ptr(&c.o_full[i]), 1);
        }
        for (int i = 0; i < kPieceRing; ++i) {
            mbar_init(smem_ptr(&c.piece_full[i]), 1);
            mbar_init(smem_ptr(&c.piece_free[i]), kPieceReaders);
        }
        mbar_init(smem_ptr(&c.merge_full), 4);
        mbar_init(smem_ptr(&c.merge_free), 4);
        mbar_init(smem_ptr(&c.drained), 1);
        mbar_init_fence();
        c.gave_up = 0;
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
        tma_prefetch_map(&q_map);
    }
    if (warp == 9) {  // all 512 columns: one block per multiprocessor
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_ptr(&c.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&c.tmem);
    pdl_wait();  // the plan is written

    // The next piece, for a whole warp or one thread; false at the end, or when a wait was given up.
    auto next_piece = [&](Ring<kPieceRing>& at, Piece& p, bool one_thread) {
        bool ok = mbar_wait(smem_ptr(&c.piece_full[at.stage]), at.phase, &c.gave_up);
        if (!one_thread) ok = __all_sync(0xffffffffu, ok);
        const int4* src = reinterpret_cast<const int4*>(&c.piece[at.stage]);
        int4* dst = reinterpret_cast<int4*>(&p);
#pragma unroll
        for (int i = 0; i < int(sizeof(Piece) / 16); ++i) dst[i] = src[i];
        if (!one_thread) __syncwarp();
        if (one_thread || lane == 0) mbar_arrive(smem_ptr(&c.piece_free[at.stage]));
        at.step();
        return ok && p.take > 0;
    };
    Ring<kPieceRing> piece_at;
    Piece w;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // -------------------------------------------------------- loads
            const int ppt = max(kKeyTile >> a.page_shift, 1), rows = min(1 << a.page_shift, kKeyTile);
            const int pg = lane % ppt, half = lane / ppt;  // a lane for each page and 64 columns
            Ring<STAGES> at;
            Ring<kLiveRing> tile;
            int n = 0;
            bool go = true;
            while (go && next_piece(piece_at, w, false)) {
                const int32_t* table = a.table + w.request * a.table_stride;
                auto page_of = [&](int i) {  // this lane's page of tile i, -1: none
                    const int k0 = w.key0 + i * kKeyTile + (pg << a.page_shift);
                    return half < HALVES && i < w.take && k0 < w.hi && k0 + rows > w.lo ? table[k0 >> a.page_shift] : -1;
                };
                int page = page_of(0);
                for (int i = 0; go && i < w.take; ++i) {
                    const int next = page_of(i + 1);  // on its way while this tile waits for room
                    const int slot0 = (w.key0 + i * kKeyTile + (pg << a.page_shift)) & ((1 << a.page_shift) - 1);
                    const bool load = page >= 0 && page < a.pages;
                    const uint32_t mask = __ballot_sync(0xffffffffu, load && half == 0);
#pragma unroll 1
                    for (int is_v = 0; is_v < 2; ++is_v, ++n, at.step()) {
                        if (n >= STAGES)
                            go = __all_sync(0xffffffffu, mbar_wait(smem_ptr(&c.empty[at.stage]), at.phase ^ 1, &c.gave_up));
                        if (!go) break;
                        const uint32_t full = smem_ptr(is_v ? &c.v_full[tile.stage] : &c.k_full[tile.stage]);
                        if (lane == 0) {
                            if (!is_v) *(volatile uint32_t*)&c.live[tile.stage] = mask;
                            mbar_arrive_tx(full, uint32_t(__popc(mask)) * uint32_t(rows) * 128u * HALVES);
                        }
                        __syncwarp();
                        if (load)
                            tma_load_box(smem_ptr(ring + at.stage * C::TILE + half * kHalfBytes + pg * rows * 128),
                                         is_v ? &v_map : &k_map, full, half * 64, slot0, w.head, page);
                    }
                    page = next;
                    if (go) tile.step();
                }
            }
            // No copy is left in flight when the block ends, after a wait that was given up too: the last tiles' barriers (the
            // earlier ones have been waited for, or their places would not have been free).
            if (lane == 0) {
                int late = 0;
                Ring<kLiveRing> last = tile;
                for (int i = 0; i < min((n + 1) / 2, STAGES / 2 + 2); ++i) {
                    if (i > 0 || n % 2 == 0) last.back();
                    mbar_wait(smem_ptr(&c.k_full[last.stage]), last.phase, &late);
                    if (i > 0 || n % 2 == 0) mbar_wait(smem_ptr(&c.v_full[last.stage]), last.phase, &late);
                }
                if (late) *(volatile int*)&c.gave_up = 1;
            }
        } else if (warp == 9) {
            // ----------------------------------------------------- products
            // One thread, so that nothing between two products waits for a warp, and one loop with each product in one place: the
            // code that it runs between two pieces would otherwise come from beyond the instruction caches, which the
            // softmax warps keep for themselves (7000 cycles a piece instead of 1000).
            if (elect_one()) {
                constexpr uint32_t s_idesc = tc_idesc<BF16>(kKeyTile, false), o_idesc = tc_idesc<BF16>(D, true);
                const uint32_t q_desc = tc_desc(smem_ptr(q_smem), 1), k_desc = tc_desc(smem_ptr(ring), 1);
                const uint32_t v_desc = tc_desc(smem_ptr(ring), kHalfBytes >> 4);
                Ring<STAGES> k, v;  // of the next K and V; the ring holds K0 V0 K1 V1 ...
                v.step();
                Ring<kLiveRing> k_tile, tile;
                uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
                bool go = true;
                auto await = [&](uint64_t& bar, uint32_t parity) {
                    go = go && mbar_wait(smem_ptr(&bar), parity, &c.gave_up);
                    tc_fence_after();
                };
                while (go && next_piece(piece_at, w, true)) {
                    const int ahead = w.shared ? 2 : 1;  // key tiles between a half's products
#pragma unroll 1
                    for (int i = -ahead; go && i < w.take; ++i) {  // the product with V of tile i, the scores of tile i + ahead
                        const bool more = i + ahead < w.take;
                        if (i >= 0) await(c.clean[tile.stage], tile.phase);
#pragma unroll 1
                        for (int h = w.shared ? i & 1 : 0; go && h < (w.shared ? (i & 1) + 1 : 2); ++h) {
                            const int count = h ? w.count[1] : w.count[0];
                            // of the half's tiles
                            const int of_v = w.shared ? i >> 1 : i, of_k = w.shared ? (i + 2) >> 1 : i + 1;
                            const uint32_t p = tmem + h * 128;
                            if (i >= 0 && of_v < count) {  // O_h += P_h V
                                await(c.p_full[h], h ? p_phase[1] : p_phase[0]);
                                (h ? p_phase[1] : p_phase[0]) ^= 1;
                                if (!go) break;
                                uint32_t vd = v_desc + v.stage * (C::TILE >> 4);
                                asm volatile("" : "+r"(vd));  // the steps are added here, not kept in registers
#pragma unroll
                                for (int x = 0; x < kKeyTile / 16; ++x) {
                                    tc_mma_ta(p + 256, p + 8 * x, vd + 128 * x, o_idesc, of_v > 0 || x > 0);
                                    if constexpr (BF16) tc_mma_ta(p + 256, p + 64 + 8 * x, vd + 128 * x, o_idesc, true);
                                }
                                tc_commit(smem_ptr(&c.o_full[h]));
                            }
                            const bool last = w.shared || h == 1;  // of the halves that read this V and K
                            if (i >= 0 && last) tc_commit(smem_ptr(&c.empty[v.stage]));
                            if (more && (w.shared || h == 0)) await(c.k_full[k_tile.stage], k_tile.phase);
                            if (!go) break;
                            if (more && of_k < count) {  // S_h = Q_h K^T; the last of a piece frees Q
                                if (of_k == 0) {
                                    await(c.q_full[h], h ? q_phase[1] : q_phase[0]);
                                    (h ? q_phase[1] : q_phase[0]) ^= 1;
                                    if (!go) break;
                                }
                                uint32_t qd = q_desc + h * (C::TILE >> 4), kd = k_desc + k.stage * (C::TILE >> 4);
                                asm volatile("" : "+r"(qd), "+r"(kd));
#pragma unroll
                                for (int x = 0; x < D / 16; ++x) {
                                    const uint32_t step = (x >> 2) * (kHalfBytes >> 4) + (x & 3) * 2;
                                    tc_mma(p, qd + step, kd + step, s_idesc, x > 0);
                                }
                                tc_commit(smem_ptr(&c.s_full[h]));
                                if (of_k + 1 == count) tc_commit(smem_ptr(&c.q_free[h]));
                            }
                            if (more && last) tc_commit(smem_ptr(&c.empty[k.stage]));
                        }
                        if (i >= 0) {
                            v.step();
                            v.step();
                            tile.step();
                        }
                        if (more) {
                            k_tile.step();
                            k.step();
                            k.step();
                        }
                    }
                }
                // no product is in flight when tensor memory is freed
                int late = 0;
                tc_commit(smem_ptr(&c.drained));
                mbar_wait(smem_ptr(&c.drained), 0, &late);
                if (late) *(volatile int*)&c.gave_up = 1;
            }
            __syncwarp();
        } else if (warp == 10) {
            // ----------------------------------------------- clearing of V
            // Values that no row sees may be anything, and 0 * NaN is NaN: their rows are cleared before the product.
            Ring<STAGES> at;
            Ring<kLiveRing> tile;
            const int ppt = max(kKeyTile >> a.page_shift, 1);
            const uint32_t all = uint32_t((1ull << ppt) - 1);
            bool go = true;
            while (go && next_piece(piece_at, w, false)) {
                for (int i = 0; go && i < w.take; ++i, tile.step()) {
                    at.step();  // past K
                    go = __all_sync(0xffffffffu, mbar_wait(smem_ptr(&c.v_full[tile.stage]), tile.phase, &c.gave_up));
                    const int key0 = w.key0 + i * kKeyTile;
                    const uint32_t live = *(volatile uint32_t*)&c.live[tile.stage];
                    if (key0 < w.lo || key0 + kKeyTile > w.hi || live != all) {
                        for (int r0 = 0; r0 < kKeyTile; r0 += 2) {
                            const int r = r0 + (lane >> 4), half = (lane >> 3) & 1;
                            const bool seen = key0 + r >= w.lo && key0 + r < w.hi && (live >> (r >> a.page_shift) & 1u);
                            if (!seen && half < HALVES)
                                *reinterpret_cast<uint4*>(ring + at.stage * C::TILE + half * kHalfBytes + r * 128 +
                                                          (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        proxy_fence();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(smem_ptr(&c.clean[tile.stage]));
                    at.step();
                }
            }
        } else if (lane == 0) {
            // -------- the pieces, their Q, and the row tile that this block begins and does not end
            const ChunkStart start = plan.start[blockIdx.x];
            ChunkWalk x;
            x.begin(a, plan, start);
            AttnSplit split{0, 0, 0, 0, -1};
            uint32_t pieces[2] = {0, 0};
            bool go = true;
            for (int n = 0; go; ++n) {
                if (n >= kPieceRing)
                    go = mbar_wait(smem_ptr(&c.piece_free[piece_at.stage]), piece_at.phase ^ 1, &c.gave_up);
                if (!go) break;
                if (x.left <= 0) w.take = 0;
                if (x.left > 0) {
                    const bool whole = x.whole();
                    w.take = x.take;
                    w.count[0] = x.tiles_of(a, 0);
                    w.count[1] = x.tiles_of(a, 1);
                    w.shared = x.t.shared;
                    w.row = x.q.begin + x.t.token0;
                    w.n = x.t.n;
                    w.pos = x.q.kv - x.q.n + x.t.token0;
                    w.kv = x.q.kv;
                    w.key0 = (x.t.first + x.tile) * kKeyTile;
                    w.lo = x.t.lo;
                    w.hi = x.t.hi;
                    w.head = x.head;
                    w.request = x.r;
                    w.slot = whole ? -1 : x.tile > 0 ? 0 : 1;
                    if (!whole && x.tile == 0)  // the last piece
                        split = AttnSplit{w.row, 0, w.n * a.group, x.head, x.last_block(start)};
                }
                c.piece[piece_at.stage] = w;
                mbar_arrive(smem_ptr(&c.piece_full[piece_at.stage]));
                piece_at.step();
                if (x.left <= 0) break;
                x.next(a, plan);  // before the wait for room for Q
                for (int h = 0; h < 2; ++h) {
                    if (w.count[h] == 0) break;
                    // As soon as the piece's last scores are there its Q is not read any more: the next one's loads run beside
                    // the last tile's exponentials, its product and the results.
                    if (pieces[h] > 0) go = go && mbar_wait(smem_ptr(&c.q_free[h]), (pieces[h] - 1) & 1, &c.gave_up);
                    if (!go) break;
                    ++pieces[h];
                    const uint32_t full = smem_ptr(&c.q_full[h]);
                    mbar_arrive_tx(full, uint32_t(HALVES * a.half_tokens * a.group) * 128u);
                    for (int y = 0; y < HALVES; ++y)
                        tma_load_rows(smem_ptr(q_smem + h * C::TILE + y * kHalfBytes), &q_map, full, 64 * y, w.head * a.group,
                                      w.row + (w.shared ? 0 : h * a.half_tokens));
                }
            }
            int late = 0;
            for (int h = 0; h < 2; ++h)
                if (pieces[h] > 0) mbar_wait(smem_ptr(&c.q_full[h]), (pieces[h] - 1) & 1, &late);
            if (late) *(volatile int*)&c.gave_up = 1;
            ws.split[blockIdx.x] = split;
        }
    } else {
        // ------------------------------------------- softmax of one half
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int h = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t s_at = tmem + h * 128 + lanes, o_at = tmem + 256 + h * 128 + lanes;
        const float sc = a.scale * kLog2e;
        constexpr float lift = kLift<BF16, 7>;
        auto wait = [&](uint64_t& bar, uint32_t parity) {
            mbar_wait(smem_ptr(&bar), parity, &c.gave_up);
            __syncwarp();
            tc_fence_after();
        };
        const int row_token = a.by_group.of(row), row_head = row - row_token * a.group;
        int n_s = 0;    // tiles of this half so far
        int tiles = 0;  // tiles of the block before this piece
        uint32_t merges = 0;
        for (; next_piece(piece_at, w, false); tiles += w.take) {
            const int count = h ? w.count[1] : w.count[0];
            if (count == 0) continue;
            const int first = w.shared ? 0 : h * a.half_tokens, n_tokens = min(w.n - first, a.half_tokens);
            const bool mine = row_token < n_tokens;
            const int token = first + min(row_token, n_tokens - 1), head = w.head * a.group + row_head;
            const int lo = keys_from(a, w.pos + token), hi = keys_to(a, w.kv, w.pos + token);
            // keys [all_lo, all_hi) are seen by every row of the half
            const int all_lo = keys_from(a, w.pos + first + n_tokens - 1), all_hi = keys_to(a, w.kv, w.pos + first);
            const int ppt = max(kKeyTile >> a.page_shift, 1);
            const uint32_t all = uint32_t((1ull << ppt) - 1);
            // p = 2^(s sc + neg), lifted in fp16.  neg is the fp32 number nearest to lift - m sc, and rest what it leaves of that; a
            // huge m sc (far) would leave no digits for the difference, there s - m is taken first and neg is the lift.
            float m = -INFINITY, l = 0.0f, neg = 0.0f, rest = 0.0f;
            bool far = false;
            for (int j = 0; j < count; ++j, ++n_s) {
                const int i = w.shared ? 2 * j + h : j;  // of the piece's tiles
                const int key0 = w.key0 + i * kKeyTile;
                wait(c.s_full[h], n_s & 1);
                const uint32_t live = *(volatile uint32_t*)&c.live[(tiles + i) % kLiveRing];
                if (key0 < all_lo || key0 + kKeyTile > all_hi || live != all) {
                    // Keys that the row does not see, in place.  This and the other rare parts are loops over 16 columns in tensor
                    // memory: unrolled over registers they would push the common part out of the instruction caches.
                    const int from = lo - key0, to = hi - key0;
#pragma unroll 1
                    for (int x = 0; x < kKeyTile; x += 16) {
                        const bool page = live >> (x >> a.page_shift) & 1u;
                        const uint32_t see = page ? low_bits(to - x) & ~low_bits(from - x) : 0u;
                        if (__all_sync(0xffffffffu, (see & 0xffffu) == 0xffffu)) continue;
                        float y[16];
                        if (__any_sync(0xffffffffu, (see & 0xffffu) != 0u)) {
                            tm_load16(y, s_at + x);
                            tm_wait<16>(y);
                        }
#pragma unroll
                        for (int z = 0; z < 16; ++z)
                            if (!(see & 1u << z)) y[z] = -INFINITY;
                        tm_store16(s_at + x, reinterpret_cast<const uint32_t*>(y));
                    }
                    tc_wait_st();
                }
                float s[kKeyTile];
                auto load_scores = [&] {
#pragma unroll
                    for (int x = 0; x < kKeyTile; x += 32) tm_load(s + x, s_at + x);
                    tm_wait<kKeyTile>(s);
                };
                load_scores();
                float tops[4];  // four chains: one would be all latency
#pragma unroll
                for (int x = 0; x < 4; ++x) tops[x] = fmaxf(s[2 * x], s[2 * x + 1]);
#pragma unroll
                for (int x = 8; x < kKeyTile; x += 2) tops[x / 2 & 3] = max3(tops[x / 2 & 3], s[x], s[x + 1]);
                const float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]);
                // the reference moves when p would pass 2^kSlack
                const bool moves = top > m && !((top - m) * sc <= kSlack);
                if (__any_sync(0xffffffffu, moves)) {
                    const float m_new = moves ? top : m, scaled = m_new * sc;
                    const bool huge = fabsf(scaled) > kExactRef;
                    const float rest_new = beyond_reference<BF16>(m_new, sc);
                    if (__any_sync(0xffffffffu, moves && m != -INFINITY)) {
                        const float f = moves && m != -INFINITY ? exp2_fast(__fmaf_rn(m - m_new, sc, rest_new - rest)) : 1.0f;
                        wait(c.o_full[h], (n_s - 1) & 1);  // the previous product has added to O
                        l *= f;
#pragma unroll 1
                        for (int x = 0; x < D; x += 16) {
                            float o[16];
                            tm_load16(o, o_at + x);
                            tm_wait<16>(o);
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] *= f;
                            tm_store16(o_at + x, reinterpret_cast<const uint32_t*>(o));
                        }
                        tc_wait_st();
                    }
                    if (moves) {  // O and l are zero as long as m is -infinity
                        m = m_new;
                        rest = rest_new;
                        neg = huge ? lift : lift - scaled;
                        far = huge;
                    }
                }
                if (__any_sync(0xffffffffu, far)) {  // a reference too large for one fp32 number: subtract first
                    const float by = far ? m : 0.0f;
#pragma unroll 1
                    for (int x = 0; x < kKeyTile; x += 16) {
                        float y[16];
                        tm_load16(y, s_at + x);
                        tm_wait<16>(y);
#pragma unroll
                        for (int z = 0; z < 16; ++z) y[z] -= by;
                        tm_store16(s_at + x, reinterpret_cast<const uint32_t*>(y));
                    }
                    tc_wait_st();
                    load_scores();
                }
                const float2 neg2 = make_float2(neg, neg), cc = make_float2(sc, sc);
                float2 sums[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) sums[x] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int x0 = 0; x0 < kKeyTile / 2; x0 += 16) {
                    uint32_t p[16], p_low[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        float2 e = fma2(make_float2(s[2 * (x0 + x)], s[2 * (x0 + x) + 1]), cc, neg2);
                        e.x = exp2_fast(e.x);
                        e.y = exp2_fast(e.y);
                        sums[x & 3] = add2(sums[x & 3], e);
                        p[x] = pack2<BF16>(e.x, e.y);
                        if constexpr (BF16) p_low[x] = pack2<true>(e.x - bf16_low(p[x]), e.y - bf16_high(p[x]));
                    }
                    tm_store16(s_at + x0, p);
                    if constexpr (BF16) tm_store16(s_at + 64 + x0, p_low);
                }
                const float2 sum = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
                l += sum.x + sum.y;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_ptr(&c.p_full[h]));
            }

            // ------------------------------------------------------- results
            wait(c.o_full[h], (n_s - 1) & 1);
            float to_m = exp2_fast(-rest) * (1.0f / kLifted<BF16, 7>);  // from the reference to m
            l *= to_m;
            const bool both = w.shared && w.take > 1, whole = w.slot < 0;
            float to_other = 0.0f;  // the other half's part in the result
            if (both) {
                if (h == 1) {
                    c.m[row] = m;
                    c.l[row] = l;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_ptr(&c.merge_full));
                    wait(c.merge_free, merges++ & 1);  // the first half has read O
                    continue;
                }
                wait(c.merge_full, merges++ & 1);
                const float m1 = c.m[row], top = fmaxf(m, m1);
                const float f0 = m == -INFINITY ? 0.0f : exp2_fast((m - top) * sc);
                const float f1 = m1 == -INFINITY ? 0.0f : exp2_fast((m1 - top) * sc);
                l = l * f0 + c.l[row] * f1;
                to_m *= f0;
                to_other = exp2_fast(-beyond_reference<BF16>(m1, sc)) * (1.0f / kLifted<BF16, 7>) * f1;
                m = top;
            }
            if (whole) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                to_m *= inv;
                to_other *= inv;
            }
            const int piece = (2 * blockIdx.x + w.slot) * 2 + h;  // a piece's half in the workspace
            uint16_t* out =
                static_cast<uint16_t*>(a.out) + int64_t(w.row + token) * a.out_token_stride + head * a.out_head_stride;
#pragma unroll 1
            for (int x0 = 0; x0 < D; x0 += 32) {
                float o[32];
                tm_load(o, o_at + x0);
                tm_wait<32>(o);
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= to_m;
                if (both) {
                    float o1[32];
                    tm_load(o1, o_at + 128 + x0);
                    tm_wait<32>(o1);
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = __fmaf_rn(o1[x], to_other, o[x]);
                }
                if (mine && whole) {
#pragma unroll
                    for (int x = 0; x < 32; x += 16) {
                        uint32_t p[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) p[y] = pack2<BF16>(o[x + 2 * y], o[x + 2 * y + 1]);
                        if (a.out_by_32) {
                            store32(out + x0 + x, p);
                        } else {
                            *reinterpret_cast<uint4*>(out + x0 + x) = make_uint4(p[0], p[1], p[2], p[3]);
                            *reinterpret_cast<uint4*>(out + x0 + x + 8) = make_uint4(p[4], p[5], p[6], p[7]);
                        }
                    }
                } else if (mine) {
                    // 8 columns of the 128 rows together, so that a warp writes 1 KB in one piece
#pragma unroll
                    for (int x = 0; x < 32; x += 8)
                        store32(ws.o + (int64_t(piece) * D + x0 + x) * 128 + row * 8, reinterpret_cast<const uint32_t*>(o + x));
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (both && lane == 0) mbar_arrive(smem_ptr(&c.merge_free));
            if (mine && whole) {
                if (a.lse != nullptr)
                    a.lse[int64_t(w.row + token) * a.q_heads + head] = l > 0.0f ? m * a.scale + logf(l) : -INFINITY;
            } else if (mine) {
                ws.ml[piece * 128 + row] = make_float2(m, l);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *(volatile int*)&c.gave_up) atomicAdd(&g_gave_up, 1ull);
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <int D, bool BF16>
int launch_chunk(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm,
                 const AttnWorkspace& ws, const ChunkPlan& plan) {
    if (!ensure_smem(reinterpret_cast<const void*>(attention_chunk_kernel<D, BF16>), Chunk<D>::SMEM)) return NQ_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kAttnGrid);
    cfg.blockDim = dim3(kThreadsChunk);
    cfg.dynamicSmemBytes = Chunk<D>::SMEM;
    cfg.stream = a.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attention_chunk_kernel<D, BF16>, a, km, vm, qm, ws, plan);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

template <bool BF16>
int launch_chunk(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm,
                 const AttnWorkspace& ws, const ChunkPlan& plan) {
    switch (a.head_dim) {
        case 64: return launch_chunk<64, BF16>(a, km, vm, qm, ws, plan);
        case 96: return launch_chunk<96, BF16>(a, km, vm, qm, ws, plan);
        default: return launch_chunk<128, BF16>(a, km, vm, qm, ws, plan);
    }
}

}  // namespace

uint64_t chunk_workspace(int64_t tokens, int group, int requests, int head_dim) {
    uint64_t bytes = 0;
    chunk_plan(nullptr, chunk_pairs(tokens, 128 / group, requests), requests, &bytes);
    return attn_workspace(nullptr, kChunkRows, head_dim).total + bytes;
}

int launch_attention_chunk(const AttnArgs& a) {
    CUtensorMap km, vm, qm;
    if (!make_pool_maps(a, &km, &vm) || !make_query_map(a, &qm)) return NQ_ERR_CUDA;
    char* base = static_cast<char*>(a.workspace) + (a.mixed ? attn_workspace(nullptr, kSmallRows, a.head_dim).total : 0);
    const AttnWorkspace ws = attn_workspace(base, kChunkRows, a.head_dim);
    uint64_t bytes = 0;
    const int64_t pairs = chunk_pairs(a.tokens, a.half_tokens, a.requests);
    const ChunkPlan plan = chunk_plan(base + ws.total, pairs, a.requests, &bytes);
    attention_plan_kernel<<<1, kPlanThreads, 0, a.stream>>>(a, plan, pairs);
    if (cudaGetLastError() != cudaSuccess) return NQ_ERR_CUDA;
    const int st = a.bf16 ? launch_chunk<true>(a, km, vm, qm, ws, plan) : launch_chunk<false>(a, km, vm, qm, ws, plan);
    return st == NQ_OK ? launch_join_many_rows(a, ws) : st;
}

int read_chunk_gave_up(uint64_t* blocks, cudaStream_t stream) {
    return cudaMemcpyFromSymbolAsync(blocks, g_gave_up, sizeof(uint64_t), 0, cudaMemcpyDeviceToHost, stream) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

}  // namespace nq
