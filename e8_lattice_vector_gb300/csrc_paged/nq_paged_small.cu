// nq_paged_small.cu -- attention of a few rows per request over the paged cache (single tokens and short drafts:
// 16 rows for each KV head, rows being tokens times the query heads that share it; the few requests of a step that
// have up to twice as many get a second row tile, which reads their keys again).
//
// The time is that of reading K and V once: 2 * 2 * head_dim bytes a key against 4 * rows * head_dim operations, 16
// operations a byte at most.  So the design is about bytes in flight: one block per multiprocessor with a ring of
// 128-key tiles in shared memory (192 KB, four times what the memory's latency needs), filled by one warp with
// one TMA box per page and 64 columns, and eight warps that take 16 keys each of every tile with no barrier between
// them.  A warp keeps its own running maximum, sum and 16 x head_dim accumulator in registers
// (mma m16n8k16); the eight are joined through shared memory when a row tile ends.  tcgen05 has no shape this small that
// would help: the tensor pipe is busy 17% of the time as it is.
//
// Measured: 64 requests over 16384 (32 query heads on 8 KV heads, head_dim 128, fp16, pages of 16) 619 us, 6.9 TB/s of K and V,
// above the measured copy rate; one request over 131072 (40 on 8, bf16) 88 us, 6.1 TB/s; one over 1501 10.3 us, of which
// the launches, the first loads and the joining launch are all but one.  Bound by memory, and by about 12 us at both ends.
#include "nq_paged_device.cuh"

namespace nq {
namespace {

__device__ unsigned long long g_gave_up;  // blocks that gave up a wait, ever

constexpr int kWarps = 8;
constexpr int kConsumers = kWarps * 32;
constexpr int kThreadsSmall = kConsumers + 32;  // the last warp loads

// Place of (row, column) in a warp's 16 x 64 block of the join buffer: rows shifted so that eight of them do not share banks.
__device__ __forceinline__ int join_at(int warp, int row, int col) {
    return (warp * 16 + row) * 64 + (col ^ ((row & 7) << 3));
}

template <int D>
struct Small {
    static constexpr int HALVES = D > 64 ? 2 : 1;
    static constexpr int STAGE = 2 * HALVES * kHalfBytes;  // K then V
    static constexpr int STAGES = 192 * 1024 / STAGE;
    static constexpr int JOIN = kWarps * kSmallRows * 64 * 4;
    static constexpr int SMEM = 1024 + STAGES * STAGE + JOIN;
};

struct Control {
    uint64_t full[6], empty[6];
    uint32_t live[6];  // per stage: which of the tile's pages are loaded
    int gave_up;
    int request, row_tile, head, tile;  // where the block's share begins
    long long pos, end, total;
    long long warp_sum[kThreadsSmall / 32];
    float m[kWarps][kSmallRows], l[kWarps][kSmallRows];
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles of one row tile of a request: the same for each of its row tiles (several for the longer drafts and for groups
// of more heads than a row tile has rows), at least one so that rows without keys are written too.
struct Span {
    int first, count;  // key tiles
    int row_tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Request& q) {
    Span s;
    s.row_tiles = (q.n * a.group + kSmallRows - 1) / kSmallRows;
    if (a.mixed && s.row_tiles > 1) s.row_tiles = 0;  // the large kernel's
    const int lo = min(keys_from(a, q.kv - q.n), q.kv);
    s.first = lo / kKeyTile;
    s.count = max((q.kv + kKeyTile - 1) / kKeyTile - s.first, 1);
    return s;
}

// Walks the pieces of a block's share.
struct Walk {
    int r, row_tile, head, tile;
    long long left;
    Request q;
    Span s;

    __device__ __forceinline__ void begin(const AttnArgs& a, const Control& c) {
        r = c.request;
        row_tile = c.row_tile;
        head = c.head;
        tile = c.tile;
        left = c.end - c.pos;
        if (left > 0) {
            q = load_request(a, r);
            s = span_of(a, q);
        }
    }
    // Tiles [tile, tile + take()) of the current row tile are this block's.
    __device__ __forceinline__ int take() const { return int(min((long long)(s.count - tile), left)); }
    __device__ __forceinline__ void next(const AttnArgs& a, int kv_heads) {
        const int n = take();
        left -= n;
        tile += n;
        if (tile < s.count) return;  // left == 0
        tile = 0;
        if (++row_tile < s.row_tiles) return;  // the same keys once more, out of the L2
        row_tile = 0;
        if (++head < kv_heads) return;
        head = 0;
        if (left <= 0) return;
        do {
            if (++r >= a.requests) {  // not reached while the lengths stay as they were summed
                left = 0;
                return;
            }
            q = load_request(a, r);
            s = span_of(a, q);
        } while (s.row_tiles == 0);
    }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreadsSmall, 1)
    attention_small_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                           const __grid_constant__ CUtensorMap v_map, const AttnWorkspace ws) {
    using S = Small<D>;
    constexpr int HALVES = S::HALVES, NT = D / 8, KS = D / 16;
    extern __shared__ char smem_raw[];
    __shared__ Control c;
    char* ring = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* join = reinterpret_cast<float*>(ring + S::STAGES * S::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(smem_ptr(&c.full[i]), 1);
            mbar_init(smem_ptr(&c.empty[i]), kWarps);
        }
        mbar_init_fence();
        c.gave_up = 0;
        c.pos = c.end = 0;
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
    }
    pdl_trigger();

    // The share: tiles [pos, end) of all tiles in order.  Every thread sums the tiles of its requests.
    const int per = (a.requests + kThreadsSmall - 1) / kThreadsSmall;
    const int r0 = min(int(threadIdx.x) * per, a.requests), r1 = min(r0 + per, a.requests);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) {
        const Span s = span_of(a, load_request(a, r));
        mine += (long long)s.row_tiles * s.count * a.kv_heads;
    }
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) c.warp_sum[warp] = sum;
    __syncthreads();
    long long before = sum - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreadsSmall / 32; ++w) {
        if (w < warp) before += c.warp_sum[w];
        total += c.warp_sum[w];
    }
    const Shares shares(total);
    const long long pos = shares.begin(blockIdx.x), end = shares.begin(blockIdx.x + 1);
    if (pos < end && pos >= before && pos < before + mine) {
        long long at = pos - before;
        int r = r0;
        Span s = span_of(a, load_request(a, r));
        for (;; s = span_of(a, load_request(a, ++r))) {
            const long long n = (long long)s.row_tiles * s.count * a.kv_heads;
            if (at < n) break;
            at -= n;
        }
        const long long per_head = (long long)s.count * s.row_tiles;
        c.request = r;
        c.head = int(at / per_head);
        at %= per_head;
        c.row_tile = int(at / s.count);
        c.tile = int(at % s.count);
        c.pos = pos;
        c.end = end;
        c.total = total;
    }
    __syncthreads();

    Walk w;
    w.begin(a, c);
    if (warp == kWarps) {
        // ------------------------------------------------------------ loads
        const int pages_per_tile = max(kKeyTile >> a.page_shift, 1);
        const int rows = min(1 << a.page_shift, kKeyTile);
        const int pg = lane % pages_per_tile, rest = lane / pages_per_tile;
        const int half = rest % HALVES, is_v = rest / HALVES;
        int n = 0;
        bool go = true;
        while (go && w.left > 0) {
            const int take = w.take();
            const int p0 = w.q.kv - w.q.n + a.by_group.of(w.row_tile * kSmallRows);
            const int p1 = w.q.kv - w.q.n + a.by_group.of(min((w.row_tile + 1) * kSmallRows, w.q.n * a.group) - 1);
            const int lo = keys_from(a, p0), hi = keys_to(a, w.q.kv, p1);
            const int32_t* table = a.table + w.r * a.table_stride;
            auto page_of = [&](int i) {  // this lane's page of tile i of the piece, -1: none
                const int k0 = (w.s.first + w.tile + i) * kKeyTile + (pg << a.page_shift);
                return rest < 2 * HALVES && i < take && k0 < hi && k0 + rows > lo ? table[k0 >> a.page_shift] : -1;
            };
            int page = page_of(0);
            for (int i = 0; i < take; ++i, ++n) {
                const int next = page_of(i + 1);  // on its way while this tile waits for room
                const int k0 = (w.s.first + w.tile + i) * kKeyTile + (pg << a.page_shift);
                const bool load = page >= 0 && page < a.pages;
                const int st = n % S::STAGES;
                if (n >= S::STAGES)
                    go = __all_sync(0xffffffffu, mbar_wait(smem_ptr(&c.empty[st]), (n / S::STAGES - 1) & 1, &c.gave_up));
                if (!go) break;
                const uint32_t mask = __ballot_sync(0xffffffffu, load && rest == 0);
                const uint32_t full = smem_ptr(&c.full[st]);
                if (lane == 0) {
                    c.live[st] = mask;
                    mbar_arrive_tx(full, uint32_t(__popc(mask)) * uint32_t(rows) * 128u * HALVES * 2u);
                }
                __syncwarp();
                if (load) {
                    const uint32_t dst = smem_ptr(ring + st * S::STAGE + (is_v * HALVES + half) * kHalfBytes + pg * rows * 128);
                    tma_load_box(dst, is_v ? &v_map : &k_map, full, half * 64, k0 & ((1 << a.page_shift) - 1), w.head, page);
                }
                page = next;
            }
            w.next(a, a.kv_heads);
        }
        // no copy is left in flight when the block ends, after a wait that was given up too
        if (lane == 0) {
            int late = 0;
            for (int i = max(n - S::STAGES, 0); i < n; ++i)
                mbar_wait(smem_ptr(&c.full[i % S::STAGES]), (i / S::STAGES) & 1, &late);
            if (late || *(volatile int*)&c.gave_up) atomicAdd(&g_gave_up, 1ull);
        }
        return;
    }

    // -------------------------------------------------------------- compute
    const float sc = a.scale * kLog2e;
    constexpr float lifted = kLifted<BF16, 14>;
    const int rq = lane >> 2, cq = lane & 3;  // this lane's rows rq, rq + 8 and its column pair
    if (threadIdx.x == 0) ws.split[blockIdx.x].last_block = -1;
    int n = 0;
    bool first = true;
    for (; w.left > 0; first = false) {
        const int take = w.take();
        const int row0 = w.row_tile * kSmallRows, n_rows = min(w.q.n * a.group - row0, kSmallRows);
        const int pbase = w.q.kv - w.q.n;
        // rows of the tile: positions and the fragments of q
        int pos2[2];
        uint32_t qf[KS][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = rq + 8 * e;
            const int gi = row0 + min(row, n_rows - 1), t = a.by_group.of(gi), h = w.head * a.group + gi - t * a.group;
            pos2[e] = pbase + t;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                                    (w.q.begin + t) * a.q_token_stride +
                                                                    h * a.q_head_stride);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][e] = __ldg(src + 8 * k + cq);
                qf[k][e + 2] = __ldg(src + 8 * k + cq + 4);
            }
        }
        const int p_min = pbase + a.by_group.of(row0), p_max = pbase + a.by_group.of(row0 + n_rows - 1);
        const int lo = keys_from(a, p_min), hi = keys_to(a, w.q.kv, p_max);
        // keys [all_lo, all_hi) are seen by every row
        const int all_lo = keys_from(a, p_max), all_hi = keys_to(a, w.q.kv, p_min);
        float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;

        for (int i = 0; i < take; ++i, ++n) {
            const int st = n % S::STAGES;
            mbar_wait(smem_ptr(&c.full[st]), (n / S::STAGES) & 1, &c.gave_up);
            const int key = (w.s.first + w.tile + i) * kKeyTile + warp * 16;  // this warp's 16 keys
            // the same for all lanes, given up or not
            const bool live =
                __any_sync(0xffffffffu, key < hi && key + 16 > lo && (c.live[st] >> (warp * 16 >> a.page_shift) & 1u));
            if (live) {
                const uint32_t kb = smem_ptr(ring + st * S::STAGE), vb = kb + HALVES * kHalfBytes;
                float s[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.0f;
                {
                    const int row = warp * 16 + (lane >> 4) * 8 + (lane & 7);
                    const uint32_t rb = kb + row * 128;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const int ch = 2 * k + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldsm4(b, rb + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (row & 7)) << 4));
                        mma16816<BF16>(s[0], qf[k], b[0], b[1]);
                        mma16816<BF16>(s[1], qf[k], b[2], b[3]);
                    }
                }
                const bool partial = key < all_lo || key + 16 > all_hi;
                if (partial) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int kk = key + 8 * j + 2 * cq + (e & 1), p = pos2[e >> 1];
                            if (kk < keys_from(a, p) || kk >= keys_to(a, w.q.kv, p)) s[j][e] = -INFINITY;
                        }
                }
                bool grew = false;
                float base[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    base[e] = fmaxf(m[e], x);
                    grew |= base[e] > m[e];
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // m = -inf: nothing summed yet (and base may be -inf too, which would make a NaN)
                        const float keep = m[e] == -INFINITY ? 0.0f : exp2_fast((m[e] - base[e]) * sc);
                        m[e] = base[e];
                        l[e] *= keep;
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            o[j][2 * e] *= keep;
                            o[j][2 * e + 1] *= keep;
                        }
                    }
                }
                // p in 16 bits, lifted in fp16 (o is 2^14 times too large until it is joined): fp16's rounding error (2^-11 of p)
                // is what out's own rounding costs at most, bf16's (2^-8) would show beside it in a mean of many, so there p
                // goes in as the sum of two bf16 (2^-17); its second product hides behind the loads
                uint32_t pf[4], pl[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mm = m[e] == -INFINITY ? 0.0f : m[e];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // subtracted before it is scaled: exact for the largest scores too
                        const float p0 = exp2_fast((s[j][2 * e] - mm) * sc), p1 = exp2_fast((s[j][2 * e + 1] - mm) * sc);
                        l[e] += p0 + p1;
                        pf[2 * j + e] = pack2<BF16>(p0 * lifted, p1 * lifted);
                        if constexpr (BF16)
                            pl[2 * j + e] = pack2<true>(p0 - bf16_low(pf[2 * j + e]), p1 - bf16_high(pf[2 * j + e]));
                    }
                }
                const int row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
                const uint32_t rb = vb + row * 128;
                // a value that no row sees may be anything, and 0 * NaN is NaN: such keys' values are cleared
                uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                const bool edge = key < lo || key + 16 > hi;
                if (edge) {
                    const int k0 = key + 2 * cq;
                    keep0 = (k0 >= lo && k0 < hi ? 0xffffu : 0u) | (k0 + 1 >= lo && k0 + 1 < hi ? 0xffff0000u : 0u);
                    keep1 = (k0 + 8 >= lo && k0 + 8 < hi ? 0xffffu : 0u) |
                            (k0 + 9 >= lo && k0 + 9 < hi ? 0xffff0000u : 0u);
                }
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    const int ch = 2 * j + (lane >> 4);
                    uint32_t b[4];
                    ldsm4_t(b, rb + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (row & 7)) << 4));
                    mma16816<BF16>(o[2 * j], pf, b[0] & keep0, b[1] & keep1);
                    mma16816<BF16>(o[2 * j + 1], pf, b[2] & keep0, b[3] & keep1);
                    if constexpr (BF16) {
                        mma16816<BF16>(o[2 * j], pl, b[0] & keep0, b[1] & keep1);
                        mma16816<BF16>(o[2 * j + 1], pl, b[2] & keep0, b[3] & keep1);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_ptr(&c.empty[st]));
        }

        // -------------------------------- join the eight warps' accumulators
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (cq == 0) {
                c.m[warp][rq + 8 * e] = m[e];
                c.l[warp][rq + 8 * e] = l[e];
            }
        }
        named_barrier<1, kConsumers>();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = c.m[0][rq + 8 * e];
#pragma unroll
            for (int v = 1; v < kWarps; ++v) top = fmaxf(top, c.m[v][rq + 8 * e]);
            const float f = m[e] == -INFINITY ? 0.0f : exp2_fast((m[e] - top) * sc) * (1.0f / lifted);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j][2 * e] *= f;
                o[j][2 * e + 1] *= f;
            }
        }
        const int row = threadIdx.x >> 4, col4 = (threadIdx.x & 15) * 4;  // this thread's outputs in each 64 columns
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) top = fmaxf(top, c.m[v][row]);
#pragma unroll
        for (int v = 0; v < kWarps; ++v)
            sum += c.m[v][row] == -INFINITY ? 0.0f : c.l[v][row] * exp2_fast((c.m[v][row] - top) * sc);
        const bool whole = w.tile == 0 && take == w.s.count;
        const int slot = 2 * blockIdx.x + (first && w.tile > 0 ? 0 : 1);
        const int token = a.by_group.of(row0 + row), t = w.q.begin + token, h = w.head * a.group + row0 + row - token * a.group;
#pragma unroll
        for (int x = 0; x < D; x += 64) {
            if (x) named_barrier<1, kConsumers>();  // the first 64 columns are read
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (x / 8 + j >= NT) break;
                *reinterpret_cast<float2*>(join + join_at(warp, rq, 8 * j + 2 * cq)) =
                    make_float2(o[x / 8 + j][0], o[x / 8 + j][1]);
                *reinterpret_cast<float2*>(join + join_at(warp, rq + 8, 8 * j + 2 * cq)) =
                    make_float2(o[x / 8 + j][2], o[x / 8 + j][3]);
            }
            named_barrier<1, kConsumers>();
            if (row < n_rows && x + col4 < D) {
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    const float4 y = *reinterpret_cast<const float4*>(join + join_at(v, row, col4));
                    acc.x += y.x;
                    acc.y += y.y;
                    acc.z += y.z;
                    acc.w += y.w;
                }
                if (whole) {
                    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
                    uint2 packed;
                    packed.x = pack2<BF16>(acc.x * inv, acc.y * inv);
                    packed.y = pack2<BF16>(acc.z * inv, acc.w * inv);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + t * a.out_token_stride +
                                              h * a.out_head_stride + x + col4) = packed;
                    if (x + col4 == 0 && a.lse != nullptr)
                        a.lse[int64_t(t) * a.q_heads + h] = sum > 0.0f ? top * a.scale + logf(sum) : -INFINITY;
                } else {
                    *reinterpret_cast<float4*>(ws.o + (int64_t(slot) * kSmallRows + row) * D + x + col4) = acc;
                    if (x + col4 == 0) ws.ml[slot * kSmallRows + row] = make_float2(top, sum);
                }
            }
        }
        if (threadIdx.x == 0 && w.tile == 0 && !whole) {
            // this block began the row tile: the block of its last tile is the one whose share holds it
            ws.split[blockIdx.x] =
                AttnSplit{w.q.begin, row0, n_rows, w.head, share_holding(c.total, c.end - 1 + (w.s.count - take))};
        }
        named_barrier<1, kConsumers>();  // the join buffer and the sums are read
        w.next(a, a.kv_heads);
    }
    if (threadIdx.x == 0 && *(volatile int*)&c.gave_up) atomicAdd(&g_gave_up, 1ull);
}

}  // namespace

template <int D, bool BF16>
static int launch_small(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const AttnWorkspace& ws) {
    if (!ensure_smem(reinterpret_cast<const void*>(attention_small_kernel<D, BF16>), Small<D>::SMEM)) return NQ_ERR_CUDA;
    attention_small_kernel<D, BF16><<<kAttnGrid, kThreadsSmall, Small<D>::SMEM, a.stream>>>(a, km, vm, ws);
    return cudaGetLastError() == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

template <bool BF16>
static int launch_small(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const AttnWorkspace& ws) {
    switch (a.head_dim) {
        case 64: return launch_small<64, BF16>(a, km, vm, ws);
        case 96: return launch_small<96, BF16>(a, km, vm, ws);
        default: return launch_small<128, BF16>(a, km, vm, ws);
    }
}

int launch_attention_small(const AttnArgs& a) {
    CUtensorMap km, vm;
    if (!make_pool_maps(a, &km, &vm)) return NQ_ERR_CUDA;
    const AttnWorkspace ws = attn_workspace(a.workspace, kSmallRows, a.head_dim);
    const int st = a.bf16 ? launch_small<true>(a, km, vm, ws) : launch_small<false>(a, km, vm, ws);
    return st == NQ_OK ? launch_join_few_rows(a, ws) : st;
}

int read_small_gave_up(uint64_t* blocks, cudaStream_t stream) {
    return cudaMemcpyFromSymbolAsync(blocks, g_gave_up, sizeof(uint64_t), 0, cudaMemcpyDeviceToHost, stream) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

}  // namespace nq
