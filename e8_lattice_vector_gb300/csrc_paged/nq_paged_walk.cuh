// nq_paged_walk.cuh -- which rows and key tiles each block of the large attention kernel takes: the plan's arrays, where a
// block's share begins, and the walk through its pieces.  Plain arithmetic on the step's lengths, for the device and the host.
#pragma once

#include "nq_paged_device.cuh"

namespace nq {

// A row tile costs about this many key tiles on top of its own: its Q, the first scores, the results.  Shares are equal in
// key tiles plus these, or the block whose share is many short row tiles (the beginning of a prompt) would be the last
// to end.  Not counted when a share has few tiles: there a block's idle time is worth more than an even cost.
constexpr int kRowTileCost = 3, kCostFrom = 16;

// Where a block's share begins: `unit` counts the row tile's cost, then its key tiles.
struct ChunkStart {
    int request, row_tile, head, unit;
    long long begin, end, total;
    int cost;
};

// A request's rows of q that are the large kernel's.
struct RowRange {
    int begin, n;
};

struct ChunkPlan {
    ChunkStart* start;     // [kAttnGrid]
    RowRange* rows;        // [requests]
    long long* unit_sum;   // [pairs + 1]: units of the (request, row tile) pairs before, for one KV head
    int* pair_request;     // [pairs]
    int* pair_row_tile;    // [pairs]
};

// Room for the (request, row tile) pairs of any row starts: the requests' rows do not overlap.
inline int64_t chunk_pairs(int64_t tokens, int half_tokens, int requests) { return tokens / (2 * half_tokens) + requests; }

inline ChunkPlan chunk_plan(char* p, int64_t pairs, int requests, uint64_t* total) {
    ChunkPlan c;
    uint64_t off = 0;
    auto take = [&](uint64_t bytes) {
        char* at = p + off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    c.start = reinterpret_cast<ChunkStart*>(take(kAttnGrid * sizeof(ChunkStart)));
    c.rows = reinterpret_cast<RowRange*>(take(uint64_t(requests) * sizeof(RowRange)));
    c.unit_sum = reinterpret_cast<long long*>(take(uint64_t(pairs + 1) * sizeof(long long)));
    c.pair_request = reinterpret_cast<int*>(take(uint64_t(pairs) * sizeof(int)));
    c.pair_row_tile = reinterpret_cast<int*>(take(uint64_t(pairs) * sizeof(int)));
    *total = off;
    return c;
}

// Row starts may decrease, by mistake; a request then has those of its rows that lie past the end of all earlier requests'
// (`top`), so that no row belongs to two requests and the pairs never pass their room.  The requests that the small kernel
// takes, by their rows as they are given, have none here.
__host__ __device__ __forceinline__ RowRange row_range(const AttnArgs& a, const Request& q, int top) {
    const bool smalls = a.mixed && q.n * a.group <= kSmallRows;
    const int begin = max(q.begin, top);
    return RowRange{begin, smalls ? 0 : max(q.begin + q.n - begin, 0)};
}
// The end of the request's rows as they are given, 0 when it has none.
__host__ __device__ __forceinline__ int rows_end(const Request& q) { return q.n > 0 ? q.begin + q.n : 0; }
__host__ __device__ __forceinline__ Request planned_request(const AttnArgs& a, const ChunkPlan& plan, int r) {
    const RowRange rows = plan.rows[r];
    return Request{rows.begin, rows.n, load_kv(a, r)};
}

__host__ __device__ __forceinline__ int row_tiles_of(const AttnArgs& a, const Request& q) {
    return (q.n + 2 * a.half_tokens - 1) / (2 * a.half_tokens);
}

// The tokens and keys of one row tile.
struct RowTile {
    int token0, n, lo, hi;  // n tokens; keys [lo, hi) are seen by some of them
    int first, count;       // key tiles, at least one so that rows without keys are written too
    bool shared;            // one half's tokens, for both halves
};
__host__ __device__ __forceinline__ RowTile row_tile_of(const AttnArgs& a, const Request& q, int row_tile) {
    RowTile t;
    t.token0 = row_tile * 2 * a.half_tokens;
    t.n = min(q.n - t.token0, 2 * a.half_tokens);
    t.shared = t.n <= a.half_tokens;
    const int p0 = q.kv - q.n + t.token0;
    t.lo = keys_from(a, p0);
    t.hi = keys_to(a, q.kv, p0 + t.n - 1);
    t.first = min(t.lo, t.hi) / kKeyTile;
    t.count = max((t.hi + kKeyTile - 1) / kKeyTile - t.first, 1);
    return t;
}

// Where block b's share of `units` begins; the sums over all pairs are written.
__host__ __device__ __forceinline__ ChunkStart chunk_start(const AttnArgs& a, const ChunkPlan& plan, long long pairs,
                                                           long long units, int cost, int b) {
    const Shares shares(units);
    const long long begin = shares.begin(b);
    ChunkStart start{0, 0, 0, 0, begin, shares.begin(b + 1), units, cost};
    if (begin >= units) return start;
    // the last pair that begins at or before `at`
    auto last_at = [&](long long lo, long long hi, long long heads, long long at) {
        while (hi - lo > 1) {
            const long long mid = (lo + hi) >> 1;
            if (plan.unit_sum[mid] * heads <= at)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    // a pair of the request (the requests before it count for all heads)
    const long long some = last_at(0, pairs, a.kv_heads, begin);
    const long long p0 = some - plan.pair_row_tile[some];
    start.request = plan.pair_request[some];
    const long long p1 = min(p0 + row_tiles_of(a, planned_request(a, plan, start.request)), pairs);
    const long long from = plan.unit_sum[p0];
    const long long of_head = plan.unit_sum[p1] - from, at = begin - from * a.kv_heads;
    start.head = int(at / of_head);
    const long long rest = at - start.head * of_head + from, p = last_at(p0, p1, 1, rest);
    start.row_tile = int(p - p0);
    start.unit = int(rest - plan.unit_sum[p]);
    return start;
}

// Walks the pieces of a block's share.
struct ChunkWalk {
    int r, row_tile, head, unit, cost;
    long long left;  // units
    Request q;
    int row_tiles;
    RowTile t;
    int tile, take;  // the piece: key tiles [tile, tile + take) of the row tile; take > 0 while left > 0

    __host__ __device__ __forceinline__ void begin(const AttnArgs& a, const ChunkPlan& plan, const ChunkStart& s) {
        r = s.request;
        row_tile = s.row_tile;
        head = s.head;
        unit = s.unit;
        cost = s.cost;
        left = s.end - s.begin;
        if (left > 0) {
            q = planned_request(a, plan, r);
            row_tiles = row_tiles_of(a, q);
            t = row_tile_of(a, q, row_tile);
            if (!piece()) next(a, plan);
        }
    }
    __host__ __device__ __forceinline__ bool piece() {
        const int end = int(min((long long)(t.count + cost), unit + left));
        tile = max(unit - cost, 0);
        take = end - cost - tile;
        return take > 0;
    }
    // The piece is the row tile from its first key tile to its last.
    __host__ __device__ __forceinline__ bool whole() const { return tile == 0 && take == t.count; }
    // Of the row tile that this share begins and does not end: the block whose share holds its last key tile.
    __host__ __device__ __forceinline__ int last_block(const ChunkStart& s) const {
        return share_holding(s.total, s.end - 1 + (t.count - take));
    }
    // Half h's key tiles of the piece (at least one unless shared: its results are written in any case).
    __host__ __device__ __forceinline__ int tiles_of(const AttnArgs& a, int h) const {
        if (t.shared) return (take + 1 - h) >> 1;
        if (h == 1) return take;
        const int hi = keys_to(a, q.kv, q.kv - q.n + t.token0 + a.half_tokens - 1);
        return min(max((hi + kKeyTile - 1) / kKeyTile - t.first - tile, 1), take);
    }
    __host__ __device__ __forceinline__ void next(const AttnArgs& a, const ChunkPlan& plan) {
        do {
            const int n = int(min((long long)(t.count + cost - unit), left));
            left -= n;
            if (left <= 0) return;
            unit = 0;
            if (++row_tile >= row_tiles) {
                row_tile = 0;
                if (++head >= a.kv_heads) {
                    head = 0;
                    do {
                        if (++r >= a.requests) {  // not reached while the lengths stay as they were summed
                            left = 0;
                            return;
                        }
                        q = planned_request(a, plan, r);
                        row_tiles = row_tiles_of(a, q);
                    } while (row_tiles == 0);
                }
            }
            t = row_tile_of(a, q, row_tile);
        } while (!piece());
    }
};

}  // namespace nq
