// Host arithmetic of the paged attention, compiled from its own headers for tests that need no GPU.
#include "../e8_lattice_vector_gb300/csrc_paged/nq_paged.h"

extern "C" void workspace_places(uint64_t base, int rows, int head_dim, uint64_t* places) {
    const nq::AttnWorkspace w = nq::attn_workspace(reinterpret_cast<void*>(base), rows, head_dim);
    places[0] = reinterpret_cast<uint64_t>(w.split);
    places[1] = reinterpret_cast<uint64_t>(w.ml);
    places[2] = reinterpret_cast<uint64_t>(w.o);
    places[3] = w.total;
}

// The large kernel's plan, its sums formed one after the other, and every block's walk through it.  Each piece is eleven
// numbers: block, row of q, tokens, KV head, request, first key tile of the piece, key tiles of the piece, of the row tile, whether
// the halves share its rows, and each half's key tiles.
// `last_block`: per block, of the row tile that it begins and does not end, or -1.  Returns the pieces, -1 when there are
// more than `room`; *planned the pairs, *space their room.
#include <vector>

#include "../e8_lattice_vector_gb300/csrc_paged/nq_paged_walk.cuh"

extern "C" long long chunk_pieces(int tokens, int group, int kv_heads, int requests, int table_cols, int page_shift, int causal,
                                  int window, int mixed, const int* q_start, const int* kv_lens, int* pieces, long long room,
                                  int* last_block, long long* planned, long long* space) {
    nq::AttnArgs a = {};
    a.tokens = tokens;
    a.group = group;
    a.kv_heads = kv_heads;
    a.requests = requests;
    a.table_cols = table_cols;
    a.page_shift = page_shift;
    a.causal = causal;
    a.window = window;
    a.mixed = mixed;
    a.half_tokens = 128 / group;
    a.q_start = q_start;
    a.kv_lens = kv_lens;
    std::vector<nq::RowRange> rows(requests);
    std::vector<long long> sums;
    std::vector<int> request, row_tile;
    nq::ChunkPlan plan = {};
    plan.rows = rows.data();
    long long tiles = 0;
    int top = 0;
    for (int r = 0; r < requests; ++r) {
        const nq::Request given = nq::load_request(a, r);
        rows[r] = nq::row_range(a, given, top);
        top = max(top, nq::rows_end(given));
        const nq::Request q = nq::planned_request(a, plan, r);
        for (int i = 0; i < nq::row_tiles_of(a, q); ++i) {
            sums.push_back(tiles);
            request.push_back(r);
            row_tile.push_back(i);
            tiles += nq::row_tile_of(a, q, i).count;
        }
    }
    sums.push_back(tiles);
    const long long pairs = (long long)request.size();
    *planned = pairs;
    *space = nq::chunk_pairs(tokens, a.half_tokens, requests);
    const int cost = tiles * kv_heads >= (long long)nq::kCostFrom * nq::kAttnGrid ? nq::kRowTileCost : 0;
    for (long long p = 0; p <= pairs; ++p) sums[p] += cost * p;
    plan.unit_sum = sums.data();
    plan.pair_request = request.data();
    plan.pair_row_tile = row_tile.data();
    long long n = 0;
    for (int b = 0; b < nq::kAttnGrid; ++b) {
        const nq::ChunkStart start = nq::chunk_start(a, plan, pairs, sums[pairs] * kv_heads, cost, b);
        nq::ChunkWalk x;
        x.begin(a, plan, start);
        last_block[b] = -1;
        for (; x.left > 0; x.next(a, plan)) {
            if (n == room) return -1;
            const int piece[11] = {b,      x.q.begin + x.t.token0, x.t.n,      x.head,           x.r,             x.tile,
                                   x.take, x.t.count,              x.t.shared, x.tiles_of(a, 0), x.tiles_of(a, 1)};
            for (int v : piece) *pieces++ = v;
            ++n;
            if (x.tile == 0 && !x.whole()) last_block[b] = x.last_block(start);
        }
    }
    return n;
}

extern "C" int share_holding(long long total, long long at) { return nq::share_holding(total, at); }

// One GiveUps through a sequence of reads (device, small, chunk); grew[i]: what the i-th says.
extern "C" void give_ups(const uint64_t* reads, int n, int* grew) {
    nq::GiveUps g;
    for (int i = 0; i < n; ++i) grew[i] = g.grew(int(reads[3 * i]), reads[3 * i + 1], reads[3 * i + 2]);
}
