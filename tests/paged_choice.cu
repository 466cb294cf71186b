// Which kernel a call for drafted trees goes to, compiled from the kernels' own headers for a test that needs no GPU.
#include "../e8_lattice_vector_gb300/csrc_paged/nq_paged_walk.cuh"

extern "C" int few_tree_tiles(int tokens, int max_q, int requests, int group, int kv_heads, int head_dim, int page_size, int table_cols,
                              int window) {
    nq_attention a = {};
    a.tokens = tokens;
    a.max_q = max_q;
    a.requests = requests;
    a.q_heads = group * kv_heads;
    a.table_cols = table_cols;
    a.window = window;
    nq_pool p = {};
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    return nq::few_tree_tiles(&a, &p, group);
}
