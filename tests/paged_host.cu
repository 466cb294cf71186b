// Host arithmetic of the paged attention, compiled from its own headers for tests that need no GPU.
#include "../e8_lattice_vector_gb300/csrc_paged/nq_paged.h"

extern "C" void workspace_places(uint64_t base, int rows, int head_dim, uint64_t* places) {
    const nq::AttnWorkspace w = nq::attn_workspace(reinterpret_cast<void*>(base), rows, head_dim);
    places[0] = reinterpret_cast<uint64_t>(w.split);
    places[1] = reinterpret_cast<uint64_t>(w.ml);
    places[2] = reinterpret_cast<uint64_t>(w.o);
    places[3] = w.total;
}
