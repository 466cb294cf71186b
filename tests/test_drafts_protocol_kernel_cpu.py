"""The model of the barriers with three score buffers (test_drafts_protocol_cpu) against the kernel: its numbers are the source's, and it
runs with the pieces that the kernel's own walk gives its blocks."""
import os
import re

import numpy as np

import test_drafts_protocol_cpu as model
from test_paged_host_cpu import host, walk  # noqa: F401  (host is a fixture)
from test_paged_protocol_cpu import PIECE_RING, READERS, TILE_RING

FOLDER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "e8_lattice_vector_gb300", "csrc_paged")


def _source():
    return "".join(open(os.path.join(FOLDER, f)).read() for f in ("nq_paged_device.cuh", "nq_paged_chunk.cu"))


def test_the_model_has_the_kernels_numbers():
    source = _source()

    def number(name, **known):
        """A constant's expression of whole numbers and the names that are known."""
        text = re.search(r"constexpr int %s = ([^;]+);" % name, source).group(1).replace("/", "//")
        return eval(text, {"__builtins__": {}}, known)

    half = number("kHalfBytes", kKeyTile=number("kKeyTile"))
    halves = re.search(r"constexpr int HALVES = D > 64 \? (\d) : (\d);", source)
    assert halves.groups() == ("2", "1")  # of a tile; at head_dim 64 one
    tile = number("TILE", HALVES=1, kHalfBytes=half)
    assert number("STAGES", Q=number("Q", TILE=tile), TILE=tile) == model.STAGES
    assert re.search(r"constexpr int kScoreBuffers = TREE && D == 64 \? (\d) : 2;", source).group(1) == str(model.BUFFERS)
    assert (number("kLiveRing"), number("kPieceRing"), number("kPieceReaders")) == (TILE_RING, PIECE_RING, READERS)
    # two barriers for each half that take turns, and the arrivals of each
    assert re.search(r"turn_of\(int h, int n\) \{\s+return BUFFERS == 3 \? 2 \* h \+ \(n & 1\) : h;", source)
    assert re.search(r"turn_parity\(int n\) \{\s+return \(BUFFERS == 3 \? n >> 1 : n\) & 1;", source)
    assert re.search(r"uint64_t s_full\[4\], p_full\[4\], o_full\[4\];", source)
    counts = dict(re.findall(r"mbar_init\(smem_ptr\(&c\.(\w+)(?:\[i\])?\), (\w+)\);", source))
    one = dict.fromkeys(("empty", "k_full", "v_full", "clean", "q_full", "q_free", "s_full", "o_full", "piece_full", "drained"), "1")
    assert counts == dict(one, p_full="4", merge_full="4", merge_free="4", piece_free="kPieceReaders")


def test_three_buffers_with_the_pieces_of_real_batches(host):  # noqa: F811
    """Trees of one half's rows and of two, several pieces in a block, and row tiles that several blocks share."""
    rng, most, shared = np.random.default_rng(2), 0, set()
    for nodes, group, kv_heads in ((20, 4, 8), (64, 4, 8), (100, 3, 8), (150, 1, 2)):
        lens = rng.integers(nodes // 2, nodes + 1, 12)
        kv = (lens + rng.integers(0, 1500, 12) * (rng.random(12) < 0.8)).tolist()
        starts = np.concatenate([[0], np.cumsum(lens)])
        blocks = {}
        for p in walk(host, starts, kv, int(starts[-1]), group, kv_heads)[0]:
            mine = blocks.setdefault(p[0], [])
            mine.append({"id": len(mine), "take": p[6], "shared": bool(p[8]), "count": p[9:11]})
            shared.add(bool(p[8]))
        most = max(most, *(len(b) for b in blocks.values()))
        for b in list(blocks)[::9]:
            model.simulate(b, blocks[b])
    assert most > 1 and shared == {False, True}
