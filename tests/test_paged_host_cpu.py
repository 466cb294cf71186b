"""Host arithmetic of the paged attention, compiled from its own headers (paged_host.cu): no GPU is needed."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    from e8_lattice_vector_gb300 import build as nqbuild

    out = str(tmp_path_factory.mktemp("paged") / "paged_host.so")
    subprocess.run([nqbuild._nvcc()] + nqbuild.ARCH + ["-std=c++17", "-O1", "-Xcompiler", "-fPIC", "-shared", "-I",
                                                       nqbuild.INCLUDE, os.path.join(HERE, "paged_host.cu"), "-o", out],
                   check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("rows", [16, 256])
@pytest.mark.parametrize("head_dim", [64, 96, 128])
@pytest.mark.parametrize("base", [1 << 20, (1 << 20) + 16, (1 << 20) + 48, (1 << 20) + 240])
def test_workspace_is_aligned_for_any_caller(host, rows, head_dim, base):
    """A scratch buffer on any 16-byte boundary: every array in it begins on a 32-byte boundary at least (the widest store),
    the arrays do not overlap, and they end within the size that is asked for, which does not depend on the buffer."""
    grid, split_bytes = 152, 20
    got, none = (ctypes.c_uint64 * 4)(), (ctypes.c_uint64 * 4)()
    host.workspace_places(ctypes.c_uint64(base), rows, head_dim, got)
    host.workspace_places(ctypes.c_uint64(0), rows, head_dim, none)
    split, ml, o, total = got
    assert total == none[3]
    assert split % 32 == 0 and ml % 32 == 0 and o % 32 == 0
    assert base <= split and split + grid * split_bytes <= ml and ml + grid * 2 * rows * 8 <= o
    assert o + grid * 2 * rows * head_dim * 4 <= base + total


def walk(host, q_start, kv_lens, tokens, group, kv_heads, P=16, cols=1000, causal=1, window=0, mixed=0):
    R, room = len(kv_lens), 1 << 18
    pieces, last = np.zeros((room, 11), np.int32), np.zeros(152, np.int32)
    starts, lens = np.array(q_start, np.int32), np.array(kv_lens, np.int32)
    planned, space = ctypes.c_longlong(), ctypes.c_longlong()
    host.chunk_pieces.restype = ctypes.c_longlong
    p = lambda x: x.ctypes.data_as(ctypes.c_void_p)
    n = host.chunk_pieces(tokens, group, kv_heads, R, cols, P.bit_length() - 1, causal, window, mixed, p(starts), p(lens),
                          p(pieces), ctypes.c_longlong(room), p(last), ctypes.byref(planned), ctypes.byref(space))
    assert n >= 0
    return pieces[:n].tolist(), last.tolist(), planned.value, space.value


def check_walk(host, q_start, kv_lens, tokens, group, kv_heads, mixed=0, **kw):
    """Every row tile's key tiles are taken once, in order; a row tile that several blocks share is begun by one that names its
    last block, and the parts in between are the first pieces of their blocks; no row lies outside q or in two requests."""
    pieces, last, planned, space = walk(host, q_start, kv_lens, tokens, group, kv_heads, mixed=mixed, **kw)
    assert planned <= space, "%d pairs, room for %d" % (planned, space)
    parts, owner = {}, np.full(tokens + 1, -1)
    seen_first = set()
    for b, row, n, head, r, tile, take, count, shared, first, second in pieces:
        assert (first + second == take) if shared else (second == take and 1 <= first <= take)
        assert 0 <= row and n > 0 and row + n <= tokens and 0 <= head < kv_heads and take > 0
        if tile > 0:  # slot 0 of the block's two
            assert b not in seen_first
        seen_first.add(b)
        mine = owner[row:row + n]
        assert ((mine == -1) | (mine == r)).all(), "rows of two requests"
        mine[:] = r
        parts.setdefault((r, row, head), []).append((b, tile, take, count))
    begun = [-1] * 152
    for (r, row, head), p in parts.items():
        at = 0
        for i, (b, tile, take, count) in enumerate(p):
            assert tile == at and b == p[0][0] + i and count == p[0][3]
            at += take
        assert at == p[0][3]
        if len(p) > 1:
            assert begun[p[0][0]] == -1
            begun[p[0][0]] = p[-1][0]
    assert begun == last
    return owner


@pytest.mark.parametrize("q_start,lens", [([0, 4000, 0, 4000], [4000, 4000, 4000]), ([0, 3999, 0, 4000, 0], [9000] * 4),
                                          ([0, 4000] * 40, [5000] * 79), ([4000, 0, 4000], [4000, 4000]),
                                          ([0, 4000, 3000, 3500, 1, 4000, 4000], [6000] * 6),
                                          ([2 ** 31 - 1, -5, 77, 77, 4000], [100, 200, 300, 5000])])
@pytest.mark.parametrize("group", [1, 3, 4, 48])
@pytest.mark.parametrize("mixed", [0, 1])
def test_row_starts_that_decrease_stay_in_the_plan(host, q_start, lens, group, mixed):
    owner = check_walk(host, q_start, lens, 4000, group, 8 if group < 48 else 1, mixed=mixed)
    top = 0
    for r in range(len(lens)):  # a request has its rows past the end of all earlier ones
        taken = np.flatnonzero(owner == r)
        begin, end = (min(max(q, 0), 4000) for q in q_start[r:r + 2])
        if mixed and max(end - begin, 0) * group <= 16:
            assert taken.size == 0
        else:
            assert taken.tolist() == list(range(max(begin, top), end))
        if end > begin:
            top = max(top, end)


@pytest.mark.parametrize("seed", range(40))
def test_shares_and_walk(host, seed):
    """Random batches: starts in order, and starts at random."""
    rng = np.random.default_rng(seed)
    R = int(rng.integers(1, 60))
    lens = rng.integers(0, 200 if seed % 3 else 3, R) * (rng.random(R) < 0.8)
    ctx = rng.integers(0, 5000, R)
    group, kv_heads = int(rng.choice([1, 2, 3, 4, 7, 8, 50, 128])), int(rng.choice([1, 2, 8]))
    kw = dict(mixed=int(rng.integers(0, 2)), causal=int(rng.integers(0, 2)), window=int(rng.choice([0, 0, 1, 300])))
    q_start = np.concatenate([[0], np.cumsum(lens)])
    T = int(q_start[-1])
    owner = check_walk(host, q_start, (ctx + lens).tolist(), T, group, kv_heads, **kw)
    for r in range(R):
        if lens[r] and not (kw["mixed"] and lens[r] * group <= 16):
            assert (owner[q_start[r]:q_start[r + 1]] == r).all()
    wild = rng.integers(-10, T + 10, R + 1)
    check_walk(host, wild, (ctx + lens).tolist(), T, group, kv_heads, **kw)


def test_no_share_lies_past_the_grid(host):
    for total, at in ((1, 5), (152, 152), (1000, 1000), (1000, 10 ** 6), (10 ** 9, 10 ** 9 + 7)):
        assert 0 <= host.share_holding(ctypes.c_longlong(total), ctypes.c_longlong(at)) < 152


def test_every_wait_that_was_given_up_is_reported(host):
    """Counts that only grow: each growth is reported once, also one that comes between another read and its report, for
    either kernel and each device by itself, of any size."""
    reads = [(0, 0, 0, 0), (0, 2, 0, 1), (0, 2, 0, 0), (0, 3, 0, 1), (0, 3, 5, 1), (0, 3, 5, 0),
             (0, 2, 5, 0),  # copied before the last but one report, compared after it
             (1, 0, 0, 0), (1, 1, 0, 1), (0, 3, 6, 1), (0, 2 ** 31 - 1, 6, 1), (0, 2 ** 32 - 1, 6, 1), (0, 2 ** 40, 6, 1), (0, 2 ** 40, 6, 0)]
    flat = np.array([r[:3] for r in reads], np.uint64)
    grew = np.zeros(len(reads), np.int32)
    host.give_ups(flat.ctypes.data_as(ctypes.c_void_p), len(reads), grew.ctypes.data_as(ctypes.c_void_p))
    assert grew.tolist() == [r[3] for r in reads]


def test_barriers_with_the_pieces_of_real_batches(host):
    """The model of the large kernel's barriers, run with the pieces that the kernel's own walk gives its blocks."""
    from test_paged_protocol_cpu import simulate

    rng = np.random.default_rng(1)
    lens = rng.integers(1, 260, 12)
    kv = (lens + rng.integers(0, 900, 12) * (rng.random(12) < 0.7)).tolist()
    starts = np.concatenate([[0], np.cumsum(lens)])
    for group, kv_heads, window in ((4, 8, 0), (1, 2, 300), (3, 8, 0)):
        blocks = {}
        for p in walk(host, starts, kv, int(starts[-1]), group, kv_heads, window=window)[0]:
            b, take, shared, count = p[0], p[6], bool(p[8]), p[9:11]
            mine = blocks.setdefault(b, [])
            mine.append({"id": len(mine), "take": take, "shared": shared, "count": count})
        for b in list(blocks)[::7]:
            for stages in (5, 12):
                simulate(b, stages, blocks[b])


def test_the_model_has_the_kernels_numbers():
    """Ring lengths and arrival counts, from the kernel's source."""
    import re

    import test_paged_protocol_cpu as model

    folder = os.path.join(os.path.dirname(HERE), "e8_lattice_vector_gb300", "csrc_paged")
    source = open(os.path.join(folder, "nq_paged_chunk.cu")).read()
    number = lambda name: int(re.search(r"constexpr int %s = (\d+);" % name, source).group(1))
    assert (number("kLiveRing"), number("kPieceRing"), number("kPieceReaders")) == (model.TILE_RING, model.PIECE_RING, model.READERS)
    counts = dict(re.findall(r"mbar_init\(smem_ptr\(&c\.(\w+)(?:\[i\])?\), (\w+)\);", source))
    one = dict.fromkeys(("empty", "k_full", "v_full", "clean", "q_full", "q_free", "s_full", "o_full", "piece_full", "drained"), "1")
    assert counts == dict(one, p_full="4", merge_full="4", merge_free="4", piece_free="kPieceReaders")
