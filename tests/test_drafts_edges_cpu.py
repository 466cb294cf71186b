"""Refusals and bookkeeping around drafted trees that test_drafts_cpu leaves out: no GPU is needed."""
import pytest
import torch

from test_drafts_cpu import run
from test_paged_cpu import ARG, I32, I64, P2, P16, UNSUPPORTED, _Fake, nq  # noqa: F401


def test_release_that_clears_refusals(nq):
    f = nq.lib().nq_page_release_clear
    good = [P16, 7, 7, P16, P16, 3, 16, P16, 5, P16, None]
    run(f, good, [(i, None, ARG) for i in (0, 3, 4, 7, 9)] + [(i, -1, ARG) for i in (2, 5, 8)] + [(1, 6, ARG)] +
        [(i, P2, ARG) for i in (0, 3, 4, 7, 9)] + [(6, v, UNSUPPORTED) for v in (0, -16, 8, 24, 512)])
    import e8_lattice_vector_gb300 as pkg

    table, lens = _Fake((3, 7), I32), _Fake((3,), I32)
    for text, kw in (("free_pages must be", {"free": _Fake((9,), I64)}), ("keep_lens has", {"k": _Fake((4,), I32)}),
                     ("top is 10", {"top": 10})):
        a = dict({"free": _Fake((9,), I32), "k": lens, "top": 4}, **kw)
        with pytest.raises(ValueError, match=text):
            pkg.page_release(table, lens, a["k"], 16, a["free"], a["top"], clear=True)


class _Steps:
    """A PagedCache on the CPU whose calls of the library are written down."""

    def __init__(self, monkeypatch, requests=2, tokens=16 * 500, counts=None):
        from e8_lattice_vector_gb300 import serve
        from e8_lattice_vector_gb300.drafts import DraftTree, draft_tree
        from e8_lattice_vector_gb300.paged import PageMap

        self.calls, none = [], torch.zeros(0)
        monkeypatch.setattr(serve, "page_map", lambda ctx, new, free, *a: self.calls.append(("map", ctx.tolist(), new.tolist(), free.numel()))
                            or PageMap(none, ctx + new, none, none, none))
        monkeypatch.setattr(serve, "draft_tree", lambda parents, q, kv, most: self.calls.append(("tree", most)) or DraftTree(none, none)
                            if most <= 4096 else draft_tree(parents, q, kv, most))
        monkeypatch.setattr(serve, "paged_compact", lambda *a: self.calls.append(("compact",)))
        monkeypatch.setattr(serve, "paged_append", lambda *a: self.calls.append(("append",)))
        monkeypatch.setattr(serve, "paged_attention", lambda *a, **kw: self.calls.append(("attention",)))
        monkeypatch.setattr(serve, "page_release", lambda table, lens, keep, size, free, top: self.calls.append(
            ("release", lens.tolist(), keep.tolist(), top)) or (counts.pop(0) if counts else None))
        self.cache = serve.PagedCache(1, requests, 1, 64, 16, tokens, torch.float16, torch.device("cpu"))

    def state(self):
        return list(self.cache.lengths), self.cache.top, self.cache.free.tolist(), len(self.calls)


def test_a_tree_that_is_refused_changes_nothing(monkeypatch):
    s = _Steps(monkeypatch)
    s.cache.extend([30, 5])
    before = s.state()
    for trees in ([[-1] + list(range(4096)), []], [[], [-1] * 5000]):
        with pytest.raises(ValueError, match="nodes"):
            s.cache.draft(trees)
        assert s.state() == before
    for trees in ([[-1, "x"], []], [[-1, 2 ** 40], []]):  # parents that are no 32-bit numbers
        with pytest.raises((TypeError, ValueError, RuntimeError, OverflowError)):
            s.cache.draft(trees)
        assert s.state() == before
    step = s.cache.draft([[-1] + list(range(4095)), [-1]])
    assert step.nodes == [4096, 1] and s.cache.lengths == [30 + 4096, 6]


def _verdict(accepted, rows):
    from e8_lattice_vector_gb300.drafts import Verdict

    return Verdict(torch.tensor(accepted, dtype=torch.int32), torch.zeros(rows, dtype=torch.int32), None)


def test_a_step_is_kept_once_and_before_the_next_change(monkeypatch):
    """keep() counts pages from the cache's lengths, and the device from the step's: they must be the same step's."""
    def refused(c, s, step, rows):
        before = s.state()
        with pytest.raises(ValueError, match="drafted last"):
            c.keep(step, _verdict([1, 1], rows))
        with pytest.raises(ValueError, match="drafted last"):
            c.draft_step(*(torch.zeros(1, rows, 1, 64),) * 3, step)
        assert s.state() == before

    for change in ("keep", "extend", "draft", "end"):
        s = _Steps(monkeypatch)
        c = s.cache
        c.extend([30, 5])
        step = c.draft([[-1, 0, 0], [-1, 0]])
        c.draft_step(*(torch.zeros(1, 5, 1, 64),) * 3, step)  # as often as it takes
        c.draft_step(*(torch.zeros(1, 5, 1, 64),) * 3, step)
        if change == "keep":
            assert c.keep(step, _verdict([2, 1], 5)) == [2, 1] and c.lengths == [32, 6]
        elif change == "extend":
            c.extend([1, 1])
        elif change == "draft":
            newer = c.draft([[-1, 0], [-1]])
        else:
            c.end([1])
        refused(c, s, step, 5)
        if change == "draft":  # the newer one is the cache's
            assert c.keep(newer, _verdict([1, 1], 3)) == [1, 1] and c.lengths == [34, 8]
            refused(c, s, newer, 3)


def test_a_verdict_of_another_step_is_refused(monkeypatch):
    s = _Steps(monkeypatch)
    step = s.cache.draft([[-1, 0, 0], [-1, 0]])
    before = s.state()
    for accepted, rows in (([1], 5), ([1, 1, 1], 5), ([1, 1], 4), ([1, 1], 6)):
        with pytest.raises(ValueError, match="verdict is of"):
            s.cache.keep(step, _verdict(accepted, rows))
        assert s.state() == before
    assert s.cache.keep(step, _verdict([3, 2], 5)) == [3, 2] and s.cache.lengths == [3, 2]


def test_requests_that_are_not_there_cannot_end(monkeypatch):
    s = _Steps(monkeypatch, requests=3)
    s.cache.extend([30, 16, 1])
    before = s.state()
    for gone in ([3], [-1], [0, 7], range(-2, 1)):
        with pytest.raises(ValueError, match="there are 3 requests"):
            s.cache.end(gone)
        assert s.state() == before
    s.cache.end(r for r in (2, 0, 2))
    assert s.cache.lengths == [0, 16, 0]


def test_the_free_list_can_be_set(monkeypatch):
    """As an attribute: to other pages, a part of them, none; what requests hold still finds its place on it."""
    s = _Steps(monkeypatch, requests=2, tokens=160, counts=[torch.tensor(x) for x in ([1, 0], [2, 0], [5, 0])])
    c, pages = s.cache, s.cache.free.tolist()
    assert sorted(pages) == list(range(20))
    c.free = c.free.flip(0)
    assert c.free.tolist() == pages[::-1] and c.top == 0
    c.extend([33, 16])  # three pages and one
    assert c.free.tolist() == pages[::-1][4:]
    c.free = c.free[4:9]
    assert c.free.tolist() == pages[::-1][8:13] and c.top >= 4
    top = c.top
    c.extend([20, 0])  # one more
    assert c.top == top + 1 and c.free.tolist() == pages[::-1][9:13]
    c.end([1])  # a column with its page
    assert c.top == top
    c.free = c.free[:2]
    left = c.free.tolist()
    c.extend([60, 20])  # four and two more, where two are left
    assert c.free.tolist() == [] and s.calls[-1][3] == 2 and len(left) == 2
    top = c.top
    c.end([1])  # asked for two and got none or some: the device says how many came back
    assert c.top == top - 2
    c.end([0])
    assert c.top == top - 7
    c.free = torch.zeros(0, dtype=torch.int32)
    assert c.free.numel() == 0
    c.free = torch.arange(50, dtype=torch.int32)  # more than there were
    assert c.free.tolist() == list(range(50)) and c.lengths == [0, 0]


def test_verify_refuses_results_over_its_inputs(nq):
    """A request's results are written while other requests read: none may lie over any input, or over another."""
    f = nq.lib().nq_verify_drafts
    at = lambda i: 4096 * i
    good = [at(1), 100, at(2), 100, 2, 100, at(3), at(4), at(5), 4, at(6), 2, at(7), at(8), at(9), None]
    rows = 4 * (3 * 100 + 100)
    cases = [(12, 6, 0), (12, 7, 12), (12, 8, -4), (12, 10, 8), (12, 10, -4), (12, 13, 4), (12, 14, 12)]  # accepted
    cases += [(i, j, by) for i in (12, 13, 14) for j in (0, 2) for by in (0, -4, rows - 4)]  # over probabilities
    for i, j, by in cases:
        args = list(good)
        args[i] = good[j] + by
        assert f(*args) == ARG, (i, j, by)
    wide = list(good)
    wide[1], wide[13] = 2 ** 62, good[0] + 2 ** 40  # a stride beyond all memory
    assert f(*wide) == ARG


@pytest.mark.parametrize("apart", [1.0, 1e-2, 1e-4, 1e-6])
def test_what_is_left_is_off_by_a_fraction_of_the_whole(apart):
    """The verification's arithmetic (pairs of fp32, from the kernel's formulas) against fractions: after k rejections the sum of what is left
    is off by at most (k + 1) 2^-37 of the sum of p, of which the terms alone, added exactly here, take 10 (k + 1) 2^-48.  It is no such fraction of
    itself: with a draft near the model little is left, and p - A q has p's roundings."""
    from fractions import Fraction

    import numpy as np

    f, of = np.float32, lambda x: Fraction(float(x))

    def normal(s, e):
        t = f(s + e)
        return t, f(e - f(t - s))

    def add(a, b):
        t = f(a[0] + b[0])
        v = f(t - a[0])
        return normal(t, f(f(f(a[0] - f(t - v)) + f(b[0] - v)) + f(a[1] + b[1])))

    def fma(a, b, c):  # 48 bits of product and a sum in 64: a second rounding past the 53rd bit
        return (np.float64(a) * b.astype(np.float64) + c.astype(np.float64)).astype(f)

    def left(p, q, taken):
        h = taken[0] * q
        below = fma(taken[1], q, fma(taken[0], q, -h))
        d = p - h
        low = ((p - d) - h) - below
        return np.where(d + low > 0, d, f(0)), np.where(d + low > 0, low, f(0))

    rng = np.random.default_rng(3)
    x = rng.standard_normal(1000) * 2
    p, q = (np.exp(z) / np.exp(z).sum() for z in (x, x + apart * rng.standard_normal(1000)))
    p, q = p.astype(f), q.astype(f)
    P, Q = [of(v) for v in p], [of(v) for v in q]
    taken, total, A, S, worst = (f(0), f(0)), (f(1), f(0)), Fraction(0), Fraction(1), 0
    for k in range(1, 9):
        taken, A = add(taken, total), A + S
        got = sum(of(v) for part in left(p, q, taken) for v in part)
        S = sum(max(a - A * b, 0) for a, b in zip(P, Q))
        assert abs(got - S) <= Fraction(10 * (k + 1), 2 ** 48) * sum(P)
        worst = max(worst, abs(got - S) / S)
        total = normal(f(float(got)), f(float(got - of(f(float(got))))))
    assert (worst > Fraction(1, 2 ** 38)) == (apart < 1e-2)


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    import ctypes
    import os
    import subprocess

    from e8_lattice_vector_gb300 import build as nqbuild

    out = str(tmp_path_factory.mktemp("choice") / "paged_choice.so")
    subprocess.run([nqbuild._nvcc()] + nqbuild.ARCH + ["-std=c++17", "-O1", "-Xcompiler", "-fPIC", "-shared", "-I", nqbuild.INCLUDE,
                                                       os.path.join(os.path.dirname(os.path.abspath(__file__)), "paged_choice.cu"), "-o", out],
                   check=True)
    f = ctypes.CDLL(out).few_tree_tiles

    def few(requests, ctx, rows, dim=128, window=0, room=None, group=4, kv_heads=8):
        n = rows // group
        room = ctx + n if room is None else room
        return bool(f(requests * n, n, requests, group, kv_heads, dim, 16, -(-room // 16), window))

    return few


def test_short_trees_go_to_the_kernel_that_was_measured_as_faster(choice):
    """The rule's comment: requests, cached tokens, rows for each KV head; some with a window, a table with room for more, other head_dims."""
    small = [(1, 1500, 32), (1, 1500, 64), (1, 6000, 32), (4, 1500, 32), (1, 3000, 64), (4, 300, 32), (8, 300, 32)]
    large = [(16, 300, 32), (16, 150, 64), (16, 60, 64), (1, 6000, 64), (4, 1500, 48), (4, 300, 128), (32, 150, 32), (32, 60, 48)]
    assert [choice(*c) for c in small] == [True] * len(small)
    assert [choice(*c) for c in large] == [False] * len(large)
    # a window bounds the keys whatever the table has room for
    for room in (8100, 100000, 2 ** 20):
        assert choice(1, 8000, 64, window=1024, room=room) and choice(1, 8000, 32, window=4096, room=room)
        assert not choice(4, 8000, 64, window=1024, room=room) and not choice(16, 8000, 32, window=256, room=room)
    assert choice(16, 300, 32, dim=64) and choice(4, 8000, 32, dim=64, window=1024)
    assert not choice(32, 150, 64, dim=64) and not choice(1, 8000, 32, room=2 ** 20)
    assert not choice(2 ** 20, 2 ** 20, 64, room=2 ** 27) and choice(0, 10, 32)  # no sum of it wraps
