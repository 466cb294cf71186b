"""Calls on drafted trees that test_drafts_gpu leaves out: releases of columns without pages, verification of drafts that are all but
the model's and of wide stars that are rejected, trees that are plain runs, and repeated calls."""
import os
import random
import subprocess
import sys

import pytest
import torch

from test_drafts_gpu import ROWS, TreeStep, check_verify, make_tree
from test_paged_gpu import DEV, TYPES, _i32, nq  # noqa: F401  (nq is the fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- release


def ref_release_pages(table, lens, keep, P, free, top):
    """The header's words: columns without a page give nothing back."""
    free, k, cols = list(free), 0, len(table[0]) if table else 0
    for row, n, m in zip(table, lens, keep):
        for c in range(-(-max(m, 0) // P), min(-(-max(n, 0) // P), cols)):
            if row[c] < 0:
                continue
            if top - 1 - k >= 0:
                free[top - 1 - k] = row[c]
            k += 1
    return free, [k, max(k - top, 0)]


@pytest.mark.parametrize("share", [0.02, 0.5, 1.0])
@pytest.mark.parametrize("R", [1, 13, 511, 1024, 1025, 3000])
def test_release_of_columns_without_pages(nq, R, share):
    """Entries below zero are nobody's pages: they are neither counted nor put on the list, and take no page's place there."""
    rng = random.Random(R)
    for cols, most in ((1, 16), (9, 200), (300, 16 * 300)):
        if R * cols > 400000:
            continue
        lens = [rng.choice([0, 1, 16, 17, -3, rng.randrange(most), most]) for _ in range(R)]
        keep = [rng.choice([0, n, n - 1, n - 16, -1]) for n in lens]
        table = [[rng.choice([-1, -1, -2 ** 31]) if rng.random() < share else rng.randrange(10 ** 6) for _ in range(cols)] for _ in range(R)]
        total = ref_release_pages(table, lens, keep, 16, [], 0)[1][0]
        for top in (total, total + 5, max(total - 3, 0), 0):
            free = [rng.randrange(10 ** 6) for _ in range(top + 4)]
            want, counts = ref_release_pages(table, lens, keep, 16, free, top)
            dev, at = _i32(free), torch.tensor(table, dtype=torch.int32, device=DEV).view(R, cols)
            got = nq.page_release(at, _i32(lens), _i32(keep), 16, dev, top)
            assert got.tolist() == counts and dev.tolist() == want


def test_release_of_more_columns_than_a_round(nq):
    """Hundreds of thousands of columns, of many requests and of one, some without pages."""
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    for R, cols in ((700, 700), (2, 300000)):
        table = torch.randint(0, 10 ** 6, (R, cols), generator=g, device=DEV, dtype=torch.int32)
        table[torch.rand((R, cols), generator=g, device=DEV) < 0.01] = -1
        lens, keep = _i32([16 * (cols - r % 5) for r in range(R)]), _i32([0 if r % 7 else 16 * 9 for r in range(R)])
        col = torch.arange(cols, device=DEV)
        gone = table[(col >= (keep // 16)[:, None]) & (col < (lens // 16)[:, None])]
        gone = gone[gone >= 0]
        for spare in (3, -1000):
            top = gone.numel() + spare
            free = torch.full((top + 2,), -7, dtype=torch.int32, device=DEV)
            got = nq.page_release(table, lens, keep, 16, free, top)
            put = min(gone.numel(), top)
            assert got.tolist() == [gone.numel(), gone.numel() - put]
            assert torch.equal(free[top - put:top].flip(0), gone[:put])
            assert bool((free[:top - put] == -7).all()) and bool((free[top:] == -7).all())


def test_a_free_list_that_ran_out_and_a_release(nq):
    """Steps that ask for more pages than there are, and releases after them: no page is lost or handed out twice, and the list
    holds nothing but pages."""
    P, R, pages = 16, 6, 16
    rng = random.Random(5)
    free, top = torch.randperm(pages, device=DEV).to(torch.int32), 0
    table = torch.full((R, 20), -1, dtype=torch.int32, device=DEV)
    lens, ran_out = [0] * R, 0
    for step in range(60):
        new = [rng.randrange(60) if n < 200 else 0 for n in lens]
        m = nq.page_map(_i32(lens), _i32(new), free[top:], table, P, sum(new))
        taken, lacked = m.counts.tolist()[1:3]
        ran_out += lacked > 0
        top += taken - lacked
        lens = [a + b for a, b in zip(lens, new)]
        keep = [0 if rng.random() < 0.3 else rng.randrange(n + 1) for n in lens]
        released, no_room = nq.page_release(table, _i32(lens), _i32(keep), P, free, top).tolist()
        assert no_room == 0
        top -= released
        lens = keep
        held = [p for r in range(R) for p in table[r, :-(-lens[r] // P)].tolist() if p >= 0]
        assert sorted(held + free[top:].tolist()) == list(range(pages))
    assert ran_out > 5


@pytest.mark.parametrize("R", [1, 13, 512, 1500])
def test_release_that_clears_the_table(nq, R):
    """Columns whose pages went on the list become -1, all others stay (those past the columns too); a second call gives nothing back."""
    rng = random.Random(R)
    for cols, most in ((1, 16), (9, 200), (200, 16 * 200)):
        lens = [rng.choice([0, 1, 16, 17, -3, rng.randrange(most), most]) for _ in range(R)]
        keep = [rng.choice([0, n, n - 1, n - 16, -1]) for n in lens]
        table = [[-1 if rng.random() < 0.1 else rng.randrange(10 ** 6) for _ in range(cols)] for _ in range(R)]
        total = ref_release_pages(table, lens, keep, 16, [], 0)[1][0]
        for top in (total, total + 5, max(total - 3, 0)):
            free = [rng.randrange(10 ** 6) for _ in range(top + 4)]
            want, counts = ref_release_pages(table, lens, keep, 16, free, top)
            left, k = [list(row) for row in table], 0
            for row, n, m in zip(left, lens, keep):
                for c in range(-(-max(m, 0) // 16), min(-(-max(n, 0) // 16), cols)):
                    if row[c] >= 0:
                        k += 1
                        if k <= top:
                            row[c] = -1
            wide = torch.full((R, cols + 3), 5, dtype=torch.int32, device=DEV)
            wide[:, :cols] = torch.tensor(table, dtype=torch.int32, device=DEV).view(R, cols)
            dev = _i32(free)
            args = (wide[:, :cols], _i32(lens), _i32(keep), 16, dev)
            assert nq.page_release(*args, top, clear=True).tolist() == counts
            assert dev.tolist() == want and wide[:, :cols].tolist() == left and bool((wide[:, cols:] == 5).all())
            lost, put = counts[1], counts[0] - counts[1]
            assert nq.page_release(*args, top - put, clear=True).tolist() == [lost, max(lost - (top - put), 0)]
            assert dev[top - put:].tolist() == want[top - put:]


def test_a_step_past_its_room_after_a_release_that_clears(nq):
    """A request gives pages back, another gets them, and then the first one's step has more tokens than its room: kv_lens counts tokens
    whose columns were never written, and neither the attention nor the next step's append reaches the other's pages through them."""
    P, H, D, pages = 16, 2, 64, 12
    table = torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
    free, top = torch.arange(pages, dtype=torch.int32, device=DEV), 0
    Kp, Vp = (torch.randn(pages, H, P, D, device=DEV).half() for _ in range(2))
    nq.page_map(_i32([0, 0]), _i32([80, 0]), free[top:], table, P, 80)
    top += 5
    top -= int(nq.page_release(table, _i32([80, 0]), _i32([20, 0]), P, free, top, clear=True)[0])
    nq.page_map(_i32([20, 0]), _i32([0, 70]), free[top:], table, P, 70)  # the other request takes them
    top += 5
    others = table[1, :5].tolist()
    assert set(others) & {0, 1, 2, 3, 4}
    m = nq.page_map(_i32([20, 70]), _i32([50, 0]), free[top:], table, P, 3)  # room for three of fifty
    assert m.counts.tolist()[0] == 50 and m.kv_lens.tolist() == [70, 70]
    assert not set(table[0].tolist()) & set(others)
    Q = torch.randn(3, 4, D, device=DEV).half()
    saw = []
    for value in (1.0, 500.0):
        Kp[others], Vp[others] = value, value
        saw.append(nq.paged_attention(Q, Kp, Vp, table, m.q_start, m.kv_lens, max_q=3, causal=False))
    assert torch.equal(*saw)
    m = nq.page_map(m.kv_lens, _i32([1, 0]), free[top:], table, P, 1)
    nq.paged_append(*(torch.randn(1, H, D, device=DEV).half() for _ in range(2)), Kp, Vp, m.slots)
    assert m.slots.tolist() == [-1] and bool((Kp[others] == 500).all()) and bool((Vp[others] == 500).all())


def test_a_paged_cache_that_runs_out_of_pages(nq):
    """With fewer free pages than its requests may ask for: lengths go on, columns go without, and all pages are there in the end."""
    from e8_lattice_vector_gb300.serve import PagedCache

    cache = PagedCache(1, 3, 2, 64, 16, 160, torch.float16, torch.device(DEV, 0))
    some = cache.free[:9].clone()
    cache.free = some
    m = cache.extend([40, 20, 10])  # 3 + 2 + 1
    assert bool((m.slots >= 0).all()) and cache.free.tolist() == some[6:].tolist()
    m = cache.extend([100, 1, 30])  # 6 + 0 + 2 of 3
    assert m.counts.tolist() == [131, 8, 5, 0] and cache.free.numel() == 0
    assert int((m.slots >= 0).sum()) == 8 + 48 + 1 + 6  # the rest of begun pages, and three new ones
    cache.end([1, 2])
    assert sorted(cache.free.tolist()) == sorted(some[3:6].tolist())
    cache.extend([0, 33, 0])
    assert cache.free.numel() == 0
    cache.end([0, 1])
    assert sorted(cache.free.tolist()) == sorted(some.tolist()) and cache.lengths == [0, 0, 0]


# -------------------------------------------------------------- verification


@pytest.mark.parametrize("apart", [1e-1, 1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("V", [3000, 32000, 128256])
def test_verify_drafts_near_the_model(nq, V, apart):
    """Drafts all but the model's, the first of them rejected: what is left is as small as the difference, and the later ones are accepted or
    not by it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(V)
    kept = tried = 0
    for shape in ("star", "star", "wide", "random"):
        n = 14
        x = torch.randn(n, V, generator=g, device=DEV) * 2
        probs = torch.softmax(x, 1)
        draft = torch.softmax(x + apart * torch.randn(n, V, generator=g, device=DEV), 1)
        tree = make_tree(shape, n, 1)
        ids = torch.multinomial(draft[[max(p, 0) for p in tree]], 1, generator=g).squeeze(1).to(torch.int32)
        ids[1] = int((probs[0] / draft[0]).argmin())  # the least of p / q
        u = torch.rand(n, generator=g, device=DEV)
        u[1] = 1 - 2.0 ** -24
        kept += check_verify(nq, [tree], V, torch.float32, True, probs=probs, draft=draft, ids=ids, u=u)
        tried += 1
    assert kept > tried  # some draft is accepted after a rejection


@pytest.mark.parametrize("dtype", ROWS)
@pytest.mark.parametrize("V", [50, 1003, 32000])
@pytest.mark.parametrize("n", [66, 67, 301])
def test_verify_wide_stars_that_are_rejected(nq, dtype, V, n):
    """More chosen drafts than a warp keeps of its part, all rejected: over a few tokens, with repeated ones, at the row's beginning, among
    its 16-byte pieces and at its end, rows that begin on any boundary."""
    rng = random.Random(n * V)
    g = torch.Generator(device=DEV)
    g.manual_seed(n + V)
    for places in ((0, V), (0, min(V, 40)), (max(V - 40, 0), V), (V // 2 - 20, V // 2 + 20)):
        some = [rng.randrange(*places) for _ in range(n if V > 1003 else 30)]
        ids = [0] + [rng.choice(some) for _ in range(n - 1)]
        probs = torch.rand(n, V, generator=g, device=DEV) + 0.1
        probs[:, sorted(set(ids[1:]))] *= 1e-3  # little on the drafted tokens
        probs = (probs / probs.sum(1, keepdim=True)).to(dtype)
        for u0 in (0.0, 0.3, 0.9999) if V < 32000 else (0.6,):
            u = torch.full((n,), 0.9999, device=DEV)
            u[0] = u0
            for stride in (None, V + 5):
                kept = check_verify(nq, [make_tree("star", n)], V, dtype, False, probs=probs, draft=None, ids=_i32(ids), u=u, stride=stride)
                assert kept == 1  # the root alone


@pytest.mark.parametrize("V", [40, 2000])
def test_verify_wide_stars_that_leave_nothing(nq, V):
    """All mass on drafted tokens whose own numbers reject them: nothing is left, and the node's own probabilities decide."""
    n = 300
    rng = random.Random(V)
    ids = [0] + [rng.randrange(30) for _ in range(n - 1)]
    probs = torch.zeros(n, V, device=DEV)
    probs[:, sorted(set(ids[1:]))] = 1.0 / 32
    for u0 in (0.0, 0.5, 0.97):
        u = torch.full((n,), 1.0, device=DEV)
        u[0] = u0
        assert check_verify(nq, [make_tree("star", n), [-1, 0]], V, torch.float32, False, probs=torch.cat([probs, probs[:2]]), draft=None,
                            ids=_i32(ids + [0, 1]), u=torch.cat([u, u[:2]])) == 2


def test_verify_repeats_bit_for_bit(nq):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    n, V = 12, 70001
    probs = torch.softmax(torch.randn(20 * n, V, generator=g, device=DEV) * 2, 1)
    draft = torch.softmax(torch.randn(20 * n, V, generator=g, device=DEV), 1) / 3 + probs * (2 / 3)
    ids = torch.multinomial(draft, 1, generator=g).squeeze(1).to(torch.int32)
    args = (probs, ids, _i32(make_tree("wide", n) * 20), _i32(list(range(0, 20 * n + 1, n))), torch.rand(20 * n, generator=g, device=DEV), draft)
    want = nq.verify_drafts(*args)
    for _ in range(5):
        got = nq.verify_drafts(*args)
        assert all(torch.equal(a, b) for a, b in ((got.accepted, want.accepted), (got.path, want.path), (got.tokens, want.tokens)))


# ----------------------------------------------------------------- attention


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,D", [(3, 128), (14, 64), (40, 64), (40, 96), (40, 128), (100, 64), (100, 128)])
def test_tree_attention_repeats_bit_for_bit(nq, n, D, dtype):
    s = TreeStep([(5000, make_tree("wide", n)), (100, make_tree("random", n)), (2500, make_tree("chain", n))], 8, 2, D, 16, dtype, seed=n)
    first = s.check(nq)
    ws = nq.paged_attention_workspace(s.Q, s.Kp, s.table, max_q=s.max_q)
    ws.fill_(255)  # NaN everywhere: nothing in the scratch has to start at zero
    for _ in range(3):
        assert torch.equal(first, s.call(nq, ws=ws))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("n", [1, 2, 4])
def test_a_short_chain_is_a_causal_run_bit_for_bit(nq, n, D, dtype):
    """Up to 16 rows for each KV head go to the small kernel with a tree and without: the same sums in the same order."""
    s = TreeStep([(500, make_tree("chain", n)), (3000, make_tree("chain", n)), (0, make_tree("chain", n))], 8, 2, D, 16, dtype, seed=n)
    plain = nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=n)
    assert torch.equal(s.call(nq), plain)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("n", [33, 130])
def test_a_long_chain_is_a_causal_run_bit_for_bit(nq, n, D, dtype):
    """In the large kernel, too: rows of one half and of two, and at head_dim 64 three score buffers against two."""
    s = TreeStep([(500, make_tree("chain", n)), (3000, make_tree("chain", n)), (0, make_tree("chain", n))], 8, 2, D, 16, dtype, seed=n)
    plain = nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=n)
    assert torch.equal(s.call(nq), plain)


@pytest.mark.parametrize("n", [4, 40])
def test_the_rows_of_a_star_are_single_tokens(nq, n):
    """Without a cached token a star's row sees its root and itself: the call over those two keys alone, within both bounds."""
    s = TreeStep([(0, make_tree("star", n))], 8, 2, 128, 16, torch.float16, seed=n)
    got, tol = s.check(nq), s.reference(128 ** -0.5)[2]
    k, v = s.k[0], s.v[0]
    for i in range(n):
        Kp, Vp = (torch.zeros(1, 2, 16, 128, dtype=torch.float16, device=DEV) for _ in range(2))
        for slot, j in enumerate((0, i) if i else (0,)):
            Kp[0, :, slot], Vp[0, :, slot] = k[j], v[j]
        one = nq.paged_attention(s.Q[i:i + 1], Kp, Vp, _i32([[0]]), _i32([0, 1]), _i32([2 if i else 1]))
        assert bool(((one[0].double() - got[i].double()).abs() <= 2 * tol[i]).all())


def test_steps_in_a_row_from_one_graph(nq):
    """Everything of a step but the map and the release in one graph, these two around it with the free list's place as it moves: the
    same tokens, lengths and kept rows as steps that are called one by one."""
    R, n, P, H, D, V, L = 3, 9, 16, 2, 64, 200, 2
    T, cols, pages = R * n, 10, 30
    dev = torch.device(DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    q, k, v = (torch.zeros(L, T, h, D, dtype=torch.float16, device=dev) for h in (4, H, H))
    probs, draft, u = torch.zeros(T, V, device=dev), torch.zeros(T, V, device=dev), torch.zeros(T, device=dev)
    ids, parents = torch.zeros(T, dtype=torch.int32, device=dev), _i32(make_tree("wide", n) * R)

    class Side:
        def __init__(self):
            self.pools = [torch.zeros(L, pages, H, P, D, dtype=torch.float16, device=dev) for _ in range(2)]
            self.table = torch.full((R, cols), -1, dtype=torch.int32, device=dev)
            self.free, self.top, self.lens = torch.arange(pages, dtype=torch.int32, device=dev), 0, [0] * R
            self.m, self.out = nq.PageMap.empty(R, T, dev), torch.zeros_like(q)
            self.tree, self.verdict = nq.DraftTree.empty(T, n, dev), nq.Verdict.empty(R, T, dev)

        def map(self):
            nq.page_map(_i32(self.lens), _i32([n] * R), self.free[self.top:], self.table, P, T, out=self.m)
            self.top += int(self.m.counts[1])

        def middle(self):
            m = self.m
            nq.draft_tree(parents, m.q_start, m.kv_lens, n, out=self.tree)
            for l in range(L):
                nq.paged_append(k[l], v[l], self.pools[0][l], self.pools[1][l], m.slots)
                nq.paged_attention(q[l], self.pools[0][l], self.pools[1][l], self.table, m.q_start, m.kv_lens, max_q=n, tree=self.tree,
                                   out=self.out[l])
            nq.verify_drafts(probs, ids, parents, m.q_start, u, draft_probs=draft, out=self.verdict)
            nq.paged_compact(*self.pools, self.table, m.q_start, m.kv_lens, self.verdict.path)

        def release(self):
            keep = [a + b for a, b in zip(self.lens, self.verdict.accepted.tolist())]
            counts = nq.page_release(self.table, self.m.kv_lens, _i32(keep), P, self.free, self.top)
            self.top -= int(counts[0] - counts[1])
            self.lens = keep

    one, other, warm = Side(), Side(), Side()
    warm.map()
    warm.middle()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.middle()
    tops = set()
    for step in range(12):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device=dev).half())
        probs.copy_(torch.softmax(torch.randn(T, V, generator=g, device=dev) * 2, 1))
        draft.copy_(torch.softmax(probs.log() + 0.3 * torch.randn(T, V, generator=g, device=dev), 1))
        source = torch.tensor([r * n + max(p, 0) for r in range(R) for p in make_tree("wide", n)], device=dev)
        ids.copy_(torch.multinomial(draft[source], 1, generator=g).squeeze(1))
        u.copy_(torch.rand(T, generator=g, device=dev))
        one.map()
        one.middle()
        one.release()
        other.map()
        graph.replay()
        other.release()
        tops.add(other.top)
        assert one.lens == other.lens and one.top == other.top
        assert torch.equal(one.out, other.out) and torch.equal(one.table, other.table) and torch.equal(one.free[one.top:], other.free[other.top:])
        assert torch.equal(one.verdict.tokens, other.verdict.tokens) and torch.equal(one.verdict.path, other.verdict.path)
        assert all(torch.equal(a, b) for a, b in zip(one.pools, other.pools))
    assert len(tops) > 1


def test_a_first_call_may_be_a_captured_one():
    """Release and verification of a new process, whose first calls (of the largest cluster, too) are made while a graph is captured."""
    code = """
import torch, e8_lattice_vector_gb300 as nq
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
R, cols = 600, 500
table = torch.arange(R * cols, dtype=torch.int32, device="cuda").view(R, cols)
lens, keep, free, counts = i32([16 * cols] * R), i32([0] * R), torch.full((R * cols,), -1, dtype=torch.int32, device="cuda"), i32([0, 0])
probs, ids, parents, starts, u = torch.full((3, 9000), 1 / 9000, device="cuda"), i32([0, 5, 6]), i32([-1, 0, 1]), i32([0, 3]), torch.zeros(3, device="cuda")
v = nq.Verdict.empty(1, 3)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    nq.page_release(table, lens, keep, 16, free, R * cols, out=counts)
    nq.verify_drafts(probs, ids, parents, starts, u, out=v)
assert counts.tolist() == [0, 0]
graph.replay()
torch.cuda.synchronize()
assert counts.tolist() == [R * cols, 0] and torch.equal(free.flip(0), table.view(-1)) and v.tokens.tolist() == [5, 6, 0]
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
