"""Drafted trees over the paged cache against plain implementations: the map, the verification, the compaction and the release
value by value, the attention against its definition in 64 bits.

Attention tolerances are bounds, computed per element from the 64-bit reference.  With u half a step of the pool's type (2^-11
fp16, 2^-8 bf16), w that of the weights (2^-11; 2^-17 in bf16, where they are the sum of two), e = 2^-24, n keys and
A = sum p |v| / l:
  a score is off by at most  S = (D + 4) e scale max_j sum_d |q_d k_jd|  (exact products, D additions, the scaling),
  each p by a factor 1 +- (S + 4 e) and its rounding w (fp16 weights below the normal range by 2^-32 of the largest), the
  sums of n terms by (n + 8) e each, above and below the fraction, the output by u or 2^-25 in fp16's subnormals.
  |out - exact| <= u |exact| + 2^-25 + A (w + 2 S + 2 (n + 8) e) (1 + u) + 2^-32 sum |v| / l
  |lse - exact| <= S + (n + 8) e + 4 e |exact|
"""
import random

import numpy as np
import pytest
import torch

from test_paged_gpu import DEV, E32, TYPES, Step, _i32, _pool, nq  # noqa: F401  (nq is the fixture)

pytestmark = pytest.mark.gpu

TREES = ["chain", "star", "wide", "random", "forest"]


def make_tree(shape, n, seed=0):
    rng = random.Random(seed * 1000 + n)
    parents = []
    for i in range(n):
        if i == 0:
            parents.append(-1)
        elif shape == "chain":
            parents.append(i - 1)
        elif shape == "star":
            parents.append(0)
        elif shape == "wide":
            parents.append((i - 1) // 3)
        elif shape == "random":
            parents.append(rng.randrange(i))
        else:
            parents.append(rng.choice([-1, rng.randrange(i), i - 1]))
    return parents


def ways(parents):
    """Per node: itself and its ancestors, nearest first.  A number that is not below the node's own is no parent."""
    got = []
    for i, p in enumerate(parents):
        got.append([i] + (got[p] if 0 <= p < i else []))
    return got


def bits_of(way, words):
    x = sum(1 << j for j in way if j < 64 * words)
    row = [(x >> (64 * k)) & (2 ** 64 - 1) for k in range(words)]
    return [v - 2 ** 64 if v >= 2 ** 63 else v for v in row]


# --------------------------------------------------------------- the tree's map


def check_draft_tree(nq, trees, ctx, window=0, max_q=None, pad=0, seed=0):
    lens = [len(t) for t in trees]
    T = sum(lens) + pad
    max_q = max(lens + [0]) if max_q is None else max_q
    words = max(-(-max_q // 64), 1)
    want_bits, want_pos = [], []
    for c, parents in zip(ctx, trees):
        for way in ways(parents):
            want_bits.append(bits_of(way[:window] if window else way, words))
            want_pos.append(c + len(way) - 1)
    out = nq.DraftTree(torch.full((T, words), 77, dtype=torch.int64, device=DEV),
                       torch.full((T,), 77, dtype=torch.int32, device=DEV))
    q_start = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    kv = _i32([c + n for c, n in zip(ctx, lens)])
    parents = _i32([p for t in trees for p in t] + [3] * pad)
    t = nq.draft_tree(parents, q_start, kv, max_q, window=window, out=out)
    assert t is out
    live = T - pad
    assert t.ancestors[:live].tolist() == want_bits
    assert t.positions[:live].tolist() == want_pos
    assert bool((t.ancestors[live:] == 77).all()) and bool((t.positions[live:] == 77).all())


@pytest.mark.parametrize("shape", TREES)
@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 200])
@pytest.mark.parametrize("window", [0, 1, 3, 1000])
def test_draft_tree(nq, shape, n, window):
    trees = [make_tree(shape, m, s) for s, m in enumerate((n, 0, 1, (n + 1) // 2, n))]
    check_draft_tree(nq, trees, [5, 9, 0, 1000, 77], window, pad=3)


def test_draft_tree_of_any_size(nq):
    check_draft_tree(nq, [make_tree("chain", 2049), make_tree("wide", 4096), make_tree("random", 2048)], [1, 2, 3])
    check_draft_tree(nq, [make_tree("wide", 17, s) for s in range(700)], list(range(700)))
    check_draft_tree(nq, [], [], pad=2)
    check_draft_tree(nq, [[], []], [4, 0])


def test_draft_tree_parents_that_are_none(nq):
    """Numbers at or past the node's own, and negative ones, are no parents."""
    check_draft_tree(nq, [[0, 5, 2, 2, 3, -7, 2 ** 31 - 1, 6, -2 ** 31]], [10])


def test_draft_tree_more_rows_than_the_bound(nq):
    """Bits that the words have no room for are left out; positions count all ancestors."""
    check_draft_tree(nq, [make_tree("chain", 150), make_tree("wide", 150)], [0, 8], max_q=60)
    check_draft_tree(nq, [make_tree("chain", 3000)], [0], max_q=100)


def test_draft_tree_device_data_is_clamped(nq):
    """Row starts and lengths outside their ranges reach nothing outside the buffers."""
    guard = torch.full((30, 1), 77, dtype=torch.int64, device=DEV)
    pos = torch.full((30,), 77, dtype=torch.int32, device=DEV)
    parents = _i32([-1] + list(range(9)))
    starts = _i32([-5, 4, 2, 2 ** 31 - 1])
    nq.draft_tree(parents, starts, _i32([6, -3, 2 ** 31 - 1]), 10, out=nq.DraftTree(guard[10:20], pos[10:20]))
    assert bool((guard[:10] == 77).all()) and bool((guard[20:] == 77).all())
    assert bool((pos[:10] == 77).all()) and bool((pos[20:] == 77).all())
    # request 0 has rows 0 .. 4 (its start is clamped), request 2 rows 2 .. 10, whose parents are numbers of its own
    assert pos[10:12].tolist() == [2, 3]


# ----------------------------------------------------------------- attention


class TreeStep(Step):
    """A step whose rows are drafted trees."""

    def __init__(self, requests, heads, kv_heads, D, P, dtype, window=0, max_q=None, **kw):
        self.trees = [t for _, t in requests]
        super().__init__([(c, len(t)) for c, t in requests], heads, kv_heads, D, P, dtype, **kw)
        self.window = window
        self.words = max(-(-(self.max_q if max_q is None else max_q) // 64), 1)
        rows, pos = [], []
        for c, t in requests:
            for way in ways(t):
                rows.append(bits_of(way[:window] if window else way, self.words))
                pos.append(c + len(way) - 1)
        self.bits = torch.tensor(rows, dtype=torch.int64, device=DEV).view(-1, self.words)
        self.pos = _i32(pos)

    def seen(self, r, L):
        """[nodes, L]: what the definition says, from the bits."""
        c, n = self.lens[r]
        t0 = sum(m for _, m in self.lens[:r])
        see = torch.zeros(n, L, dtype=torch.bool)
        bits, pos = self.bits[t0:t0 + n].tolist(), self.pos[t0:t0 + n].tolist()
        base = min(c + n, self.cols * self.P) - n  # a length that the table cuts moves the rows
        for i in range(n):
            p = min(max(pos[i], base), base + i)
            lo = max(0, p - self.window + 1) if self.window else 0
            see[i, lo:max(base, 0)] = True
            for j in range(i + 1):
                if j < 64 * self.words and (bits[i][j >> 6] >> (j & 63)) & 1 and 0 <= base + j < L:
                    see[i, base + j] = True
        for hr, hc in self.hidden:
            if hr == r:
                see[:, hc * self.P:(hc + 1) * self.P] = False
        return see.to(DEV)

    def reference(self, scale):
        T, H, D, G = self.tokens, self.heads, self.D, self.heads // self.kv_heads
        half = self.dtype == torch.float16
        u, w = (2.0 ** -11, 2.0 ** -11) if half else (2.0 ** -8, 2.0 ** -17)
        out, tol = (torch.zeros(T, H, D, dtype=torch.float64, device=DEV) for _ in range(2))
        lse = torch.full((T, H), -float("inf"), dtype=torch.float64, device=DEV)
        tol_lse = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        t0 = 0
        for r, (c, n) in enumerate(self.lens):
            L = min(c + n, self.cols * self.P)
            rows = slice(t0, t0 + n)
            t0 += n
            if n == 0 or L == 0:
                continue
            seen = self.seen(r, L)[:, None]
            k = self.k[r][:L].double().repeat_interleave(G, 1)
            v = self.v[r][:L].double().repeat_interleave(G, 1)
            q = self.Q[rows].double()
            s = (torch.einsum("thd,jhd->thj", q, k) * scale).masked_fill(~seen, -float("inf"))
            mag = (torch.einsum("thd,jhd->thj", q.abs(), k.abs()) * scale).masked_fill(~seen, 0.0)
            m = s.amax(-1, keepdim=True)
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            some = l > 0
            weight = torch.where(some, p / l, torch.zeros_like(p))
            A = torch.einsum("thj,jhd->thd", weight, v.abs())
            S, cnt = (D + 4) * E32 * mag.amax(-1, keepdim=True), (L + 8) * E32
            out[rows] = torch.einsum("thj,jhd->thd", weight, v)
            tol[rows] = u * out[rows].abs() + 2.0 ** -25 + A * (w + 2 * S + 2 * cnt) * (1 + u)
            if half:
                sv = torch.einsum("thj,jhd->thd", seen.expand_as(weight).double(), v.abs())
                tol[rows] += torch.where(some, 2.0 ** -32 * sv / l.clamp(min=1e-30), torch.zeros_like(sv))
            ls = m + torch.log(l)
            lse[rows] = ls.squeeze(-1)
            tol_lse[rows] = (S + cnt + 4 * E32 * torch.where(some, ls, torch.zeros_like(ls)).abs()).squeeze(-1)
        return out, lse, tol, tol_lse

    def call(self, nq, **kw):
        kw.setdefault("max_q", self.max_q)
        return nq.paged_attention(self.Q, self.Kp, self.Vp, self.table, self.q_start, self.kv_lens, window=self.window,
                                  tree=nq.DraftTree(self.bits, self.pos), **kw)

    def check(self, nq, scale=None, with_lse=True, **kw):
        lse = torch.full((self.tokens, self.heads), 7.0, device=DEV) if with_lse else None
        got = self.call(nq, scale=scale, lse=lse, **kw)
        o = got[0] if with_lse else got
        ref, ref_lse, tol, tol_lse = self.reference(self.D ** -0.5 if scale is None else scale)
        assert bool(torch.isfinite(o).all()), "an output is not finite"
        err = (o.double() - ref).abs()
        assert bool((err <= tol).all()), "out: worst error / tolerance %.3g" % float((err / tol).max())
        if with_lse:
            none = torch.isinf(ref_lse)
            assert torch.equal(torch.isinf(lse), none) and bool((lse[none] < 0).all())
            err = (lse.double() - ref_lse).abs()[~none]
            assert bool((err <= tol_lse[~none]).all()), "lse: worst error / tolerance %.3g" % float((err / tol_lse[~none]).max())
        return o


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n", [1, 4, 7, 40, 150])
def test_tree_types_dims_pages(nq, dtype, D, P, n):
    """Contexts that end inside a page, at its end and after it, none and one token among them; trees of every kind."""
    reqs = [(c, make_tree(TREES[i % 5], n, i)) for i, c in enumerate((0, 1, P - 1, P, 3 * P + 5, 700))]
    TreeStep(reqs, 8, 2, D, P, dtype, seed=P + n).check(nq)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (3, 1), (10, 2), (7, 1), (16, 2), (24, 1), (40, 8), (96, 2), (130, 1)])
@pytest.mark.parametrize("n", [2, 5, 20, 70])
def test_tree_head_groups(nq, dtype, heads, kv_heads, n):
    TreeStep([(333, make_tree("wide", n)), (64, make_tree("chain", 1)), (0, make_tree("random", n))], heads, kv_heads, 128, 16, dtype,
             seed=heads).check(nq)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "slice", "packed"])
@pytest.mark.parametrize("q_layout", ["plain", "fused", "head_major"])
@pytest.mark.parametrize("n", [3, 40])
def test_tree_strides(nq, layout, q_layout, n):
    s = TreeStep([(100, make_tree("wide", n)), (517, make_tree("random", n))], 6, 2, 96, 32, torch.float16, layout=layout, seed=3,
                 q_layout=q_layout)
    wide = torch.full((s.tokens, 3, s.heads, s.D), 5.0, dtype=torch.float16, device=DEV)
    s.check(nq, out=wide[:, 1])
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 2] == 5).all())


@pytest.mark.parametrize("window", [1, 2, 15, 64, 130, 1000])
@pytest.mark.parametrize("n", [1, 6, 50, 200])
def test_tree_windows(nq, window, n):
    """A row's window counts from its position, which in a tree is before its place in the row order."""
    reqs = [(c, make_tree(s, n, c)) for c, s in ((0, "wide"), (900, "random"), (129, "chain"), (128, "star"), (1500, "wide"))]
    TreeStep(reqs, 4, 2, 64, 16, torch.bfloat16, window=window, seed=window).check(nq)


@pytest.mark.parametrize("n", [5, 16, 33, 64, 130])
def test_a_chain_is_a_causal_run(nq, n):
    """A tree without branches is what the call without a tree computes, bit by bit where the same kernel takes it; a star's rows are
    single tokens that see the root."""
    s = TreeStep([(500, make_tree("chain", n)), (3000, make_tree("chain", n))], 8, 2, 128, 16, torch.bfloat16, seed=n)
    s.check(nq)
    plain = nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=n)
    tree = s.call(nq)
    # both are within the bound of the exact result
    tol = s.reference(128 ** -0.5)[2]
    assert bool(((plain.double() - tree.double()).abs() <= 2 * tol).all())


@pytest.mark.parametrize("max_q", ["exact", None, 0, 1, 10 ** 6])
def test_tree_bound_on_rows_changes_no_result(nq, max_q):
    s = TreeStep([(500, make_tree("star", 1)), (30, make_tree("wide", 90)), (0, make_tree("random", 17)), (77, []),
                  (1200, make_tree("chain", 4))], 8, 2, 128, 16, torch.float16, seed=5)
    s.check(nq, **({} if max_q == "exact" else {"max_q": max_q}))


@pytest.mark.parametrize("n", [1, 30])
def test_tree_requests_without_rows_or_keys(nq, n):
    TreeStep([(0, []), (10, []), (0, make_tree("wide", n)), (40, []), (0, []), (5, make_tree("star", n)), (0, [])], 4, 1, 64, 16,
             torch.float16).check(nq)
    s = TreeStep([(10, []), (0, [])], 4, 1, 64, 16, torch.float16)
    assert s.check(nq).shape[0] == 0


@pytest.mark.parametrize("n", [3, 9, 140])
def test_tree_rows_that_see_nothing(nq, n):
    """Rows without bits and without cached tokens, pages outside the pool, bits that name nodes behind the row or past the
    words, and lengths below the row count."""
    s = TreeStep([(0, make_tree("wide", n)), (64, make_tree("wide", n)), (300, make_tree("random", n)), (16, make_tree("star", n))], 8, 2, 128, 16,
                 torch.float16, seed=n, holes=[(1, c) for c in range((64 + n + 15) // 16)] + [(2, 0), (2, 7), (2, 18), (3, 1)])
    s.bits[0:n:2] = 0
    s.bits[n // 2] = -1  # every bit: those up to the row's own count
    s.bits[3 * n + n // 2] = -1
    s.check(nq)
    s = TreeStep([(0, make_tree("chain", n + 20)), (0, make_tree("chain", n + 20))], 8, 2, 128, 16, torch.bfloat16, seed=n)
    s.kv_lens = _i32([n + 5, 0])
    lse = torch.empty(s.tokens, 8, device=DEV)
    o, _ = s.call(nq, lse=lse)
    m = n + 20
    assert bool((o[:15] == 0).all()) and bool((o[m:] == 0).all())
    assert bool((lse[:15] == -float("inf")).all()) and bool((lse[m:] == -float("inf")).all())
    assert torch.equal(o[15], s.v[0][0].repeat_interleave(4, 0))  # node 15 stands at position 0 and sees itself


@pytest.mark.parametrize("n", [2, 33, 100])
def test_tree_lengths_past_the_table(nq, n):
    s = TreeStep([(400, make_tree("wide", n)), (100, make_tree("random", n))], 4, 2, 64, 16, torch.float16, cols=20)
    s.check(nq)


@pytest.mark.parametrize("n", [40, 100])
def test_tree_bits_past_the_words(nq, n):
    """More rows than the words have bits for: those nodes are seen by nobody, themselves included."""
    TreeStep([(200, make_tree("wide", n + 60)), (31, make_tree("chain", n))], 4, 2, 64, 16, torch.float16, max_q=64).check(nq)


@pytest.mark.parametrize("n", [2, 60])
def test_tree_wild_positions_are_clamped(nq, n):
    s = TreeStep([(300, make_tree("wide", n)), (31, make_tree("chain", n))], 4, 2, 64, 16, torch.float16, window=50)
    s.pos[0], s.pos[n - 1], s.pos[n] = -2 ** 31, 2 ** 31 - 1, 0
    s.check(nq)


def test_tree_wild_rows_and_lengths(nq):
    """Row starts and lengths outside their ranges reach nothing outside the buffers."""
    for n in (3, 90):
        s = TreeStep([(100, make_tree("wide", n)), (50, make_tree("wide", n))], 8, 2, 128, 16, torch.float16)
        out = torch.full((s.tokens + 8, 8, 128), 7.0, dtype=torch.float16, device=DEV)
        for starts, lens in (([-9, n, 2 ** 31 - 1], [2 ** 31 - 1, -5]), ([2 * n, 0, n], [-1, 60]), ([0, 0, 0], [1, 1])):
            nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, _i32(starts), _i32(lens), max_q=n, tree=nq.DraftTree(s.bits, s.pos),
                               out=out[4:-4], window=9)
            assert bool((out[:4] == 7).all()) and bool((out[-4:] == 7).all())
        nq.paged_status()


def test_tree_long_contexts_split_over_blocks(nq):
    for n, heads in ((3, 8), (8, 32), (24, 32), (64, 32)):
        s = TreeStep([(30011, make_tree("wide", n)), (77, make_tree("random", n))], heads, 8, 128, 64, torch.float16, seed=n)
        s.check(nq)
        nq.paged_status()


def test_tree_in_a_graph_and_on_a_stream(nq):
    """Captured once, replayed with other lengths, trees and rows; two graphs share a scratch buffer."""
    side = torch.cuda.Stream()
    for n in (4, 50):
        a = TreeStep([(500, make_tree("wide", n)), (90, make_tree("random", n))], 8, 2, 128, 16, torch.float16, seed=1)
        b = TreeStep([(500, make_tree("random", n, 7)), (60, make_tree("chain", n))], 8, 2, 128, 16, torch.float16, seed=1)
        ws = nq.paged_attention_workspace(a.Q, a.Kp, a.table, max_q=n)
        outs, graphs = [], []
        tree = nq.DraftTree(a.bits.clone(), a.pos.clone())
        lens = a.kv_lens.clone()
        for _ in range(2):
            out = torch.empty_like(a.Q)
            with torch.cuda.stream(side):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    nq.paged_attention(a.Q, a.Kp, a.Vp, a.table, a.q_start, lens, max_q=n, tree=tree, out=out, ws=ws)
            graphs.append(g)
            outs.append(out)
        torch.cuda.synchronize()
        for bits, pos, kv in ((a.bits, a.pos, a.kv_lens), (b.bits, b.pos, b.kv_lens), (a.bits, a.pos, a.kv_lens)):
            tree.ancestors.copy_(bits), tree.positions.copy_(pos), lens.copy_(kv)
            want = nq.paged_attention(a.Q, a.Kp, a.Vp, a.table, a.q_start, kv, max_q=n, tree=nq.DraftTree(bits, pos))
            torch.cuda.synchronize()
            for g, out in zip(graphs, outs):
                out.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, want)


@pytest.mark.parametrize("n", [3, 40])
def test_tree_pools_past_32_bits(nq, n):
    """Pages at the far end of pools with more than 2^31 elements."""
    heads, P, D = 8, 256, 128
    pages = 2 ** 31 // (heads * P * D) + 8
    s = TreeStep([(700, make_tree("wide", n)), (90, make_tree("random", n))], 16, heads, D, P, torch.float16, seed=n)
    want = s.check(nq)
    held = s.Kp.shape[0]
    big = [torch.empty(pages, heads, P, D, dtype=torch.float16, device=DEV) for _ in range(2)]
    big[0][-held:], big[1][-held:] = s.Kp, s.Vp
    s.Kp, s.Vp = big
    s.table = torch.where((s.table >= 0) & (s.table < held), s.table + (pages - held), torch.full_like(s.table, -1))
    assert torch.equal(s.check(nq), want)


def test_tree_calls_at_once_on_two_streams(nq):
    """Calls of both kernels on two streams, each with its own scratch and outputs."""
    steps = [TreeStep([(c, make_tree("wide", n, c)) for c in (3000, 500, 90)], 8, 2, D, 16, torch.bfloat16, seed=n)
             for n, D in ((4, 128), (40, 128), (40, 64), (90, 64))]
    want = [s.call(nq) for s in steps]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in enumerate(steps):
            with torch.cuda.stream(streams[i % 2]):
                got.append((i, s.call(nq)))
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, want[i])
    nq.paged_status()


# -------------------------------------------------------------- verification


def ref_verify(probs, draft, ids, parents, u):
    """One request in 64 bits, from the header's words: (path, tokens)."""
    p = np.nan_to_num(probs.astype(np.float64), nan=0.0, posinf=np.inf).clip(0)
    q = None if draft is None else np.nan_to_num(draft.astype(np.float64), nan=0.0).clip(0)
    n, V = p.shape
    if n == 0:
        return [], []
    path, said, cur, w, S = [0], [], 0, p[0].copy(), 1.0
    for i in range(1, n):
        x = int(ids[i])
        if parents[i] != cur or not 0 <= x < V:
            continue
        qx = 1.0 if q is None else q[cur, x]
        if float(u[i]) * (S * qx) < w[x]:
            path.append(i)
            said.append(x)
            cur, w, S = i, p[i].copy(), 1.0
        elif q is None:
            S -= w[x]
            w[x] = 0.0
        else:
            w = np.maximum(w - S * q[cur], 0.0)
            S = w.sum()
    if not w.sum() > 0:
        w = p[cur]
    if not w.sum() > 0:
        said.append(-1)
    else:
        c = np.cumsum(w)
        above = np.nonzero(c > float(u[0]) * c[-1])[0]
        said.append(int(above[0]) if len(above) else int(np.nonzero(w > 0)[0][-1]))
    return path, said


def check_verify(nq, trees, V, dtype, sampled, seed=0, pad=0, probs=None, draft=None, ids=None, u=None, stride=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lens = [len(t) for t in trees]
    T = sum(lens) + pad
    if probs is None:
        x = torch.randn(T, V, generator=g, device=DEV) * 2
        x += 6 * (torch.rand(T, V, generator=g, device=DEV) < 3 / V)
        y = x + 0.8 * torch.randn(T, V, generator=g, device=DEV)
        probs, draft = torch.softmax(x, 1).to(dtype), torch.softmax(y, 1).to(dtype) if sampled else None
        source = []
        for t in trees:
            at = len(source)
            source += [at + p if 0 <= p < i else at for i, p in enumerate(t)]
        rows = torch.softmax(y, 1)[torch.tensor(source, device=DEV, dtype=torch.long)] if T - pad else probs[:0].float()
        noise = torch.empty_like(rows).exponential_(generator=g)
        ids = _i32((rows / noise).argmax(1).tolist() + [0] * pad if T - pad else [0] * pad)
        u = torch.rand(T, generator=g, device=DEV)
    if stride:
        wide = [torch.zeros(T, stride, dtype=dtype, device=DEV) for _ in range(2)]
        wide[0][:, 1:V + 1] = probs
        probs = wide[0][:, 1:V + 1]
        if draft is not None:
            wide[1][:, 2:V + 2] = draft
            draft = wide[1][:, 2:V + 2]
    parents = _i32([p for t in trees for p in t] + [0] * pad)
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist()
    out = nq.Verdict(*(torch.full((n,), 77, dtype=torch.int32, device=DEV) for n in (len(trees), T, T)))
    v = nq.verify_drafts(probs, ids, parents, _i32(starts), u, draft_probs=draft, out=out)
    assert v is out
    P, Q = probs.double().cpu().numpy(), None if draft is None else draft.double().cpu().numpy()
    I, U = ids.cpu().numpy(), u.cpu().numpy()
    path, said, count = v.path.tolist(), v.tokens.tolist(), v.accepted.tolist()
    kept = 0
    for r, t in enumerate(trees):
        a, b = starts[r], starts[r + 1]
        want_path, want = ref_verify(P[a:b], None if Q is None else Q[a:b], I[a:b], t, U[a:b])
        rest = [-1] * (len(t) - len(want_path))
        assert (count[r], path[a:b], said[a:b]) == (len(want_path), want_path + rest, want + rest), r
        kept += len(want_path)
    assert path[T - pad:] == [77] * pad and said[T - pad:] == [77] * pad
    return kept


ROWS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", ROWS)
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 128, 1000, 4099, 32000])
def test_verify(nq, dtype, sampled, V):
    trees = [make_tree(TREES[i % 4], n, i) for i, n in enumerate((1, 2, 5, 0, 9, 17, 33, 4, 40, 8))]
    check_verify(nq, trees, V, dtype, sampled, seed=V, pad=2)
    check_verify(nq, trees, V, dtype, sampled, seed=V + 1, stride=V + 5)


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V", [128256, 200003, 524288])
def test_verify_large_vocabularies(nq, sampled, V):
    trees = [make_tree("wide", 9, i) for i in range(4)] + [make_tree("star", 12)]
    check_verify(nq, trees, V, torch.float32, sampled, seed=V)


@pytest.mark.parametrize("sampled", [True, False])
def test_verify_many_requests_and_large_trees(nq, sampled):
    check_verify(nq, [make_tree("wide", 1 + i % 7, i) for i in range(500)], 300, torch.float32, sampled)
    check_verify(nq, [make_tree("star", 300), make_tree("random", 500), make_tree("chain", 200)], 50, torch.float32, sampled)
    check_verify(nq, [[], []], 50, torch.float32, sampled, pad=3)
    check_verify(nq, [], 50, torch.float32, sampled)


def test_verify_borders(nq):
    """Exact ties: a draft is accepted when u q < p, the token that follows has u sum < its running sum; zeros on every side."""
    def one(p, q, ids, parents, u):
        p = torch.tensor(p, device=DEV)
        q = None if q is None else torch.tensor(q, device=DEV)
        check_verify(nq, [parents], p.shape[1], torch.float32, q is not None, probs=p, draft=q, ids=_i32(ids),
                     u=torch.tensor(u, device=DEV))

    p = [[0.5, 0.25, 0.25, 0.0]] * 4
    q = [[0.25, 0.5, 0.0, 0.25]] * 4
    for u0 in (0.0, 0.25, 0.5, 0.75, 0.99999994):
        for u1 in (0.0, 0.25, 0.5, 0.99999994):
            for u2 in (0.0, 0.5):
                for x1 in (0, 1, 2, 3):
                    for x2 in (1, 3):
                        u = [u0, u1, u2, 0.5]
                        for parents in ([-1, 0, 0, 0], [-1, 0, 1, 2], [-1, 0, 0, 1]):
                            one(p, q, [0, x1, x2, 1], parents, u)
                            one(p, None, [0, x1, x2, 1], parents, u)
    # p = q: nothing is left after a rejection, which only u = 1 or p(x) = 0 brings
    one(p, p, [0, 3, 3, 3], [-1, 0, 0, 0], [0.6, 0.0, 0.0, 0.0])
    # all mass on one token that was rejected: none left
    one([[0.0, 1.0, 0.0, 0.0]] * 3, None, [0, 1, 1], [-1, 0, 0], [0.3, 1.0, 0.0])
    # rows of zeros, NaN, negative numbers
    one([[0.0] * 4] * 3, None, [0, 1, 2], [-1, 0, 1], [0.3, 0.0, 0.0])
    one([[0.0] * 4] * 3, q[:3], [0, 1, 2], [-1, 0, 1], [0.3, 0.0, 0.0])
    nan = float("nan")
    one([[nan, -1.0, 0.5, 0.5]] * 3, q[:3], [0, 0, 2], [-1, 0, 0], [0.3, 0.0, 0.9])
    one([[nan, -1.0, 0.5, 0.5]] * 3, [[nan, -3.0, 0.5, 0.5]] * 3, [0, 1, 2], [-1, 0, 0], [0.3, 0.0, 0.9])
    # a number that is not in [0, 1): below 0 as 0, NaN as 0, from 1 on the last token with anything left
    want = {-1.0: 0, nan: 0, 1.0: 2, 5.0: 2}
    for u0, token in want.items():
        v = nq.verify_drafts(torch.tensor(p[:2], device=DEV), _i32([0, 3]), _i32([-1, 0]), _i32([0, 2]),
                             torch.tensor([u0, -1.0], device=DEV))
        assert v.tokens.tolist() == [token, -1] and v.accepted.tolist() == [1]
    # tokens outside the vocabulary are no drafts; parents that are not below their node are nobody's children
    one(p, q, [0, -1, 4, 1], [-1, 0, 0, 0], [0.3, 0.0, 0.0, 0.2])
    one(p, None, [0, 2 ** 31 - 1, -2 ** 31, 0], [-1, 0, 0, 0], [0.3, 0.0, 0.0, 0.2])
    one(p, q, [0, 0, 0, 0], [0, 1, 5, -3], [0.3, 0.0, 0.0, 0.0])


@pytest.mark.parametrize("sampled", [True, False])
def test_verify_gives_the_models_distribution(nq, sampled):
    """The first token of 200000 requests whose two drafts come from another distribution is distributed as the model says: every
    count within five standard deviations."""
    R, V = 200000, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    p = torch.tensor([0.3, 0.05, 0.2, 0.25, 0.0, 0.2], device=DEV)
    q = torch.tensor([0.1, 0.4, 0.2, 0.1, 0.1, 0.1], device=DEV)
    probs, draft = p.expand(3 * R, V).contiguous(), q.expand(3 * R, V).contiguous()
    ids = torch.multinomial(q, 3 * R, replacement=True, generator=g).to(torch.int32)
    if not sampled:
        ids = _i32([0, 1, 3]).repeat(R)
    v = nq.verify_drafts(probs, ids, _i32([-1, 0, 0]).repeat(R), _i32(list(range(0, 3 * R + 1, 3))),
                         torch.rand(3 * R, generator=g, device=DEV), draft_probs=draft if sampled else None)
    first = v.tokens.view(R, 3)[:, 0]
    count = torch.bincount(first.long(), minlength=V).double()
    assert bool(((count - R * p.double()).abs() <= 5 * (R * p.double() * (1 - p.double())).sqrt()).all()), count.tolist()


@pytest.mark.parametrize("sampled", [True, False])
def test_verify_rows_past_32_bits(nq, sampled):
    """Requests at the far end of more than 2^31 probabilities."""
    V, n = 131072, 5
    T = 2 ** 31 // V + 10
    probs = torch.zeros(T, V, dtype=torch.bfloat16, device=DEV)
    draft = torch.zeros_like(probs) if sampled else None
    probs[-n:] = torch.softmax(torch.randn(n, V, device=DEV) * 4, 1)
    if sampled:
        draft[-n:] = torch.softmax(torch.randn(n, V, device=DEV) * 4, 1)
    tree = make_tree("wide", n)
    ids = torch.zeros(T, dtype=torch.int32, device=DEV)
    ids[-n:] = probs[-n:].float().argmax(1).to(torch.int32).roll(1)
    parents, u = _i32([0] * (T - n) + tree), torch.rand(T, device=DEV)
    v = nq.verify_drafts(probs, ids, parents, _i32([T - n, T]), u, draft_probs=draft)
    far = lambda x: x[-n:].double().cpu().numpy()
    path, said = ref_verify(far(probs), far(draft) if sampled else None, far(ids), tree, far(u))
    assert v.path[-n:].tolist()[:len(path)] == path and v.tokens[-n:].tolist()[:len(path)] == said


def test_verify_calls_at_once_on_two_streams(nq):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    R, n, V = 30, 6, 5000
    probs = torch.softmax(torch.randn(R * n, V, generator=g, device=DEV) * 3, 1)
    draft = torch.softmax(torch.randn(R * n, V, generator=g, device=DEV) * 3, 1) / 2 + probs / 2
    ids = torch.multinomial(draft, 1, generator=g).squeeze(1).to(torch.int32)
    u = torch.rand(R * n, generator=g, device=DEV)
    args = (probs, ids, _i32(make_tree("wide", n) * R), _i32(list(range(0, R * n + 1, n))), u)
    want = [nq.verify_drafts(*args, draft_probs=d) for d in (draft, None)]
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(nq.verify_drafts(*args, draft_probs=(draft, None)[i // 2 % 2]))
    torch.cuda.synchronize()
    for i, v in enumerate(got):
        w = want[i // 2 % 2]
        assert torch.equal(v.accepted, w.accepted) and torch.equal(v.path, w.path) and torch.equal(v.tokens, w.tokens)


def test_verify_wild_row_starts(nq):
    T, V = 9, 40
    probs = torch.softmax(torch.randn(T, V, device=DEV), 1)
    buf = torch.full((2, T + 8), 77, dtype=torch.int32, device=DEV)
    for starts in ([-9, 4, 2 ** 31 - 1], [9, 0, 4], [5, 5, 5], [2 ** 31 - 1, -2 ** 31, 3]):
        out = nq.Verdict(torch.empty(2, dtype=torch.int32, device=DEV), buf[0, 4:-4], buf[1, 4:-4])
        nq.verify_drafts(probs, _i32([1] * T), _i32([-1] + [0] * (T - 1)), _i32(starts), torch.rand(T, device=DEV), out=out)
        assert bool((buf[:, :4] == 77).all()) and bool((buf[:, -4:] == 77).all())
        for r in range(2):
            a, b = (min(max(s, 0), T) for s in starts[r:r + 2])
            assert (int(out.accepted[r]) > 0) == (b > a)


# ---------------------------------------------------- compaction and release


@pytest.mark.parametrize("dtype,D", [(torch.float16, 64), (torch.bfloat16, 96), (torch.float16, 128)])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("layers,heads,P", [(1, 1, 16), (3, 8, 16), (2, 3, 128), (5, 2, 32)])
def test_compact(nq, dtype, D, layout, layers, heads, P):
    """Paths of every kind, those whose rows are sources and destinations among them, and those that end early."""
    rng = random.Random(layers * 100 + P)
    paths = [[], [0], [0, 1, 2], [0, 2, 3, 4], [1, 2, 3], [0, 5, 6, 30], list(range(3, 40)), sorted(rng.sample(range(90), 50)),
             [0, 3, 3, 4], [0, 4, 2], [0, -1, 3], [5, 40], [-2, 1]]
    sizes = [4, 1, 3, 5, 4, 31, 40, 90, 6, 5, 4, 20, 3]
    ctx = [0, 5, P - 1, P, 2 * P + 3, 7, 100, 3 * P - 7, 9, 0, 1, 33, 4]
    need = [-(-(c + n) // P) for c, n in zip(ctx, sizes)]
    pages = sum(need) + 3
    shape = (layers, pages, P, heads, D) if layout == "nhd" else (layers, pages, heads, P, D)
    pools = [torch.randn(shape, device=DEV).to(dtype) for _ in range(2)]
    views = [p.transpose(2, 3) if layout == "nhd" else p for p in pools]
    order = list(range(pages))
    rng.shuffle(order)
    cols = max(need) + 1
    table = [[order.pop() for _ in range(m)] + [-1] * (cols - m) for m in need]
    table[11][1], table[7][0] = pages, -5  # pages outside the pool: their rows are passed over
    path = []
    for p, n in zip(paths, sizes):
        path += (p + [-1] * n)[:n]
    path += [9, 9]  # rows of no request
    want = [v.cpu().clone() for v in views]
    for w in want:
        at = 0
        for r, (c, n) in enumerate(zip(ctx, sizes)):
            last = -1
            for k in range(n):
                j = path[at + k]
                if not last < j < n:
                    break
                last = j
                src, dst = table[r][(c + j) // P], table[r][(c + k) // P]
                if 0 <= src < pages and 0 <= dst < pages:
                    w[:, dst, :, (c + k) % P] = w[:, src, :, (c + j) % P]
            at += n
    starts = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    kv = [c + n for c, n in zip(ctx, sizes)]
    if layers == 1:
        got = nq.paged_compact(views[0][0], views[1][0], _i32(table), _i32(starts), _i32(kv), _i32(path))
        assert got[0].dim() == 4
    else:
        got = nq.paged_compact(views[0], views[1], _i32(table), _i32(starts), _i32(kv), _i32(path))
        assert got[0] is views[0] and got[1] is views[1]
    for g, w in zip(views, want):
        assert torch.equal(g.cpu().view(torch.int16), w.view(torch.int16))


def test_compact_offsets_past_32_bits(nq):
    """Pools of more than 2^31 elements over all layers and in one: moves at their far ends."""
    heads, P, D, layers = 8, 256, 128, 3
    pages = 2 ** 31 // (heads * P * D) + 3
    K = torch.zeros(layers, pages, heads, P, D, dtype=torch.float16, device=DEV)
    row = torch.randn(layers, heads, D, device=DEV).half()
    K[:, pages - 1, :, 5] = row
    V = K.clone()
    nq.paged_compact(K, V, _i32([[pages - 2, pages - 1]]), _i32([0, 20]), _i32([P + 10]),
                     _i32([15] + [-1] * 19))  # c = 246: token 261 becomes token 246, slot 246 of the page before
    assert torch.equal(K[:, pages - 2, :, 246], row)
    assert int(K.count_nonzero()) == 2 * int(row.count_nonzero())
    assert torch.equal(K, V)


def test_compact_device_data_is_clamped(nq):
    K = torch.randn(2, 4, 2, 16, 64, device=DEV).half()
    before, V = K.clone(), K.clone()
    path = _i32([1, 2, 3, 4])
    for starts, lens, table in (([-4, 2 ** 31 - 1], [2 ** 31 - 1], [[-1, 4]]), ([4, 0], [9], [[0, 1]]), ([0, 4], [-3], [[0, 1]]),
                                ([0, 4], [0], [[0, 1]]), ([0, 4], [3], [[2 ** 31 - 1, -2 ** 31]])):
        nq.paged_compact(K, V, _i32(table), _i32(starts), _i32(lens), path)
        assert torch.equal(K, before) and torch.equal(V, before)


def ref_release(table, lens, keep, P, free, top):
    free, k, cols = list(free), 0, len(table[0]) if table else 0
    for row, n, m in zip(table, lens, keep):
        for c in range(-(-max(m, 0) // P), min(-(-max(n, 0) // P), cols)):
            if top - 1 - k >= 0:
                free[top - 1 - k] = row[c]
            k += 1
    return free, [k, max(k - top, 0)]


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("R", [0, 1, 13, 511, 512, 513, 1500])
def test_release(nq, P, R):
    rng = random.Random(R)
    for cols, most in ((1, P), (9, 12 * P), (40, 30 * P)):
        lens = [rng.choice([0, 1, P, P + 1, -3, rng.randrange(most)]) for _ in range(R)]
        keep = [rng.choice([0, n, n - 1, n - P, n + 50, rng.randrange(most), -1]) for n in lens]
        table = [[rng.randrange(10 ** 6) for _ in range(cols)] for _ in range(R)]
        total = ref_release(table, lens, keep, P, [], 0)[1][0]
        for top in (total, total + 5, max(total - 3, 0), 0):
            free = [rng.randrange(10 ** 6) for _ in range(top + 4)]
            want, counts = ref_release(table, lens, keep, P, free, top)
            dev = _i32(free)
            wide = torch.full((R, cols + 3), 5, dtype=torch.int32, device=DEV)
            wide[:, :cols] = torch.tensor(table, dtype=torch.int32, device=DEV).view(R, cols)
            got = nq.page_release(wide[:, :cols], _i32(lens), _i32(keep), P, dev, top)
            assert got.tolist() == counts and dev.tolist() == want


def test_release_and_map_share_the_free_list(nq):
    """Pages that are given back are the next ones that the map hands out, and no page is lost or handed out twice."""
    P, R, pages = 16, 9, 200
    rng = random.Random(3)
    free, top = torch.randperm(pages, device=DEV).to(torch.int32), 0
    table = torch.full((R, 30), -1, dtype=torch.int32, device=DEV)
    lens = [0] * R
    for step in range(30):
        new = [rng.randrange(20) if n < 250 else 0 for n in lens]
        nq.page_map(_i32(lens), _i32(new), free[top:], table, P, sum(new))
        full = [a + b for a, b in zip(lens, new)]
        top += sum(-(-b // P) - -(-a // P) for a, b in zip(lens, full))
        keep = [0 if rng.random() < 0.1 else a + rng.randrange(b + 1) for a, b in zip(lens, new)]
        counts = nq.page_release(table, _i32(full), _i32(keep), P, free, top)
        top -= int(counts[0])
        lens = keep
        held = [p for r in range(R) for p in table[r, :-(-lens[r] // P)].tolist()]
        assert sorted(held + free[top:].tolist()) == list(range(pages))


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("config,kw", [("tiny", {"steps": 4, "tree": 8}), ("tiny", {"steps": 3, "tree": 70, "page_size": 32}),
                                       ("phi3mini", {"layers": 2, "tokens": 300, "q_heads": 32, "steps": 3, "tree": 5, "vocab": 1000})])
def test_serving_trees_from_a_compressed_cache(nq, config, kw):
    from e8_lattice_vector_gb300.serve import serve
    from e8_lattice_vector_gb300.synth import CONFIGS

    r = serve(CONFIGS[config], **kw)
    assert 0.01 < r["attention_rel_error"] < 1.0 and 1.0 <= r["accepted_per_step"] <= kw["tree"]
    nq.paged_status()


class ToyModel:
    """Two layers of attention and an output over 40 tokens; its states are kept in fp16 pages."""

    def __init__(self, layers=2, heads=4, kv_heads=2, D=64, V=40, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        def rand(*shape):
            return torch.randn(shape, generator=g, device=DEV)

        self.L, self.H, self.G, self.D, self.V = layers, heads, kv_heads, D, V
        W = 96
        self.E, self.P = rand(V, W), rand(500, W) * 0.5
        self.qkv = [rand(W, (heads + 2 * kv_heads) * D) * W ** -0.5 for _ in range(layers)]
        self.o = [rand(heads * D, W) * (heads * D) ** -0.5 for _ in range(layers)]

    def __call__(self, nq, cache, m, tokens, positions, max_q, tree=None):
        x = self.E[tokens.long()] + self.P[positions.long()]
        for l in range(self.L):
            y = (x @ self.qkv[l]).view(-1, self.H + 2 * self.G, self.D).half()
            nq.paged_append(y[:, self.H:self.H + self.G], y[:, self.H + self.G:], cache.K[l], cache.V[l], m.slots)
            a = nq.paged_attention(y[:, :self.H], cache.K[l], cache.V[l], cache.table, m.q_start, m.kv_lens, max_q=max_q, tree=tree)
            x = x + a.float().flatten(1) @ self.o[l]
        return x @ self.E.T


def test_speculating_with_trees_gives_the_sequential_tokens(nq):
    """Greedy decoding (the model's probabilities are one at its best token), token by token and with drafted trees that hold the right
    continuation here and there: the same tokens, and in the end every page is accounted for."""
    from e8_lattice_vector_gb300.serve import PagedCache, random_tree

    R, steps, P = 5, 40, 16
    model, rng = ToyModel(), random.Random(1)
    dev = torch.device(DEV, 0)

    def new_cache():
        torch.manual_seed(3)
        return PagedCache(2, R, 2, 64, P, 130, torch.float16, dev)

    first = [rng.randrange(40) for _ in range(R)]
    prompts = [[rng.randrange(40) for _ in range(n)] for n in (1, 15, 16, 17, 33)]
    # one token after another
    cache = new_cache()
    m = cache.extend([len(p) for p in prompts])
    model(nq, cache, m, _i32(sum(prompts, [])), m.positions, 33)
    now, truth, margin = list(first), [[] for _ in range(R)], []
    for _ in range(steps):
        m = cache.extend([1] * R)
        logits = model(nq, cache, m, _i32(now), m.positions, 1)
        top = logits.topk(2).values
        margin.append(float((top[:, 0] - top[:, 1]).min()))
        now = logits.argmax(1).tolist()
        for r in range(R):
            truth[r].append(now[r])
    assert min(margin) > 1e-3  # no choice hangs on a rounding
    # trees: some children are the right token, others are not
    cache = new_cache()
    m = cache.extend([len(p) for p in prompts])
    model(nq, cache, m, _i32(sum(prompts, [])), m.positions, 33)
    now, said = list(first), [[] for _ in range(R)]
    while min(len(s) for s in said) < steps:
        trees, ids = [], []
        for r in range(R):
            if len(said[r]) >= steps:
                trees.append([])
                continue
            t = random_tree(rng.randrange(1, 14), rng)
            depth, right = [], []  # right: the path down to the node is the true continuation
            for i, p in enumerate(t):
                depth.append(0 if i == 0 else depth[p] + 1)
                at = len(said[r]) + depth[i] - 1
                true = truth[r][at] if i > 0 and at < steps else -1
                tok = now[r] if i == 0 else true if true >= 0 and rng.random() < 0.6 else rng.randrange(40)
                right.append(i == 0 or (right[p] and tok == true))
                ids.append(tok)
            trees.append(t)
        step = cache.draft(trees)
        logits = model(nq, cache, step.map, _i32(ids), step.tree.positions, max(step.nodes), step.tree)
        probs = torch.nn.functional.one_hot(logits.argmax(1), 40).float()
        u = torch.rand(len(ids), device=DEV)
        before = list(cache.lengths)
        v = nq.verify_drafts(probs, _i32(ids), step.parents, step.map.q_start, u)
        kept = cache.keep(step, v)
        tokens, at = v.tokens.tolist(), 0
        for r, t in enumerate(trees):
            got = tokens[at:at + kept[r]]
            said[r] += got
            assert tokens[at + kept[r]:at + len(t)] == [-1] * (len(t) - kept[r])
            assert cache.lengths[r] == before[r] - len(t) + kept[r]
            if t:
                now[r] = got[-1]
            at += len(t)
        held = [p for r in range(R) for p in cache.table[r, :-(-cache.lengths[r] // P)].tolist()]
        assert sorted(held + cache.free.tolist()) == list(range(R * cache.columns))
    for r in range(R):
        assert said[r][:steps] == truth[r]
    cache.end([0, 3])
    assert cache.lengths[0] == cache.lengths[3] == 0 and cache.lengths[1] > 0
    held = [p for r in range(R) for p in cache.table[r, :-(-cache.lengths[r] // P)].tolist()]
    assert sorted(held + cache.free.tolist()) == list(range(R * cache.columns))


def test_a_step_without_drafts(nq):
    """Every request sits the step out."""
    from e8_lattice_vector_gb300.serve import PagedCache

    c = PagedCache(1, 2, 2, 64, 16, 40, torch.float16, torch.device(DEV, 0))
    c.fill(*(torch.randn(1, 2, 2, 20, 64, device=DEV).half() for _ in range(2)))
    step = c.draft([[], []])
    out = c.draft_step(*(torch.empty(1, 0, h, 64, dtype=torch.float16, device=DEV) for h in (4, 2, 2)), step)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    v = nq.verify_drafts(torch.empty(0, 50, device=DEV), none, step.parents, step.map.q_start, torch.empty(0, device=DEV))
    assert out.shape[1] == 0 and v.accepted.tolist() == [0, 0]
    assert c.keep(step, v) == [0, 0] and c.lengths == [20, 20] and c.top == 4


def test_a_whole_step_in_one_graph(nq):
    """Map, tree, append, attention, verification, compaction and release captured once, replayed over other lengths and trees."""
    R, n, P, H, D, V, L = 4, 12, 16, 2, 64, 500, 2
    T, cols, pages = R * n, 12, 60
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    pools = [rand(L, pages, H, P, D).half() for _ in range(2)]
    saved = [p.clone() for p in pools]
    q, k, v = rand(L, T, 4, D).half(), rand(L, T, H, D).half(), rand(L, T, H, D).half()
    probs, draft = torch.softmax(rand(T, V) * 2, 1), torch.softmax(rand(T, V) * 2, 1)
    draft = (draft + probs) / 2
    u = torch.rand(T, generator=g, device=DEV)
    ids = torch.multinomial(draft, 1, generator=g).squeeze(1).to(torch.int32)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    ctx, new, parents = _i32([0] * R), _i32([n] * R), _i32(make_tree("wide", n) * R)
    table = torch.full((R, cols), -1, dtype=torch.int32, device=DEV)
    free, top = order.clone(), 24  # entries before it are in the table

    def step():
        m = nq.page_map(ctx, new, free[top:], table, P, T)
        t = nq.draft_tree(parents, m.q_start, m.kv_lens, n)
        out = [None] * L
        for l in range(L):
            nq.paged_append(k[l], v[l], pools[0][l], pools[1][l], m.slots)
            out[l] = nq.paged_attention(q[l], pools[0][l], pools[1][l], table, m.q_start, m.kv_lens, max_q=n, tree=t)
        w = nq.verify_drafts(probs, ids, parents, m.q_start, u, draft_probs=draft)
        nq.paged_compact(pools[0], pools[1], table, m.q_start, m.kv_lens, w.path)
        counts = nq.page_release(table, m.kv_lens, ctx + w.accepted, P, free, top)
        return [*out, t.positions, w.accepted, w.path, w.tokens, counts]

    def setup(lens, sizes, shape):
        ctx.copy_(_i32(lens))
        new.copy_(_i32(sizes))
        parents.copy_(_i32([p for r, s in enumerate(sizes) for p in make_tree(shape, s, r)] + [-1] * (T - sum(sizes))))
        free.copy_(order)
        table.fill_(-1)
        at = 0
        for r, c in enumerate(lens):
            held = -(-c // P)
            table[r, :held] = order[at:at + held]
            at += held
        for p, s in zip(pools, saved):
            p.copy_(s)

    cases = [([10, 0, 33, 80], [12, 12, 12, 12], "wide"), ([90, 16, 15, 1], [1, 12, 7, 0], "random"), ([5, 6, 7, 8], [12, 3, 12, 12], "chain")]
    setup(*cases[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    torch.cuda.synchronize()
    for case in cases:
        setup(*case)
        graph.replay()
        torch.cuda.synchronize()
        rows, state = sum(case[1]), [pools[0].clone(), pools[1].clone(), free.clone(), table.clone()]
        one = [x.clone() for x in got]
        setup(*case)
        want = step()
        for a, b in zip(one, want):
            n_rows = rows if a.shape[0] == T else a.shape[0]
            assert torch.equal(a[:n_rows], b[:n_rows])
        for a, b in zip(state, (pools[0], pools[1], free, table)):
            assert torch.equal(a, b)
    nq.paged_status()
