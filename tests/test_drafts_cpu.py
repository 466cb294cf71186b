"""What the calls for drafted trees refuse, at the C entry points and in the binding: every case returns before any CUDA call, so
no GPU is needed."""
import ctypes

import pytest
import torch

from test_paged_cpu import ARG, BAD_POOLS, H16, I32, I64, P2, P4, P8, P16, SIZE, UNSUPPORTED, _attn, _Fake, _pool, nq  # noqa: F401

F32 = torch.float32


class _Layers(_Fake):
    """Pools of several layers; an index gives one layer's."""

    def __getitem__(self, i):
        return _Fake(self.shape[1:], self.dtype, self._strides[1:])


def run(f, good, cases):
    for i, v, status in cases:
        args = list(good)
        args[i] = v
        assert f(*args) == status, (i, v)


def test_draft_tree_refusals(nq):
    f = nq.lib().nq_draft_tree
    good = [P16, 4, P16, P16, 2, 0, 1, P16, P16, None]
    run(f, good, [(i, None, ARG) for i in (0, 2, 3, 7, 8)] + [(i, -1, ARG) for i in (1, 4, 5)] + [(6, v, ARG) for v in (0, -1, 65)] +
        [(i, P2, ARG) for i in (0, 2, 3, 8)] + [(7, P4, ARG)])
    assert f(None, 0, None, None, 2, 0, 1, None, None, None) == 0  # nothing to do
    assert f(None, 4, None, None, 0, 0, 64, None, None, None) == 0


def test_tree_attention_refusals(nq):
    L = nq.lib()
    f, pool, att, need = L.nq_paged_tree_attention, _pool(nq), _attn(nq), ctypes.c_uint64(0)
    assert L.nq_paged_attention_workspace(ctypes.byref(att), ctypes.byref(pool), ctypes.byref(need)) == 0
    good = [ctypes.byref(att), P16, P16, 1, P16, ctypes.byref(pool), P16, P16, P16, P16, P16, P16, None, P16, need.value, None]
    cases = [(i, None, ARG) for i in (0, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11, 13)]
    cases += [(1, P4, ARG), (2, P2, ARG)] + [(3, v, ARG) for v in (0, -1, 65)]
    cases += [(i, P8, ARG) for i in (4, 6, 7, 11, 13)] + [(i, P2, ARG) for i in (8, 9, 10, 12)] + [(14, need.value - 1, SIZE)]
    run(f, good, cases)
    for kw, status in BAD_POOLS:
        args = list(good)
        args[5] = ctypes.byref(_pool(nq, **kw))
        assert f(*args) == status, kw
    for kw in (dict(causal=0), dict(tokens=-1), dict(window=-1), dict(scale=0.0), dict(q_heads=12), dict(q_token_stride=4)):
        args = list(good)
        args[0] = ctypes.byref(_attn(nq, **kw))
        assert f(*args) == ARG, kw
    for kw in (dict(tokens=0), dict(requests=0)):  # nothing to do
        assert f(ctypes.byref(_attn(nq, **kw)), None, None, 1, None, good[5], *[None] * 8, 0, None) == 0


def test_verify_refusals(nq):
    f = nq.lib().nq_verify_drafts
    at = lambda i: 4096 * i
    good = [at(1), 100, at(2), 100, 2, 100, at(3), at(4), at(5), 4, at(6), 2, at(7), at(8), at(9), None]
    run(f, good, [(i, None, ARG) for i in (0, 6, 7, 8, 10, 12, 13, 14)] + [(i, 99, ARG) for i in (1, 3)] +
        [(4, v, UNSUPPORTED) for v in (-1, 3)] + [(5, v, ARG) for v in (0, -1, 2 ** 31 - 1)] + [(i, -1, ARG) for i in (9, 11)] + [(11, 1 << 28, ARG)] +
        [(i, P2, ARG) for i in (0, 2, 6, 7, 8, 10, 12, 13, 14)])
    for i, j, by in ((13, 6, 0), (14, 6, 12), (14, 7, -12), (13, 8, 0), (14, 13, 4), (13, 10, 8), (14, 12, 4)):  # outputs over others
        args = list(good)
        args[i] = good[j] + by
        assert f(*args) == ARG, (i, j)
    odd = list(good)
    odd[4], odd[0] = 0, 3  # fp16 on an odd address
    assert f(*odd) == ARG
    assert f(*[None, 0, None, 0, 2, 100, None, None, None, 0, None, 0, None, None, None, None]) == 0


def test_compact_refusals(nq):
    f, pool = nq.lib().nq_paged_compact, _pool(nq)
    good = [ctypes.byref(pool), 3, 10 * 8 * 16 * 128, P16, 2 * P16, P16, 5, 5, P16, P16, 2, P16, 4, None]
    run(f, good, [(i, None, ARG) for i in (0, 3, 4, 5, 8, 9, 11)] + [(i, -1, ARG) for i in (1, 7, 10, 12)] + [(1, 65536, ARG)] +
        [(2, v, ARG) for v in (1004, 0, -128, 64, 1 << 39)] + [(i, P8, ARG) for i in (3, 4)] + [(i, P2, ARG) for i in (5, 8, 9, 11)] +
        [(6, 4, ARG), (7, 1 << 27, ARG), (4, P16, ARG)])
    for kw, status in BAD_POOLS:
        args = list(good)
        args[0] = ctypes.byref(_pool(nq, **kw))
        assert f(*args) == status, kw
    for i in (1, 7, 10, 12):  # nothing to do
        args = [None if j in (3, 4, 5, 8, 9, 11) else v for j, v in enumerate(good)]
        args[i] = 0
        assert f(*args) == 0


def test_release_refusals(nq):
    f = nq.lib().nq_page_release
    good = [P16, 7, 7, P16, P16, 3, 16, P16, 5, P16, None]
    run(f, good, [(i, None, ARG) for i in (0, 3, 4, 7, 9)] + [(i, -1, ARG) for i in (2, 5, 8)] + [(1, 6, ARG)] +
        [(i, P2, ARG) for i in (0, 3, 4, 7, 9)] + [(6, v, UNSUPPORTED) for v in (0, -16, 8, 24, 512)])


def test_binding_refusals(nq):
    import e8_lattice_vector_gb300 as pkg

    def raises(text, fn, *a, **kw):
        with pytest.raises(ValueError, match=text):
            fn(*a, **kw)

    vec = lambda n, t=I32, **kw: _Fake((n,), t, **kw)
    lens, starts, rows = vec(3), vec(4), vec(4)
    bits, tree = _Fake((4, 1), I64), pkg.DraftTree(_Fake((4, 1), I64), vec(4))
    # the map
    raises("max_q is -1", pkg.draft_tree, rows, starts, lens, -1)
    raises("max_q is 4097", pkg.draft_tree, rows, starts, lens, 4097)
    raises("parents must be", pkg.draft_tree, vec(4, I64), starts, lens, 4)
    raises("q_start has", pkg.draft_tree, rows, lens, lens, 4)
    raises("kv_lens must be", pkg.draft_tree, rows, starts, vec(3, I64), 4)
    raises("kv_lens is on", pkg.draft_tree, rows, starts, vec(3, device="cuda:1"), 4)
    raises("out.ancestors must be", pkg.draft_tree, rows, starts, lens, 4, out=pkg.DraftTree(_Fake((4, 1), I32), rows))
    raises("out.ancestors has shape", pkg.draft_tree, rows, starts, lens, 4, out=pkg.DraftTree(_Fake((5, 1), I64), rows))
    raises("out.ancestors has 1 words", pkg.draft_tree, rows, starts, lens, 65, out=tree)
    raises("out.positions has", pkg.draft_tree, rows, starts, lens, 4, out=pkg.DraftTree(bits, vec(5)))
    raises("window is -1", pkg.draft_tree, rows, starts, lens, 4, window=-1, out=tree)
    # the attention
    pool, q, table = _Fake((10, 8, 16, 128), H16), _Fake((4, 32, 128), H16), _Fake((3, 7), I32)
    att = lambda t, **kw: pkg.paged_attention(q, pool, pool, table, starts, lens, out=q, tree=t, **kw)
    raises("tree.ancestors must be", att, pkg.DraftTree(_Fake((4, 1), I32), rows))
    raises("tree.ancestors must be", att, pkg.DraftTree(_Fake((4, 2), I64, (4, 1)), rows))
    raises("tree.ancestors has shape", att, pkg.DraftTree(_Fake((3, 1), I64), rows))
    raises("tree.ancestors has shape", att, pkg.DraftTree(_Fake((4, 65), I64), rows))
    raises("tree.ancestors has shape", att, pkg.DraftTree(_Fake((4, 0), I64), rows))
    raises("tree.ancestors is on", att, pkg.DraftTree(_Fake((4, 1), I64, device="cuda:1"), rows))
    raises("tree.positions has", att, pkg.DraftTree(bits, vec(5)))
    raises("tree is causal", att, tree, causal=False)
    # the verification
    p, u = _Fake((4, 100), F32), vec(4, F32)
    ver = lambda probs=p, tokens=rows, parents=rows, q_start=starts, uniform=u, **kw: pkg.verify_drafts(
        probs, tokens, parents, q_start, uniform, **kw)
    raises("probs must be", ver, probs=_Fake((4, 100), torch.float64))
    raises("probs must be", ver, probs=_Fake((4, 100), F32, (1, 4)))
    raises("probs must be", ver, probs=vec(4, F32))
    raises("draft_probs must have", ver, draft_probs=_Fake((4, 100), H16))
    raises("draft_probs must have", ver, draft_probs=_Fake((4, 99), F32))
    raises("draft_probs must have", ver, draft_probs=_Fake((4, 100), F32, device="cuda:1"))
    raises("draft_probs must be", ver, draft_probs=_Fake((4, 100), F32, (1, 4)))
    raises("tokens must be", ver, tokens=vec(4, I64))
    raises("parents has", ver, parents=vec(5))
    raises("uniform must be", ver, uniform=vec(4, torch.float64))
    raises("q_start has no", ver, q_start=vec(0))
    raises("out.accepted has", ver, out=pkg.Verdict(vec(4), rows, rows))
    raises("out.path has", ver, out=pkg.Verdict(vec(3), vec(3), rows))
    raises("out.tokens must be", ver, out=pkg.Verdict(vec(3), rows, vec(4, I64)))
    # the compaction
    com = lambda K=pool, V=pool, t=table, s=starts, n=lens, path=rows: pkg.paged_compact(K, V, t, s, n, path)
    raises("K_pages must be", com, K=_Fake((10, 8, 16, 128), F32))
    raises("V_pages must have", com, V=_Fake((9, 8, 16, 128), H16))
    raises("K_pages must start", com, K=_Fake((10, 8, 16, 128), H16, ptr=264))
    raises("path must be", com, path=vec(4, I64))
    raises("path is on", com, path=vec(4, device="cuda:1"))
    raises("kv_lens must be", com, n=vec(3, I64))
    raises("q_start has", com, s=lens)
    raises("block_table has", com, t=_Fake((2, 7), I32))
    deep = _Layers((3, 10, 8, 16, 128), H16)
    raises("V_pages must have", com, K=deep)
    raises("V_pages must have", com, K=deep, V=_Layers((2, 10, 8, 16, 128), H16))
    raises("has no layers", com, K=_Layers((0, 10, 8, 16, 128), H16), V=_Layers((0, 10, 8, 16, 128), H16))
    odd = _Layers((3, 10, 8, 16, 128), H16, (163844, 16384, 2048, 128, 1))
    raises("stride 163844 along axis 0", com, K=odd, V=odd)
    # the release
    rel = lambda t=table, n=lens, k=lens, P=16, free=vec(9), top=4, **kw: pkg.page_release(t, n, k, P, free, top, **kw)
    raises("top is 10", rel, top=10)
    raises("top is -1", rel, top=-1)
    raises("free_pages must be", rel, free=vec(9, I64))
    raises("keep_lens has", rel, k=vec(4))
    raises("kv_lens must be", rel, n=vec(3, I64), k=vec(3))
    raises("block_table is on", rel, t=_Fake((3, 7), I32, device="cuda:1"))
    raises("out has", rel, out=vec(3))


def test_a_paged_cache_keeps_accepted_rows_and_counts_pages(monkeypatch):
    """keep() and end() hand the right lengths on, and the free list's top follows them."""
    from e8_lattice_vector_gb300 import serve
    from e8_lattice_vector_gb300.drafts import DraftTree, Verdict
    from e8_lattice_vector_gb300.paged import PageMap

    calls = []
    monkeypatch.setattr(serve, "page_map", lambda ctx, new, free, *a: PageMap(*(torch.zeros(0),) * 5) if calls.append(
        ("map", ctx.tolist(), new.tolist(), free.numel())) else PageMap(torch.zeros(4), ctx + new, *(torch.zeros(0),) * 3))
    monkeypatch.setattr(serve, "draft_tree", lambda parents, q, kv, most: calls.append(("tree", parents.tolist(), most)) or DraftTree(
        torch.zeros(0), torch.zeros(0)))
    monkeypatch.setattr(serve, "paged_compact", lambda K, V, table, q, kv, path: calls.append(("compact", path.tolist())))
    monkeypatch.setattr(serve, "page_release", lambda table, lens, keep, size, free, top: calls.append(
        ("release", lens.tolist(), keep.tolist(), size, free.numel(), top)))
    c = serve.PagedCache(1, 3, 1, 64, 16, 60, torch.float16, torch.device("cpu"))  # four pages each
    c.extend([30, 16, 0])
    step = c.draft([[-1, 0, 0, 1], [], [-1] + list(range(39))])
    assert c.lengths == [34, 16, 40] and c.top == 3 + 1 + 3 and c.free.numel() == 5
    assert calls[-2:] == [("map", [30, 16, 0], [4, 0, 40], 9), ("tree", [-1, 0, 0, 1, -1] + list(range(39)), 40)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    path = [0, 2, -1, -1] + list(range(17)) + [-1] * 23
    assert c.keep(step, Verdict(i32([2, 0, 17]), i32(path), None)) == [2, 0, 17]
    assert calls[-2:] == [("compact", path), ("release", [34, 16, 40], [32, 16, 17], 16, 12, 7)]
    assert c.lengths == [32, 16, 17] and c.top == 2 + 1 + 2
    c.end([1, 2])
    assert calls[-1] == ("release", [32, 16, 17], [32, 0, 0], 16, 12, 5)
    assert c.lengths == [32, 0, 0] and c.top == 2 and c.free.numel() == 10
