"""What the paged-cache calls refuse, at the C entry points and in the binding: every case returns before any CUDA
call, so no GPU is needed."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def nq():
    from e8_lattice_vector_gb300 import build as nqbuild

    nqbuild.build()
    from e8_lattice_vector_gb300 import _lib

    return _lib


P16, P8, P4, P2 = 16, 8, 4, 2
ARG, UNSUPPORTED, SIZE = 1, 2, 3


def _pool(nq, **kw):
    f = dict(dtype=0, pages=10, kv_heads=8, page_size=16, head_dim=128, reserved=0, page_stride=8 * 16 * 128,
             head_stride=16 * 128, slot_stride=128)
    f.update(kw)
    return nq.Pool(**f)


def _attn(nq, **kw):
    f = dict(tokens=4, q_heads=32, requests=2, table_cols=5, max_q=2, causal=1, window=0, scale=0.1, table_stride=5,
             q_token_stride=32 * 128, q_head_stride=128, out_token_stride=32 * 128, out_head_stride=128)
    f.update(kw)
    return nq.Attention(**f)


BAD_POOLS = [(dict(kv_heads=65537), ARG), (dict(dtype=2), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
             (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
             (dict(pages=0), ARG), (dict(kv_heads=0), ARG), (dict(page_stride=100), ARG), (dict(slot_stride=132), ARG),
             (dict(slot_stride=64), ARG), (dict(head_stride=0), ARG), (dict(head_stride=-128), ARG),
             (dict(page_stride=1 << 39), ARG)]


def test_map_refusals(nq):
    f = nq.lib().nq_page_map
    good = [P16, P16, 3, P16, 5, P16, 7, 7, 16, 4, P16, P16, P16, P16, P16, None]
    cases = [(i, None, ARG) for i in (0, 1, 3, 5, 10, 11, 12, 13, 14)]
    cases += [(i, -1, ARG) for i in (2, 4, 7, 9)]
    cases += [(i, P2, ARG) for i in (0, 1, 3, 5, 10, 11, 13, 14)] + [(12, P4, ARG), (6, 6, ARG)]
    cases += [(8, v, UNSUPPORTED) for v in (0, -16, 8, 24, 512)]
    for i, v, status in cases:
        args = list(good)
        args[i] = v
        assert f(*args) == status, (i, v)


def test_append_refusals(nq):
    f = nq.lib().nq_paged_append
    pool = _pool(nq)
    good = [P16, 1024, 128, P16, 1024, 128, 4, P16, ctypes.byref(pool), P16, P16, None]
    cases = [(i, None, ARG) for i in (0, 3, 7, 8, 9, 10)] + [(6, -1, ARG)]
    cases += [(i, P8, ARG) for i in (0, 3, 9, 10)] + [(7, P4, ARG)]
    cases += [(i, v, ARG) for i in (1, 2, 4, 5) for v in (1023, -8, 1 << 39)]
    for i, v, status in cases:
        args = list(good)
        args[i] = v
        assert f(*args) == status, (i, v)
    for kw, status in BAD_POOLS:
        args = list(good)
        args[8] = ctypes.byref(_pool(nq, **kw))
        assert f(*args) == status, kw
    args = list(good)
    args[0], args[6] = None, 0  # no tokens: nothing to do
    assert f(*args) == 0


def test_attention_refusals(nq):
    L = nq.lib()
    f, pool = L.nq_paged_attention, _pool(nq)
    att = _attn(nq)
    need = ctypes.c_uint64(0)
    assert L.nq_paged_attention_workspace(ctypes.byref(att), ctypes.byref(pool), ctypes.byref(need)) == 0
    good = [ctypes.byref(att), P16, ctypes.byref(pool), P16, P16, P16, P16, P16, P16, None, P16, need.value, None]
    cases = [(i, None, ARG) for i in (0, 1, 2, 3, 4, 5, 6, 7, 8)]
    cases += [(i, P8, ARG) for i in (1, 3, 4, 8, 10)] + [(i, P2, ARG) for i in (5, 6, 7, 9)]
    if need.value:
        cases += [(10, None, ARG), (11, need.value - 1, SIZE)]
    for i, v, status in cases:
        args = list(good)
        args[i] = v
        assert f(*args) == status, (i, v)
    for kw, status in BAD_POOLS:
        args = list(good)
        args[2] = ctypes.byref(_pool(nq, **kw))
        assert f(*args) == status, kw
        assert L.nq_paged_attention_workspace(args[0], args[2], ctypes.byref(need)) == status, kw
    inf, nan = float("inf"), float("nan")
    for kw in (dict(tokens=-1), dict(requests=-1), dict(table_cols=-1), dict(max_q=-1), dict(window=-1),
               dict(causal=2), dict(causal=-1), dict(q_heads=0), dict(q_heads=12), dict(q_heads=-8), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=inf), dict(scale=nan), dict(table_cols=1 << 27, table_stride=1 << 27),
               dict(table_stride=4), dict(q_token_stride=4), dict(q_head_stride=0), dict(out_token_stride=64),
               dict(tokens=1 << 26),  dict(q_head_stride=-8), dict(out_token_stride=12),
               dict(out_head_stride=1 << 39)):
        args = list(good)
        args[0] = ctypes.byref(_attn(nq, **kw))
        assert f(*args) == ARG, kw
        assert L.nq_paged_attention_workspace(args[0], args[2], ctypes.byref(need)) == ARG, kw
    assert L.nq_paged_attention_workspace(good[0], good[2], None) == ARG
    for kw in (dict(tokens=0), dict(requests=0)):  # nothing to do
        assert f(ctypes.byref(_attn(nq, **kw)), None, good[2], *[None] * 8, 0, None) == 0


class _Fake:
    """Stand-in for a CUDA tensor, strided."""

    def __init__(self, shape, dtype, strides=None, device="cuda:0", ptr=256):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device(device), True
        dense = [1]
        for n in reversed(shape[1:]):
            dense.insert(0, dense[0] * n)
        self._strides = tuple(dense) if strides is None else tuple(strides)
        self._dense = tuple(dense) == self._strides
        self._ptr = ptr

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        return self._strides if d is None else self._strides[d]

    def is_contiguous(self):
        return self._dense

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return self._ptr

    def get_device(self):
        return self.device.index


H16, I32, I64 = torch.float16, torch.int32, torch.int64


def test_binding_refusals(nq):
    import e8_lattice_vector_gb300 as pkg

    def raises(text, fn, *a, **kw):
        with pytest.raises(ValueError, match=text):
            fn(*a, **kw)

    pool = _Fake((10, 8, 16, 128), H16)
    kv, slots, q = _Fake((4, 8, 128), H16), _Fake((4,), I64), _Fake((4, 32, 128), H16)
    # the append
    app = lambda **kw: [kw.get(n, d) for n, d in (("K", kv), ("V", kv), ("Kp", pool), ("Vp", pool), ("slots", slots))]
    raises("K_pages must be", pkg.paged_append, *app(Kp=_Fake((10, 8, 16, 128), torch.float32)))
    raises("K_pages must be", pkg.paged_append, *app(Kp=_Fake((10, 8, 128), H16)))
    raises("K_pages must be", pkg.paged_append, *app(Kp=_Fake((10, 8, 16, 128), H16, (16384, 2048, 1, 16))))
    raises("K_pages has stride", pkg.paged_append, *app(Kp=_Fake((10, 8, 16, 128), H16, (16388, 2048, 128, 1))))
    raises("K_pages must start", pkg.paged_append, *app(Kp=_Fake((10, 8, 16, 128), H16, ptr=264)))
    raises("V_pages must have", pkg.paged_append, *app(Vp=_Fake((9, 8, 16, 128), H16)))
    raises("V_pages must have", pkg.paged_append, *app(Vp=_Fake((10, 8, 16, 128), torch.bfloat16)))
    raises("V_pages must have", pkg.paged_append, *app(Vp=_Fake((10, 8, 16, 128), H16, device="cuda:1")))
    raises("K must be", pkg.paged_append, *app(K=_Fake((4, 8, 128), torch.bfloat16)))
    raises("K has shape", pkg.paged_append, *app(K=_Fake((4, 4, 128), H16)))
    raises("V has shape", pkg.paged_append, *app(V=_Fake((5, 8, 128), H16)))
    raises("K has stride", pkg.paged_append, *app(K=_Fake((4, 8, 128), H16, (1028, 128, 1))))
    raises("K is on", pkg.paged_append, *app(K=_Fake((4, 8, 128), H16, device="cuda:1")))
    raises("V must start", pkg.paged_append, *app(V=_Fake((4, 8, 128), H16, ptr=24)))
    raises("slots must be", pkg.paged_append, *app(slots=_Fake((4,), I32)))
    raises("slots has 5", pkg.paged_append, *app(slots=_Fake((5,), I64)))
    # the map
    lens, free, table = _Fake((3,), I32), _Fake((9,), I32), _Fake((3, 7), I32)
    raises("ctx_lens must be", pkg.page_map, _Fake((3,), I64), lens, free, table, 16, 4)
    raises("new_lens has", pkg.page_map, lens, _Fake((4,), I32), free, table, 16, 4)
    raises("free_pages is on", pkg.page_map, lens, lens, _Fake((9,), I32, device="cuda:1"), table, 16, 4)
    raises("block_table has", pkg.page_map, lens, lens, free, _Fake((4, 7), I32), 16, 4)
    raises("block_table must be", pkg.page_map, lens, lens, free, _Fake((3, 7), I32, (1, 3)), 16, 4)
    vec = lambda n, t=I32: _Fake((n,), t)
    raises("out.slots must be", pkg.page_map, lens, lens, free, table, 16, 4,
           out=pkg.PageMap(vec(4), vec(3), vec(4), vec(4), vec(4)))
    raises("out.q_start has", pkg.page_map, lens, lens, free, table, 16, 4,
           out=pkg.PageMap(vec(3), vec(3), vec(4, I64), vec(4), vec(4)))
    # the attention
    start = _Fake((4,), I32)
    att = lambda Q=q, Kp=pool, Vp=pool, table=table, q_start=start, kv_lens=lens, **kw: \
        pkg.paged_attention(Q, Kp, Vp, table, q_start, kv_lens, out=kw.pop("out", q), **kw)
    raises("Q must be", att, Q=_Fake((4, 4096), H16))
    raises("Q must be", att, Q=_Fake((4, 32, 128), torch.bfloat16))
    raises("Q has shape", att, Q=_Fake((4, 32, 64), H16))
    raises("cannot share", att, Q=_Fake((4, 12, 128), H16))
    raises("out has shape", att, out=_Fake((5, 32, 128), H16))
    raises("q_start has", att, q_start=lens)
    raises("kv_lens must be", att, kv_lens=_Fake((3,), I64))
    raises("block_table has", att, table=_Fake((2, 7), I32))
    raises("block_table is on", att, table=_Fake((3, 7), I32, device="cuda:1"))
    raises("lse must be", att, lse=_Fake((4, 32), H16))
    raises("lse must be", att, lse=_Fake((4, 31), torch.float32))
    raises("ws must be", att, ws=_Fake((4,), torch.float32))
    with pytest.raises(nq.NQError):
        att(scale=-1.0)
    with pytest.raises(nq.NQError):
        att(window=-1)
    with pytest.raises(nq.NQError):
        att(Kp=_Fake((10, 8, 24, 128), H16), Vp=_Fake((10, 8, 24, 128), H16))
