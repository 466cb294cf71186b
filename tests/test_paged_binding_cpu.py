"""What the paged binding hands to the library: no GPU is needed, the library's calls are recorded."""
import pytest
import torch


@pytest.fixture
def paged(monkeypatch):
    from e8_lattice_vector_gb300 import build as nqbuild

    nqbuild.build()
    from e8_lattice_vector_gb300 import paged

    paged.calls = []
    monkeypatch.setattr(paged, "_launch", lambda index, fn, *args: paged.calls.append((index, fn.__name__, args)))
    monkeypatch.setattr(paged, "_KEPT", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    return paged


def test_status_of_any_device(paged):
    for device, index in ((None, 3), ("cuda", 3), (torch.device("cuda"), 3), ("cuda:1", 1), (torch.device("cuda", 0), 0)):
        paged.paged_status(device)
        assert paged.calls.pop() == (index, "nq_paged_status", ())
    with pytest.raises(ValueError, match="CUDA device"):
        paged.paged_status("cpu")
    assert not paged.calls


def test_numbers_past_32_bits_do_not_wrap(paged, monkeypatch):
    """The library's counts are 32-bit: a bound or a window past them means the largest, a size past them is refused."""
    from test_paged_cpu import H16, I32, I64, _Fake

    pool, q, lens = _Fake((10, 8, 16, 128), H16), _Fake((4, 32, 128), H16), _Fake((3,), I32)
    table, starts, ws = _Fake((3, 7), I32), _Fake((4,), I32), _Fake((1 << 30,), torch.uint8)

    def attention(**kw):
        paged.paged_attention(q, pool, pool, kw.pop("table", table), starts, lens, out=q, ws=ws, **kw)
        return paged.calls.pop()[2][0]._obj

    assert attention(window=5).window == 5 and attention().window == 0
    for n in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 70):
        assert attention(window=n).window == 2 ** 31 - 1
        assert attention(max_q=n).max_q == 2 ** 31 - 1
    rows, sizes = _Fake((40, 32, 128), H16), []
    monkeypatch.setattr(paged, "workspace", lambda need, device: sizes.append(need))
    for n in (1, 2 ** 31 - 1, 2 ** 32 + 1):
        paged.paged_attention_workspace(rows, pool, table, max_q=n)
    assert sizes[0] < sizes[1] == sizes[2]
    for n in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(RuntimeError):
            attention(window=n)
        with pytest.raises(RuntimeError):
            attention(max_q=n)
    with pytest.raises(ValueError, match="block_table"):
        attention(table=_Fake((3, 2 ** 32 + 7), I32))
    vec = lambda n, t=I32: _Fake((n,), t)
    out = lambda tokens: paged.PageMap(vec(4), vec(3), vec(tokens, I64), vec(tokens), vec(4))
    paged.page_map(lens, lens, vec(9), table, 16, 4, out=out(4))
    assert paged.calls.pop()[2][8:10] == (16, 4)
    for name, args in (("page_size", (vec(9), table, 2 ** 32 + 16, 4, out(4))),
                       ("tokens", (vec(9), table, 16, 2 ** 32 + 4, out(2 ** 32 + 4))),
                       ("free_pages", (vec(2 ** 32 + 9), table, 16, 4, out(4))),
                       ("block_table", (vec(9), _Fake((3, 2 ** 32 + 7), I32), 16, 4, out(4)))):
        with pytest.raises(ValueError, match=name):
            paged.page_map(lens, lens, *args[:-1], out=args[-1])
    big = 2 ** 32 + 4
    with pytest.raises(ValueError, match="slots"):
        paged.paged_append(_Fake((big, 8, 128), H16), _Fake((big, 8, 128), H16), pool, pool, vec(big, I64))
    assert not paged.calls


def test_checks_run_once_for_a_free_list_of_any_length(paged, monkeypatch):
    """A free list gets shorter with almost every step: its length is no part of what the checks are kept under."""
    from test_paged_cpu import I32, I64, _Fake

    vec = lambda n, t=I32, **kw: _Fake((n,), t, **kw)
    lens, table, runs, check = vec(3), _Fake((3, 7), I32), [], paged._check_map
    out = paged.PageMap(vec(4), vec(3), vec(4, I64), vec(4), vec(4))
    monkeypatch.setattr(paged, "_check_map", lambda *a: runs.append(1) or check(*a))
    for n in (1, 900, 0, 37, 1000):
        paged.page_map(lens, lens, vec(n), table, 16, 4, out=out)
        assert paged.calls.pop()[2][4] == n
    assert len(runs) == 1
    # a single entry is contiguous whatever its stride, two are not
    one, two = vec(1, strides=(2,)), vec(2, strides=(2,))
    one._dense = True
    paged.page_map(lens, lens, one, table, 16, 4, out=out)
    with pytest.raises(ValueError, match="free_pages must be"):
        paged.page_map(lens, lens, two, table, 16, 4, out=out)
    with pytest.raises(ValueError, match="free_pages"):
        paged.page_map(lens, lens, vec(2 ** 31), table, 16, 4, out=out)


def test_new_shapes_do_not_drop_all_that_is_kept(paged):
    """Steps whose token counts vary: the checks of one shape make room for one other, not for all."""
    from test_paged_cpu import H16, I64, _Fake

    pool = _Fake((10, 8, 16, 128), H16)
    for n in range(1, 1300):
        kv = _Fake((n, 8, 128), H16)
        paged.paged_append(kv, kv, pool, pool, _Fake((n,), I64))
        assert len(paged._KEPT) == min(n, 1024)


def test_a_paged_cache_refuses_what_does_not_fit(monkeypatch):
    """More tokens than a request's table row holds would have nowhere to go: said before anything changes."""
    from e8_lattice_vector_gb300 import serve

    maps = []
    monkeypatch.setattr(serve, "page_map", lambda *a: maps.append(a))
    c = serve.PagedCache(1, 2, 1, 64, 16, 40, torch.float16, torch.device("cpu"))  # three pages each
    c.extend([40, 1])
    assert c.lengths == [40, 1] and c.free.numel() == 6 - 4 and len(maps) == 1
    for new in ([9, 0], [0, 48], [-1, 1], [1], [1, 1, 1]):
        with pytest.raises(ValueError):
            c.extend(new)
        assert c.lengths == [40, 1] and c.free.numel() == 2 and len(maps) == 1
    c.extend([8, 47])  # to the end of the pages
    assert c.lengths == [48, 48] and c.free.numel() == 0
    ctx, new, free, table, page, tokens = maps[-1]
    assert ctx.tolist() == [40, 1] and new.tolist() == [8, 47] and ctx.dtype == new.dtype == torch.int32
    assert free.numel() == 2 and (page, tokens) == (16, 55)


@pytest.mark.parametrize("dim,tokens,max_q,small", [(64, 95, 5, True), (96, 95, 5, True), (128, 95, 5, False), (128, 39, 8, True),
                                                    (128, 88, 8, False), (64, 97, 5, False), (64, 32, 1, True),
                                                    (128, 128, 4, True), (64, 39, 9, False)])
def test_which_kernel_takes_drafts(paged, dim, tokens, max_q, small):
    """32 requests, four query heads on a KV head: the large kernel's calls need scratch for its plan."""
    from test_paged_cpu import H16, I32, _Fake

    pool, table = _Fake((10, 8, 16, dim), H16), _Fake((32, 7), I32)
    q = _Fake((tokens, 32, dim), H16)
    need = paged._attention(q, q, pool, None, table, 32, max_q, None, 1, 0)[2]
    least = paged._attention(q, q, pool, None, table, 32, 1, None, 1, 0)[2]
    assert (need == least) == small
