"""The paged-cache operators against plain implementations: the page map and the append value by value, the
attention against its definition in 64 bits.

Attention tolerances are bounds, computed per element from the same 64-bit reference.  With u the unit roundoff of
the pool's type (2^-11 fp16, 2^-9 bf16), e = 2^-24 that of fp32, n keys and A = sum p |v| / l:
  a score is off by at most  S = (D + 4) e scale max_j sum_d |q_d k_jd|
  (products of two 16-bit values are exact in fp32; D additions, the scaling and the exponential's argument),
  so each p is off by a factor 1 +- (S + 4 e), p rounded to the pool's type by another u, and fp16 rounds a p below its
  normal range by up to 2^-25 of the largest; the sums of n terms in fp32 by (n + 8) e each, above and below the
  fraction; the output is rounded once by u, or by 2^-25 in fp16's subnormals.
  |out - exact| <= u |exact| + 2^-24 + A (u + 2 S + 2 (n + 8) e) (1 + u) + 2^-24 sum |v| / l
  |lse - exact| <= S + (n + 8) e + 4 e |exact|
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def nq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from e8_lattice_vector_gb300 import build as nqbuild

    nqbuild.build()
    import e8_lattice_vector_gb300 as nq

    return nq


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ page map


def ref_page_map(ctx, new, free, table, P, tokens):
    """Token by token, from the header's words."""
    table = table.copy()
    R, M = table.shape
    q_start, kv, slots, pos = [0], [], np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int32)
    taken = past = 0
    for r in range(R):
        c, n = max(ctx[r], 0), max(new[r], 0)
        held = min(-(-c // P), M)
        base = taken
        taken += min(-(-(c + n) // P), M) - held
        past += c + n > M * P
        for i in range(n):
            t, p = q_start[-1] + i, c + i
            if t >= tokens:
                break
            pos[t] = p
            col = p // P
            if col >= M:
                continue
            if col >= held:
                at = base + col - held
                page = int(free[at]) if at < len(free) else -1
                if p % P == 0:
                    table[r, col] = page
            else:
                page = int(table[r, col])
            slots[t] = page * P + p % P if page >= 0 else -1
        q_start.append(q_start[-1] + n)
        kv.append(c + n)
    counts = [q_start[-1], taken, max(taken - len(free), 0), past]
    return (np.array(q_start, np.int32), np.array(kv, np.int32), slots, pos, np.array(counts, np.int32), table)


def check_page_map(nq, ctx, new, P, cols=None, pad=0, n_free=None, seed=0, room=None, extra_stride=0):
    rng = np.random.default_rng(seed)
    R = len(ctx)
    if cols is None:
        cols = max([-(-(max(c, 0) + max(n, 0)) // P) for c, n in zip(ctx, new)] + [0]) + 2
    total = sum(max(n, 0) for n in new)
    tokens = total + pad if room is None else room
    need = total + R if n_free is None else n_free
    free = rng.permutation(need + 7).astype(np.int32)[:need]
    table = rng.integers(-1, 50, (R, cols + extra_stride)).astype(np.int32)
    full = torch.tensor(table, device=DEV)
    dev_table = full[:, :cols]
    m = nq.page_map(_i32(ctx), _i32(new), torch.tensor(free, device=DEV), dev_table, P, tokens)
    ref = ref_page_map(ctx, new, free, table[:, :cols], P, tokens)
    for name, got, want in zip(("q_start", "kv_lens", "slots", "positions", "counts", "table"),
                               (m.q_start, m.kv_lens, m.slots, m.positions, m.counts, dev_table), ref):
        assert np.array_equal(got.cpu().numpy(), want), name
    assert np.array_equal(full[:, cols:].cpu().numpy(), table[:, cols:])  # nothing past the columns


@pytest.mark.parametrize("P", [16, 64, 256])
def test_page_map_mixed_lengths(nq, P):
    rng = np.random.default_rng(P)
    ctx = [0, 1, P - 1, P, P + 1, 5 * P, 1000, 0, 17, 3]
    new = [1, 1, 1, 1, 2 * P, 0, 333, 0, 5 * P + 3, 1]
    check_page_map(nq, ctx, new, P, pad=5, extra_stride=3)
    check_page_map(nq, [int(v) for v in rng.integers(0, 400, 77)], [int(v) for v in rng.integers(0, 60, 77)], P)


@pytest.mark.parametrize("R", [1, 511, 512, 513, 1025, 3000])
def test_page_map_many_requests(nq, R):
    """Request counts around the 512-request chunks of the scan, decode steps and ragged chunks."""
    rng = np.random.default_rng(R)
    ctx = [int(v) for v in rng.integers(0, 3000, R)]
    check_page_map(nq, ctx, [1] * R, 16, pad=3, seed=R)
    check_page_map(nq, ctx, [int(v) for v in rng.integers(0, 9, R)], 32, seed=R)


def test_page_map_long_prompts_and_empty_steps(nq):
    check_page_map(nq, [0, 70], [40000, 3], 16)
    check_page_map(nq, [], [], 16, cols=4, pad=3)
    check_page_map(nq, [5, 0], [0, 0], 16, pad=2)
    check_page_map(nq, [5, 0], [0, 0], 16)
    check_page_map(nq, [-4, 7], [3, -2], 16)


def test_page_map_exhausted_free_list_table_and_room(nq):
    ctx, new = [0, 10, 100, 0], [40, 30, 90, 17]
    for n_free in (0, 1, 5, 8):
        check_page_map(nq, ctx, new, 16, n_free=n_free)
    check_page_map(nq, ctx, new, 16, cols=3)
    check_page_map(nq, ctx, new, 16, cols=0)
    for room in (0, 1, 39, 41, 100):
        check_page_map(nq, ctx, new, 16, room=room)


def test_page_map_sums_past_31_bits(nq):
    big = 2 ** 31 - 1
    m = nq.page_map(_i32([big, 5, 0]), _i32([1, big, big]), _i32([3]), torch.full((3, 2), -1, dtype=torch.int32, device=DEV),
                    16, 4)
    assert m.q_start.tolist() == [0, 1, big, big] and m.kv_lens.tolist() == [big, big, big]
    assert m.positions.tolist() == [big, 5, 6, 7] and m.slots.tolist() == [-1, -1, -1, -1]
    # request 1 holds column 0 (entry -1) and asks for column 1; request 2 asks for both its columns
    assert m.counts.tolist() == [big, 3, 2, 3]


# -------------------------------------------------------------------- append


def _pool(pages, heads, P, D, dtype, layout, fill=None):
    shape = {"hnd": (pages, heads, P, D), "nhd": (pages, P, heads, D), "slice": (2, pages, heads, P, D),
             "packed": (pages, 2, heads, P, D)}[layout]
    x = torch.randn(shape, device=DEV).to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype, device=DEV)
    if layout == "nhd":
        return x.transpose(1, 2)
    return x[1] if layout == "slice" else x[:, 1] if layout == "packed" else x


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "slice", "packed"])
@pytest.mark.parametrize("tokens,heads,P,source", [(1, 1, 16, "plain"), (77, 3, 16, "head_major"),
                                                   (300, 8, 64, "fused"), (33, 2, 256, "plain")])
def test_append(nq, dtype, D, layout, tokens, heads, P, source):
    torch.manual_seed(tokens + D)
    pages = -(-tokens // P) * 2 + 1
    Kp, Vp = _pool(pages, heads, P, D, dtype, layout), _pool(pages, heads, P, D, dtype, layout)
    if source == "plain":
        K, V = (torch.randn(tokens, heads, D, device=DEV).to(dtype) for _ in range(2))
    elif source == "head_major":
        K, V = (torch.randn(heads, tokens, D, device=DEV).to(dtype).transpose(0, 1) for _ in range(2))
    else:  # columns of one projection's output
        x = torch.randn(tokens, 4 * heads, D, device=DEV).to(dtype)
        K, V = x[:, 2 * heads:3 * heads], x[:, 3 * heads:]
    slots = torch.randperm(pages * P, device=DEV)[:tokens]
    if tokens > 10:
        slots[3], slots[5], slots[7], slots[9] = -1, pages * P, 2 ** 40, -2 ** 50
    want = []
    for pool, src in ((Kp, K), (Vp, V)):
        ref = pool.cpu().clone()
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < pages * P:
                ref[s // P, :, s % P] = src[t].cpu()
        want.append(ref)
    got = nq.paged_append(K, V, Kp, Vp, slots)
    assert got[0] is Kp and got[1] is Vp
    for g, w in zip(got, want):
        assert torch.equal(g.cpu().view(torch.int16), w.view(torch.int16))


def test_append_nothing(nq):
    Kp, Vp = _pool(2, 1, 16, 64, torch.float16, "hnd"), _pool(2, 1, 16, 64, torch.float16, "hnd")
    before = Kp.clone()
    e = torch.empty(0, 1, 64, dtype=torch.float16, device=DEV)
    nq.paged_append(e, e, Kp, Vp, torch.empty(0, dtype=torch.int64, device=DEV))
    assert torch.equal(Kp, before)


def test_append_offsets_past_32_bits(nq):
    """A pool of more than 2^32 bytes (and 2^31 elements): rows at its far end."""
    heads, P, D = 8, 256, 128
    pages = 2 ** 31 // (heads * P * D) + 5
    Kp = torch.zeros(pages, heads, P, D, dtype=torch.float16, device=DEV)
    K = torch.randn(3, heads, D, device=DEV).half()
    slots = torch.tensor([pages * P - 1, 0, (pages - 2) * P + 5], device=DEV)
    nq.paged_append(K, K, Kp, Kp, slots)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(Kp[s // P, :, s % P], K[t])
    assert int(Kp.count_nonzero()) == int(K.count_nonzero())


# ----------------------------------------------------------------- attention


class Step:
    """A step's tensors: pages in random order, NaN and infinities in every slot that no row may see, wild
    entries in the table's unused columns."""

    def __init__(self, lens, heads, kv_heads, D, P, dtype, layout="hnd", seed=0, q_layout="plain", cols=None,
                 holes=(), mult=1.5):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.lens, self.heads, self.kv_heads, self.D, self.P, self.dtype = lens, heads, kv_heads, D, P, dtype
        kv = [c + n for c, n in lens]
        R = len(lens)
        need = [-(-k // P) for k in kv]
        self.cols = max(need + [0]) + 2 if cols is None else cols
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).cpu().tolist()
        self.table = torch.randint(-(2 ** 31), 2 ** 31, (R, self.cols), generator=g, device=DEV).to(torch.int32)
        self.Kp = _pool(pages, kv_heads, P, D, dtype, layout, float("nan"))
        self.Vp = _pool(pages, kv_heads, P, D, dtype, layout, float("inf"))
        self.k, self.v, at = [], [], 0
        for r in range(R):
            k = (torch.randn(kv[r], kv_heads, D, generator=g, device=DEV) * mult).to(dtype)
            v = torch.randn(kv[r], kv_heads, D, generator=g, device=DEV).to(dtype)
            self.k.append(k)
            self.v.append(v)
            for c in range(min(need[r], self.cols)):
                page = order[at]
                at += 1
                n = min(P, kv[r] - c * P)
                self.Kp[page, :, :n] = k[c * P: c * P + n].transpose(0, 1)
                self.Vp[page, :, :n] = v[c * P: c * P + n].transpose(0, 1)
                self.table[r, c] = page
        self.hidden = set(holes)  # (request, column): a page that is not in the pool
        for i, (r, c) in enumerate(holes):
            self.table[r, c] = [-1, pages, 2 ** 31 - 1, -(2 ** 31)][i % 4]
        T = sum(n for _, n in lens)
        self.tokens = T
        if q_layout == "plain":
            self.Q = torch.randn(T, heads, D, generator=g, device=DEV).to(dtype)
        elif q_layout == "fused":
            self.Q = torch.randn(T, heads + 2 * kv_heads, D, generator=g, device=DEV).to(dtype)[:, :heads]
        else:
            self.Q = torch.randn(heads, T, D, generator=g, device=DEV).to(dtype).transpose(0, 1)
        self.q_start = _i32(np.concatenate([[0], np.cumsum([n for _, n in lens])]).tolist())
        self.kv_lens = _i32(kv)
        self.max_q = max([n for _, n in lens] + [0])

    def reference(self, causal, window, scale):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
        T, H, D, G = self.tokens, self.heads, self.D, self.heads // self.kv_heads
        u = 2.0 ** -11 if self.dtype == torch.float16 else 2.0 ** -9
        out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
        tol = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
        lse = torch.full((T, H), -float("inf"), dtype=torch.float64, device=DEV)
        tol_lse = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        t0 = 0
        for r, (c, n) in enumerate(self.lens):
            L = min(c + n, self.cols * self.P)
            rows = slice(t0, t0 + n)
            t0 += n
            if n == 0 or L == 0:
                continue
            j = torch.arange(L, device=DEV)
            i = torch.arange(L - n, L, device=DEV)[:, None]
            seen = torch.ones(n, L, dtype=torch.bool, device=DEV)
            if causal:
                seen &= j[None] <= i
            if window:
                seen &= j[None] > i - window
            for (hr, hc) in self.hidden:
                if hr == r:
                    seen[:, hc * self.P: (hc + 1) * self.P] = False
            k = self.k[r][:L].double().repeat_interleave(G, 1)
            v = self.v[r][:L].double().repeat_interleave(G, 1)
            q = self.Q[rows].double()
            s = torch.einsum("thd,jhd->thj", q, k) * scale
            mag = torch.einsum("thd,jhd->thj", q.abs(), k.abs()) * scale
            s = s.masked_fill(~seen[:, None], -float("inf"))
            mag = mag.masked_fill(~seen[:, None], 0.0)
            m = s.amax(-1, keepdim=True)
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            some = l > 0
            w = torch.where(some, p / l, torch.zeros_like(p))
            o = torch.einsum("thj,jhd->thd", w, v)
            A = torch.einsum("thj,jhd->thd", w, v.abs())
            sv = torch.einsum("thj,jhd->thd", seen[:, None].expand_as(w).double(), v.abs())
            S = (D + 4) * E32 * mag.amax(-1, keepdim=True)
            cnt = (L + 8) * E32
            out[rows] = o
            tol[rows] = u * o.abs() + 2.0 ** -24 + A * (u + 2 * S + 2 * cnt) * (1 + u) + \
                torch.where(some, 2.0 ** -24 * sv / l.clamp(min=1e-30), torch.zeros_like(sv))
            ls = m + torch.log(l)
            lse[rows] = ls.squeeze(-1)
            tol_lse[rows] = (S + cnt + 4 * E32 * torch.where(some, ls, torch.zeros_like(ls)).abs()).squeeze(-1)
        return out, lse, tol, tol_lse

    def check(self, nq, causal=True, window=0, scale=None, max_q="exact", with_lse=True, out=None, ws=None):
        kw = {} if max_q is None else {"max_q": self.max_q if max_q == "exact" else max_q}
        lse = torch.full((self.tokens, self.heads), 7.0, device=DEV) if with_lse else None
        got = nq.paged_attention(self.Q, self.Kp, self.Vp, self.table, self.q_start, self.kv_lens, scale=scale,
                                 causal=causal, window=window, lse=lse, out=out, ws=ws, **kw)
        o = got[0] if with_lse else got
        ref, ref_lse, tol, tol_lse = self.reference(causal, window, self.D ** -0.5 if scale is None else scale)
        err = (o.double() - ref).abs()
        assert bool(torch.isfinite(o).all()), "an output is not finite"
        assert bool((err <= tol).all()), "out: worst error / tolerance %.3g" % float((err / tol).max())
        if with_lse:
            none = torch.isinf(ref_lse)
            assert torch.equal(torch.isinf(lse), none) and bool((lse[none] < 0).all())
            err = (lse.double() - ref_lse).abs()[~none]
            assert bool((err <= tol_lse[~none]).all()), \
                "lse: worst error / tolerance %.3g" % float((err / tol_lse[~none]).max())
        return o


TYPES = [torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("new", [1, 7, 150])
def test_attention_types_dims_pages(nq, dtype, D, P, new):
    """Every type, head_dim and page size, for single tokens, short chunks and chunks past one row tile; contexts that
    end inside a page, at its end and just after it, none and one token among them."""
    lens = [(c, new) for c in (0, 1, P - 1, P, 3 * P + 5, 700)]
    Step(lens, 8, 2, D, P, dtype, seed=P + new).check(nq)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (3, 1), (10, 2), (7, 1), (16, 2), (24, 1), (40, 8), (96, 2)])
@pytest.mark.parametrize("new", [1, 5, 70])
def test_attention_head_groups(nq, dtype, heads, kv_heads, new):
    """Heads that do and do not divide a row tile, up to 48 query heads on a KV head."""
    Step([(333, new), (64, 1), (0, new)], heads, kv_heads, 128, 16, dtype, seed=heads).check(nq)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "slice", "packed"])
@pytest.mark.parametrize("q_layout", ["plain", "fused", "head_major"])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_strides(nq, layout, q_layout, new):
    s = Step([(100, new), (517, new)], 6, 2, 96, 32, torch.float16, layout, 3, q_layout)
    wide = torch.full((s.tokens, 3, s.heads, s.D), 5.0, dtype=torch.float16, device=DEV)
    s.check(nq, out=wide[:, 1])
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 2] == 5).all())


@pytest.mark.parametrize("window", [1, 2, 15, 64, 130, 1000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [1, 6, 300])
def test_attention_windows(nq, window, causal, new):
    Step([(0, new), (900, new), (129, new), (128, new)], 4, 2, 64, 16, torch.bfloat16, seed=window).check(
        nq, causal=causal, window=window)


@pytest.mark.parametrize("new", [1, 3, 200])
def test_attention_without_causal_mask(nq, new):
    Step([(0, new), (250, new), (1000, new)], 8, 8, 128, 64, torch.float16, seed=new).check(nq, causal=False)


@pytest.mark.parametrize("max_q", ["exact", None, 0, 1, 10 ** 6])
def test_attention_bound_on_rows_changes_no_result(nq, max_q):
    """Whatever bound is given, the right one or not."""
    Step([(500, 1), (30, 90), (0, 17), (77, 0), (1200, 4)], 8, 2, 128, 16, torch.float16, seed=5).check(nq, max_q=max_q)


@pytest.mark.parametrize("new", [1, 130])
def test_attention_requests_without_rows_or_keys(nq, new):
    Step([(0, 0), (10, 0), (0, new), (40, 0), (0, 0), (5, new), (0, 0)], 4, 1, 64, 16, torch.float16).check(nq)


def test_attention_nothing_to_do(nq):
    s = Step([(10, 0), (0, 0)], 4, 1, 64, 16, torch.float16)
    assert s.check(nq).shape[0] == 0
    s = Step([], 4, 1, 64, 16, torch.float16)
    assert s.check(nq).shape[0] == 0


@pytest.mark.parametrize("new", [1, 9, 140])
def test_attention_rows_that_see_nothing(nq, new):
    """More rows than keys (positions below zero), pages outside the pool, and both."""
    s = Step([(64, new), (300, new), (16, new), (128, new)], 8, 2, 128, 16, torch.float16, seed=new,
             holes=[(0, c) for c in range((64 + new + 15) // 16)] + [(1, 0), (1, 7), (1, 8), (3, 1), (3, 2), (3, 8)])
    s.check(nq)
    s.check(nq, window=16)
    # lengths shorter than the rows: rows before position 0 see nothing under the causal mask
    s = Step([(0, new + 20), (0, new + 20)], 8, 2, 128, 16, torch.bfloat16, seed=new)
    short = [new + 20 - 15, 0]
    s.kv_lens = _i32(short)
    lse = torch.empty(s.tokens, 8, device=DEV)
    o, _ = nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=s.max_q, lse=lse)
    n = new + 20
    assert bool((o[:15] == 0).all()) and bool((o[n:] == 0).all())
    assert bool((lse[:15] == -float("inf")).all()) and bool((lse[n:] == -float("inf")).all())
    assert bool(torch.isfinite(lse[15:n]).all())
    # row 15 sees key 0 alone
    assert torch.equal(o[15], s.v[0][0].repeat_interleave(4, 0))


@pytest.mark.parametrize("new", [1, 60])
def test_attention_lengths_past_the_table(nq, new):
    """A length that the table's columns cannot hold is cut to what they hold."""
    s = Step([(400, new), (100, new)], 4, 2, 64, 16, torch.float16, cols=20)
    s.check(nq)


@pytest.mark.parametrize("new", [1, 33])
def test_attention_values_in_device_data_are_clamped(nq, new):
    """Row starts and lengths outside their ranges reach no memory outside the buffers and leave other
    requests' rows right."""
    s = Step([(50, new), (60, new), (70, new)], 4, 2, 64, 16, torch.float16)
    want = s.check(nq)
    T = s.tokens
    guard = torch.full((T + 8, 4, 64), 3.0, dtype=torch.float16, device=DEV)
    out = guard[4:T + 4]
    for starts, kv, right in (([-7, new, 2 * new, 2 ** 31 - 1], None, [1, 2]),
                              ([0, new, 2 * new, 3 * new], [-5, None, 2 ** 31 - 1], [1])):
        q_start = _i32(starts)
        lens = [v if kv is None or kv[i] is None else kv[i] for i, v in enumerate(s.kv_lens.tolist())]
        s.table[2, -1] = s.table[2, 0]
        nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, q_start, _i32(lens), max_q=new, out=out)
        for r in right:
            assert torch.equal(out[r * new:(r + 1) * new], want[r * new:(r + 1) * new])
        assert bool((guard[:4] == 3).all()) and bool((guard[T + 4:] == 3).all())


def test_attention_leaves_rows_of_no_request(nq):
    s = Step([(50, 2), (300, 3)], 4, 2, 64, 16, torch.float16)
    pad = torch.cat([s.Q, s.Q[:2]])
    out = torch.full_like(pad, 9.0)
    lse = torch.full((7, 4), 9.0, device=DEV)
    nq.paged_attention(pad, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=3, out=out, lse=lse)
    assert torch.equal(out[:5], s.check(nq)) and bool((out[5:] == 9).all()) and bool((lse[5:] == 9).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 20, 200])
def test_attention_long_contexts(nq, dtype, new):
    """Contexts that are split over the GPU and joined, alone and beside short ones."""
    Step([(9000, new)], 8, 2, 128, 64, dtype, seed=1).check(nq)
    Step([(20000, new), (3, new), (511, new), (0, new), (4000, 1)], 2, 1, 64, 16, dtype, seed=2).check(nq)


def test_attention_many_requests(nq):
    """More requests than threads of a block, and more row tiles than multiprocessors."""
    rng = np.random.default_rng(0)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(0, 90, 700), rng.integers(0, 3, 700))]
    Step(lens, 4, 2, 64, 16, torch.float16, seed=8).check(nq)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(0, 50, 400), rng.integers(0, 70, 400))]
    Step(lens, 4, 2, 64, 16, torch.bfloat16, seed=9).check(nq)


@pytest.mark.parametrize("new", [1, 64])
def test_attention_large_and_tiny_scores(nq, new):
    """Scores of thousands (one key takes all), equal scores, and a scale near zero."""
    Step([(300, new)], 4, 2, 128, 16, torch.float16, mult=300.0, seed=1).check(nq)
    s = Step([(300, new)], 4, 2, 128, 16, torch.float16, seed=2)
    s.check(nq, scale=1e-6)
    s.check(nq, scale=4.0)
    s.Q.zero_()
    s.check(nq)


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_attention_largest_values(nq, new, dtype):
    """Keys and queries of the type's largest magnitude: scores that fp32 holds in fp16 only.  One key wins, and
    its value comes out."""
    s = Step([(200, new)], 2, 1, 64, 16, dtype, seed=4, mult=0.0)
    big = 65504.0 if dtype == torch.float16 else 2.0 ** 60
    s.Q.fill_(big)
    low, top = 37, 150
    for key, val in ((low, -big), (top, big)):
        page = int(s.table[0, key // 16])
        s.Kp[page, :, key % 16] = val
    out = nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=new)
    assert torch.equal(out, s.v[0][top].expand_as(out[:, :1]).expand_as(out))


@pytest.mark.parametrize("new", [1, 100])
def test_attention_rising_scores(nq, new):
    """Every key scores above all before it, so the running maximum moves on in each tile: by a little and by much."""
    for step in (0.01, 1.0, 40.0):
        s = Step([(1500, new)], 2, 1, 64, 32, torch.float16, seed=6)
        L = 1500 + new
        ramp = torch.arange(L, device=DEV).float() * (step / 40)
        s.k[0] = (torch.ones(L, 1, 64, device=DEV) * ramp[:, None, None] / 8).half()
        for j in range(-(-L // 32)):
            n = min(32, L - 32 * j)
            s.Kp[int(s.table[0, j]), :, :n] = s.k[0][32 * j:32 * j + n].transpose(0, 1)
        s.Q.fill_(1.0)
        s.check(nq)


@pytest.mark.parametrize("new", [1, 6, 300])
def test_attention_repeats_bit_for_bit(nq, new):
    s = Step([(5000, new), (100, new), (2500, new)], 8, 2, 128, 16, torch.bfloat16, seed=7)
    first = s.check(nq)
    ws = nq.paged_attention_workspace(s.Q, s.Kp, s.table)
    if ws is not None:
        ws.fill_(255)  # NaN everywhere: nothing in the scratch has to start at zero
    for _ in range(3):
        assert torch.equal(first, s.check(nq, ws=ws, with_lse=False))


@pytest.mark.parametrize("new", [1, 50])
def test_attention_offsets_past_32_bits(nq, new):
    """Pages past 2^32 bytes of the pool (and 2^31 elements)."""
    s = Step([(800, new)], 4, 2, 128, 256, torch.float16, seed=3)
    pages = 2 ** 31 // (2 * 256 * 128) + 40
    big = [torch.zeros(pages, 2, 256, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    need = -(-(800 + new) // 256)
    for c in range(need):
        at = int(s.table[0, c])
        far = pages - 1 - 3 * c
        big[0][far], big[1][far] = s.Kp[at], s.Vp[at]
        s.table[0, c] = far
    s.Kp, s.Vp = big
    s.check(nq)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_on_another_stream(nq, new):
    s = Step([(3000, new), (40, new)], 8, 2, 128, 16, torch.float16, seed=3)
    want = s.check(nq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=s.max_q) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_step_in_a_cuda_graph(nq):
    """Map, append and attention captured once; replayed with new lengths and values."""
    R, P, H, D, cols = 5, 16, 2, 64, 12
    dev = torch.device(DEV)
    free, table = torch.arange(60, dtype=torch.int32, device=dev), torch.full((R, cols), -1, dtype=torch.int32, device=dev)
    ctx, new = _i32([0] * R), _i32([1] * R)
    K, V = (torch.randn(16, H, D, device=dev).half() for _ in range(2))
    Q = torch.randn(16, 4, D, device=dev).half()
    Kp, Vp = (torch.zeros(60, H, P, D, dtype=torch.float16, device=dev) for _ in range(2))
    m = nq.PageMap.empty(R, 16, dev)
    out = torch.zeros_like(Q)
    ws = nq.paged_attention_workspace(Q, Kp, table)

    def step():
        nq.page_map(ctx, new, free, table, P, 16, out=m)
        nq.paged_append(K, V, Kp, Vp, m.slots)
        nq.paged_attention(Q, Kp, Vp, table, m.q_start, m.kv_lens, max_q=16, out=out, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([3, 1, 5, 0, 2], [1, 1, 1, 1, 1], [0, 9, 0, 0, 7]):
        new.copy_(_i32(lens))
        K.normal_()
        Q.normal_()
        table.fill_(-1)
        graph.replay()
        got = out.clone()
        table.fill_(-1)
        Kp.zero_()
        out.zero_()
        step()
        n = sum(lens)
        assert torch.equal(got[:n], out[:n])
        # lengths start at zero: a request's first row sees its own key alone
        first = int(m.q_start[1]) if lens[0] == 0 else 0
        assert torch.equal(out[first], V[first].repeat_interleave(2, 0))


def test_no_wait_was_given_up(nq):
    """After everything above: no kernel gave up a wait for its loads."""
    nq.paged_status()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,window", [(128, 0), (128, 700), (64, 700), (96, 0)])
@pytest.mark.parametrize("new", [5, 20, 50])
def test_attention_many_pieces_in_every_block(nq, dtype, D, window, new):
    """Blocks that work through several row tiles, whole ones and parts, of one half's rows and of two."""
    rng = np.random.default_rng(new)
    lens = [(int(c), int(n)) for c, n in zip(rng.integers(300, 2500, 60), rng.integers(1, new + 1, 60))]
    Step(lens, 16, 4, D, 32, dtype, seed=new).check(nq, window=window)


@pytest.mark.parametrize("config,kw", [("tiny", {"steps": 3, "new": 1}), ("tiny", {"steps": 2, "new": 20, "page_size": 32}),
                                       ("phi3mini", {"layers": 2, "tokens": 300, "q_heads": 32, "steps": 2, "new": 3})])
def test_serving_from_a_compressed_cache(nq, config, kw):
    """Compressed, decompressed, paged and attended to: the outputs differ from those over the original cache, by less than
    the values do (three bits for keys and two for values leave about a quarter of a value's size as noise)."""
    from e8_lattice_vector_gb300.serve import serve
    from e8_lattice_vector_gb300.synth import CONFIGS

    r = serve(CONFIGS[config], **kw)
    assert 0.01 < r["attention_rel_error"] < 1.0 and 0.1 < r["compressed_share"] < 0.3
    nq.paged_status()


def test_paged_pools_hold_what_was_decompressed(nq):
    """fill() puts every row of a decompressed cache where the table says."""
    from e8_lattice_vector_gb300.serve import PagedCache

    K, V = (torch.randn(2, 3, 2, 70, 64, device=DEV).half() for _ in range(2))
    c = PagedCache(2, 3, 2, 64, 16, 80, torch.float16, torch.device(DEV, 0))
    c.fill(K, V)
    for pool, src in ((c.K, K), (c.V, V)):
        for r in range(3):
            for t in (0, 15, 16, 69):
                page = int(c.table[r, t // 16])
                assert torch.equal(pool[:, page, :, t % 16], src[:, r, :, t])


def test_append_repeated_rows(nq):
    """One K and V row for every head (a head stride of zero)."""
    Kp, Vp = (torch.zeros(2, 4, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2))
    K = torch.randn(5, 1, 64, device=DEV).half().expand(5, 4, 64)
    nq.paged_append(K, K, Kp, Vp, torch.arange(5, device=DEV) + 14)
    assert torch.equal(Kp[0, :, 14], K[0]) and torch.equal(Kp[1, :, :3].transpose(0, 1), K[2:]) and torch.equal(Kp, Vp)


@pytest.mark.parametrize("heads,kv_heads", [(100, 1), (128, 1), (130, 1), (520, 2)])
@pytest.mark.parametrize("new", [1, 9])
def test_attention_heads_around_a_half(nq, heads, kv_heads, new):
    """Query heads on one KV head that nearly fill, fill and pass the 128 rows of a half."""
    Step([(300, new), (0, new), (17, 1)], heads, kv_heads, 64, 16, torch.float16, seed=heads).check(nq)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_table_without_columns(nq, new):
    s = Step([(0, new), (20, new)], 4, 2, 64, 16, torch.float16, cols=0)
    out, lse = nq.paged_attention(s.Q, s.Kp, s.Vp, s.table, s.q_start, s.kv_lens, max_q=new,
                                  lse=torch.zeros(s.tokens, 4, device=DEV))
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_mostly_single_tokens(nq, dtype):
    """Batches that are shared between the kernels, and batches of drafts of which some need a second tile."""
    rng = np.random.default_rng(3)
    lens = [(int(c), 1) for c in rng.integers(0, 3000, 30)] + [(1000, 200), (50, 3), (0, 0), (777, 16)]
    Step(lens, 8, 2, 128, 16, dtype, seed=5).check(nq)
    Step(lens, 8, 2, 64, 64, dtype, seed=6).check(nq, window=500)
    drafts = [(int(c), int(n)) for c, n in zip(rng.integers(0, 2000, 25), rng.integers(1, 5, 25))] + [(600, 8)]
    Step(drafts, 16, 4, 128, 32, dtype, seed=7).check(nq)
