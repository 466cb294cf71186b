"""The paged operators at the edges of what callers may pass, against the same 64-bit reference as test_paged_gpu."""
import pytest
import torch

from test_paged_gpu import DEV, E32, TYPES, Step, _i32, nq  # noqa: F401  (nq is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [0, 16, 48, 240])
@pytest.mark.parametrize("new", [1, 20, 200])
def test_attention_scratch_on_any_16_byte_boundary(nq, new, offset):
    """Row tiles shared between blocks leave their parts in the caller's scratch, wherever that begins; a buffer of exactly the
    size that is asked for, with guards around it."""
    s = Step([(9000, new), (30, 1)], 8, 2, 128, 64, torch.float16, seed=1)
    want = s.check(nq)
    need = nq.paged_attention_workspace(s.Q, s.Kp, s.table, max_q=s.max_q).numel()
    guarded = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    ws = guarded[offset:offset + need]
    assert ws.data_ptr() % 256 == offset
    assert torch.equal(s.check(nq, ws=ws), want)
    assert bool((guarded[:offset] == 255).all()) and bool((guarded[offset + need:] == 255).all())


@pytest.mark.parametrize("max_q", [None, 1])
@pytest.mark.parametrize("T", [40, 900])
def test_attention_row_starts_that_decrease(nq, T, max_q):
    """Rows that two requests claim hold one's results; a request after a larger start keeps what nobody has claimed.  Scratch of
    exactly its size, between guards."""
    s = Step([(700, T), (300, T), (500, T)], 8, 2, 128, 16, torch.float16, seed=T)
    Q = s.Q[:T]
    for starts, claims in (([0, T, 0, T], {0: (0, T), 2: (0, T)}), ([T, 0, T, 0], {1: (0, T)}), ([0, T, T, 0], {0: (0, T)}),
                           ([T - 10, T, 0, T - 10], {0: (T - 10, T), 2: (0, T - 10)})):
        need = nq.paged_attention_workspace(Q, s.Kp, s.table, max_q=max_q).numel()
        guarded = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
        out = torch.full_like(Q, 77.0)
        nq.paged_attention(Q, s.Kp, s.Vp, s.table, _i32(starts), s.kv_lens, max_q=max_q, out=out, ws=guarded[:need])
        assert bool((guarded[need:] == 255).all())
        ok = torch.zeros_like(out, dtype=torch.bool)
        for r, (b, e) in claims.items():
            want = nq.paged_attention(Q[b:e], s.Kp, s.Vp, s.table[r:r + 1], _i32([0, e - b]), s.kv_lens[r:r + 1], max_q=max_q)
            # the same sums in another order of parts: each side within its own bound of the exact ones
            L, v = int(s.kv_lens[r]), s.v[r].float().abs().max()
            S = (128 + 4) * E32 * 128 ** -0.5 * Q.float().norm(dim=-1).max() * s.k[r].float().norm(dim=-1).max()
            tol = 2 * (2.0 ** -11 * want.float().abs() + 2.0 ** -24 * (L + 1) + v * (2.0 ** -11 + 2 * S + 2 * (L + 8) * E32))
            ok[b:e] |= (out[b:e].float() - want.float()).abs() <= tol
        if starts[0] == T - 10:  # the later request's rows lie before the earlier one's: they may be left
            ok |= out == 77
        assert bool(ok.all())
    nq.paged_status()


def check_weights(nq, s, scale, new, copies=1):
    """One request's causal rows (all of `copies` requests over the same pages) against 64 bits, by a bound in which the weights have their own roundoff.  With u the type's
    unit roundoff (2^-11 fp16, 2^-8 bf16) and w the weights' (2^-11; 2^-17 in bf16, where they are the sum of two):
      |out - exact| <= u |exact| + 2^-25 + A (w + 2 S + 2 (n + 8) e) (1 + u) + 2^-32 sum |v| / l
    S, A, l, n and e as in test_paged_gpu; the last term, fp16's alone, is a weight below fp16's normal range: off by 2^-25 when
    the largest is 2^7 at least."""
    half = s.dtype == torch.float16
    u, w = (2.0 ** -11, 2.0 ** -11) if half else (2.0 ** -8, 2.0 ** -17)
    G, D, L = s.heads // s.kv_heads, s.D, s.k[0].shape[0]
    lse = torch.empty(copies * new, s.heads, device=DEV)
    starts = torch.arange(copies + 1, dtype=torch.int32, device=DEV) * new
    out, _ = nq.paged_attention(s.Q.repeat(copies, 1, 1), s.Kp, s.Vp, s.table.repeat(copies, 1), starts,
                                s.kv_lens.repeat(copies), max_q=new, scale=scale, lse=lse)
    for i in range(1, copies):
        assert torch.equal(out[i * new:(i + 1) * new], out[:new]) and torch.equal(lse[i * new:(i + 1) * new], lse[:new])
    out, lse = out[:new], lse[:new]
    hidden = torch.arange(L, device=DEV)[None] > torch.arange(L - new, L, device=DEV)[:, None]
    for h in range(s.heads):
        q, k, v = s.Q[:, h].double(), s.k[0][:, h // G].double(), s.v[0][:, h // G].double()
        x = (q @ k.T * scale).masked_fill(hidden, -float("inf"))
        p = torch.exp(x - x.amax(-1, keepdim=True))
        l = p.sum(-1, keepdim=True)
        exact, A = p @ v / l, p @ v.abs() / l
        S = (D + 4) * E32 * scale * (q.abs() @ k.abs().T).masked_fill(hidden, 0.0).amax(-1, keepdim=True)
        tol = u * exact.abs() + 2.0 ** -25 + A * (w + 2 * S + 2 * (L + 8) * E32) * (1 + u)
        if half:
            tol += 2.0 ** -32 * (~hidden).double() @ v.abs() / l
        err = (out[:, h].double() - exact).abs()
        assert bool((err <= tol).all()), "out: worst error / tolerance %.3g" % float((err / tol).max())
        z = torch.logsumexp(x, -1)
        err, tol = (lse[:, h].double() - z).abs(), S.squeeze(-1) + (L + 8) * E32 + 4 * E32 * z.abs()
        assert bool((err <= tol).all()), "lse: worst error / tolerance %.3g" % float((err / tol).max())


def put_keys(s, k, v):
    """New keys and values for the single request of a step."""
    s.k[0], s.v[0] = k.to(s.dtype), v.to(s.dtype)
    for c in range(-(-len(k) // s.P)):
        n = min(s.P, len(k) - c * s.P)
        page = int(s.table[0, c])
        s.Kp[page, :, :n] = s.k[0][c * s.P:c * s.P + n].transpose(0, 1)
        s.Vp[page, :, :n] = s.v[0][c * s.P:c * s.P + n].transpose(0, 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("place", [0, 70000, 131000])
@pytest.mark.parametrize("gap", [5.5, 10.0, 14.0, 17.0, 17.5, 20.0])
def test_attention_one_key_far_above_a_long_context(nq, dtype, new, place, gap):
    """One key that takes most of the weight, and very many that share a small part of it, which their values make the whole
    result: no weight may be lost, nor all of them rounded one way.  As many requests as the grid has blocks, each of which
    then has a whole context and one running maximum for it (the small kernel: one for each of its warps)."""
    L = 131072
    s = Step([(L - new, new)], 4, 1, 64, 256, dtype, seed=3)
    s.Q.fill_(1.0)
    k, v = torch.zeros(L, 1, 64, device=DEV), torch.rand(L, 1, 64, device=DEV) + 0.5
    k[place], v[place] = gap / 64, 0.0
    put_keys(s, k, v)
    check_weights(nq, s, 1.0, new, copies=152)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_weights_have_their_bits(nq, dtype, new, D):
    """Few keys of equal size, whose weights are not powers of two, and values of the largest magnitude: the weights' own
    roundoff, and no overflow in the sums."""
    for L, big in ((new + 2, 1.0), (3000, 1.0), (3000, 60000.0)):
        s = Step([(L - new, new)], 4, 2, D, 16, dtype, seed=L)
        put_keys(s, torch.randn(L, 2, D, device=DEV) * 0.4, (torch.rand(L, 2, D, device=DEV) + 0.05) * big)
        check_weights(nq, s, D ** -0.5, new)


def test_waits_are_limited_and_end_soon_after_another(nq, tmp_path):
    """A barrier that nothing completes: a wait gives up after its limit and says so, and when another thread has given up it
    returns within 0.1 ms."""
    import ctypes
    import os
    import subprocess

    from e8_lattice_vector_gb300 import build as nqbuild

    here = os.path.dirname(os.path.abspath(__file__))
    so = str(tmp_path / "paged_waits.so")
    subprocess.run([nqbuild._nvcc()] + nqbuild.NVCC_FLAGS + ["-shared", os.path.join(here, "paged_waits.cu"), "-o", so], check=True)
    call, result = ctypes.CDLL(so).wait_for_nothing_once, torch.zeros(3, dtype=torch.int64, device=DEV)
    assert call(0, 1, ctypes.c_void_p(result.data_ptr())) == 0
    passed, flag, ns = result.tolist()
    assert passed == 0 and flag == 1 and 1.9e9 < ns < 3e9
    assert call(1, 20, ctypes.c_void_p(result.data_ptr())) == 0
    passed, flag, ns = result.tolist()
    assert passed == 0 and flag == 1 and ns < 20 * 1e5, "20 waits after another was given up took %.1f ms" % (ns * 1e-6)


def test_serving_steps_do_not_wait_for_the_gpu(nq):
    """A step is enqueued while the GPU is still busy with what came before it: its lengths are copied without waiting."""
    import time

    from e8_lattice_vector_gb300.serve import PagedCache

    c = PagedCache(2, 3, 2, 64, 16, 200, torch.float16, torch.device(DEV, 0))
    q, k, v = (torch.randn(2, 3, h, 64, device=DEV).half() for h in (8, 2, 2))
    c.fill(*(torch.randn(2, 3, 2, 70, 64, device=DEV).half() for _ in range(2)))
    for _ in range(3):
        c.step(q, k, v, [1, 1, 1])
    torch.cuda.synchronize()
    busy = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    busy[0].record()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    busy[1].record()
    at = time.perf_counter()
    for _ in range(3):
        c.step(q, k, v, [1, 1, 1])
    took = time.perf_counter() - at
    assert not busy[1].query(), "the steps waited for the work before them (%.3f s)" % took
    torch.cuda.synchronize()
    assert took < 0.5e-3 * busy[0].elapsed_time(busy[1])


def test_the_serving_report_asks_whether_it_holds(nq, monkeypatch):
    """No report is made of outputs that are void."""
    from e8_lattice_vector_gb300 import _lib, serve
    from e8_lattice_vector_gb300.synth import CONFIGS

    def gave_up(device):
        raise _lib.NQError("nq_paged_status", 4)

    serve.serve(CONFIGS["tiny"], steps=1)
    monkeypatch.setattr(serve, "paged_status", gave_up, raising=False)
    with pytest.raises(_lib.NQError):
        serve.serve(CONFIGS["tiny"], steps=1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_attention_weights_where_values_cancel(nq, dtype, new, D):
    """Values of both signs over few keys: where they cancel, the output's own rounding is small and the weights' shows.  (In
    bf16 the weights' first part alone passes the bound five to twenty times over.)"""
    for L in (new + 2, new + 20):
        s = Step([(L - new, new)], 4, 2, D, 16, dtype, seed=L)
        put_keys(s, torch.randn(L, 2, D, device=DEV) * 0.4, torch.randn(L, 2, D, device=DEV))
        check_weights(nq, s, D ** -0.5, new)
