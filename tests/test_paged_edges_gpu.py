"""The paged operators at the edges of what callers may pass, against the same 64-bit reference as test_paged_gpu."""
import numpy as np
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
