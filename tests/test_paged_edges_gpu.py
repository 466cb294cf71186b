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
