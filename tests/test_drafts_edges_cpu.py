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
