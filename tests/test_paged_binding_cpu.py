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
