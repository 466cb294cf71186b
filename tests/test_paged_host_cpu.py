"""Host arithmetic of the paged attention, compiled from its own headers (paged_host.cu): no GPU is needed."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    from e8_lattice_vector_gb300 import build as nqbuild

    out = str(tmp_path_factory.mktemp("paged") / "paged_host.so")
    subprocess.run([nqbuild._nvcc()] + nqbuild.ARCH + ["-std=c++17", "-O1", "-Xcompiler", "-fPIC", "-shared", "-I",
                                                       nqbuild.INCLUDE, os.path.join(HERE, "paged_host.cu"), "-o", out],
                   check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("rows", [16, 256])
@pytest.mark.parametrize("head_dim", [64, 96, 128])
@pytest.mark.parametrize("base", [1 << 20, (1 << 20) + 16, (1 << 20) + 48, (1 << 20) + 240])
def test_workspace_is_aligned_for_any_caller(host, rows, head_dim, base):
    """A scratch buffer on any 16-byte boundary: every array in it begins on a 32-byte boundary at least (the widest store),
    the arrays do not overlap, and they end within the size that is asked for, which does not depend on the buffer."""
    grid, split_bytes = 152, 20
    got, none = (ctypes.c_uint64 * 4)(), (ctypes.c_uint64 * 4)()
    host.workspace_places(ctypes.c_uint64(base), rows, head_dim, got)
    host.workspace_places(ctypes.c_uint64(0), rows, head_dim, none)
    split, ml, o, total = got
    assert total == none[3]
    assert split % 32 == 0 and ml % 32 == 0 and o % 32 == 0
    assert base <= split and split + grid * split_bytes <= ml and ml + grid * 2 * rows * 8 <= o
    assert o + grid * 2 * rows * head_dim * 4 <= base + total
