"""Host-only checks of functions in csrc/cache.cuh, compiled into a small library (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

from block_sparse_video_vsa_gb300 import build as vbuild


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("header") / "libheader.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cache_host.cu")
    r = subprocess.run([vbuild._nvcc()] + vbuild.NVCC_FLAGS + [f"-I{vbuild.CSRC}", "-shared", src, "-o", so],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return ctypes.CDLL(so)


def test_a_failed_register_query_is_returned_and_asked_again(lib):
    """An error of the query is the call's; the next call asks again; an answer is kept."""
    answers = [(2, 0), (98, 7), (0, 96), (0, 50), (2, 0)]
    flat = (ctypes.c_int * 10)(*(x for a in answers for x in a))
    got = (ctypes.c_int * 10)()
    asked = lib.registers_case(flat, 5, got)
    assert list(got)[0:4:2] == [2, 98]
    assert list(got)[4:] == [0, 96, 0, 96, 0, 96]
    assert asked == 3
