"""GPU: the cache kernels' bounded wait runs out, is called off and succeeds, and says which."""
import ctypes
import os
import subprocess
import time

import pytest

from block_sparse_video_vsa_gb300 import build as vbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wait_case(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("wait") / "libwait.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cache_wait.cu")
    r = subprocess.run([vbuild._nvcc()] + vbuild.NVCC_FLAGS + [f"-I{vbuild.CSRC}", "-shared", src, "-o", so],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    fn = ctypes.CDLL(so).wait_case
    fn.argtypes = [ctypes.c_int, ctypes.c_ulonglong, ctypes.POINTER(ctypes.c_int)]

    def call(mode, limit_ns):
        got = (ctypes.c_int * 3)()
        assert fn(mode, limit_ns, got) == 0
        return list(got)

    call(2, 2_000_000)  # the first launch loads the code
    return call


def test_a_wait_that_nobody_ends_runs_out_at_its_limit(wait_case):
    for limit_ms in (5, 200):
        t = time.monotonic()
        assert wait_case(0, limit_ms * 1_000_000) == [0, 1, 1]  # false, abort raised, VSA_DEVERR_TIMEOUT
        took = time.monotonic() - t
        assert limit_ms * 1e-3 <= took < limit_ms * 1e-3 + 1.0, took


def test_a_raised_abort_ends_the_wait_without_the_timeout_bit(wait_case):
    t = time.monotonic()
    assert wait_case(1, 1_500_000_000) == [0, 1, 0]
    assert time.monotonic() - t < 1.5


def test_a_completed_phase_ends_the_wait(wait_case):
    assert wait_case(2, 1_000_000_000) == [1, 0, 0]
