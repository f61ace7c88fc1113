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


def test_steps_sum_is_the_sum_of_its_floors(lib):
    """Against the sum term by term, with the divisors a group of heads makes, odd and even; one far sum in
    closed form (g = 1: every term is k t + c)."""
    cases = [(n, k, c, g) for n in (0, 1, 2, 7, 64, 501) for k in (1, 2, 3) for c in (0, 1, 5, 63, 64, 999)
             for g in (1, 2, 3, 5, 8, 12, 64, 127)]
    far = (1 << 17, 2, 1 << 25, 1)
    wide = (1 << 17, 2, 65535 << 25, 65535)  # each side's sum passes 2^64
    flat = [x for case in cases + [far, wide] for x in case]
    got = (ctypes.c_longlong * (len(cases) + 2))()
    lib.steps_sum_case((ctypes.c_longlong * len(flat))(*flat), len(cases) + 2, got)
    for case, x in zip(cases, got):
        n, k, c, g = case
        assert x == sum((k * t + c) // g for t in range(n)), case
    n, k, c, g = far
    assert got[len(cases)] == k * n * (n - 1) // 2 + n * c
    n, k, c, g = wide
    assert got[len(cases) + 1] == sum((k * t + c) // g for t in range(n))


def test_a_causal_sequence_costs_the_sum_of_its_tiles(lib):
    """The split's closed form: pages of all tiles but the last, in which a sequence shorter than its queries
    has tiles without keys, equal the pages counted tile by tile."""
    rows = []
    want = []
    for group in (1, 2, 3, 5, 12):
        for q in (130, 257, 1000, 2011):
            for kv in (1, 40, 64, 129, q, q + 1, q + 63, 5200):
                live = -(-q * group // 128)
                pages = [max(0, -(-(kv - q + ((t + 1) * 128 - 1) // group + 1) // 64)) for t in range(live - 1)]
                lead, per = group * (kv - q + 64) + 127, 64 * group
                none = min(live - 1, -(-(per - lead) // 128)) if lead < per else 0
                rows += [live - 1 - none, 2, (lead + none * 128) // 64, group]
                want.append(sum(pages))
    got = (ctypes.c_longlong * len(want))()
    lib.steps_sum_case((ctypes.c_longlong * len(rows))(*rows), len(want), got)
    assert list(got) == want
