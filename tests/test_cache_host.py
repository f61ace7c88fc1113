"""Host-only checks of the 4-bit paged cache: the tests' plain statement of it
against hand values, and the refusals of the C ABI and the Python binding
(nothing here launches a kernel)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import cache_ref as ref
from block_sparse_video_vsa_gb300 import build as vbuild

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
A, MIS4, MIS16 = 0x10000, 0x10002, 0x10008  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    vbuild.build()
    return vsa.library()


def test_code_values_and_ties():
    # Midpoints go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4.
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 100.0])
    assert ref.E2M1[ref.nearest_code(x, ref.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6]
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.E4M3, e4m3)
    r = np.random.default_rng(0)
    y = np.abs(r.standard_normal(4000)).astype(np.float32) * 2.0 ** r.integers(-12, 9, 4000)
    y = np.minimum(y, np.float32(448))
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.E4M3[ref.nearest_code(y, ref.E4M3)], want)


def test_quantise_error_is_half_a_step():
    # code * scale is within half a code step (2^-2 of the value, a quarter below 1) of y / scale, and
    # the scale's own rounding lets the largest saturate by at most 2^-4.
    r = np.random.default_rng(1)
    x = r.standard_normal((50, 3, 64)).astype(np.float32)
    hs = np.array([1.0, 0.5, 0.037], np.float32)
    code, s = ref.quantise(x, hs)
    got = ref.value(code, s, hs)
    step = ref.E4M3[s].repeat(16, -1).reshape(x.shape) * hs[:, None]
    assert (np.abs(got - x) <= np.maximum(0.25 * np.abs(x) * 1.0625, 0.25 * step) * 1.0001).all()


def test_special_values_are_stored_finite():
    x = np.zeros((1, 64), np.float32)
    x[0, 3], x[0, 20], x[0, 40] = np.nan, np.inf, 1e-30
    code, s = ref.quantise(x, np.ones(1, np.float32))
    v = ref.value(code, s, np.ones(1))
    assert v[0, 3] == 0 and v[0, 20] == 2688 and v[0, 40] == 0


def test_pool_bytes(lib):
    assert lib.vsa_cache_pool_bytes(10, 8, 128) == 10 * 8 * 72 * 128
    assert lib.vsa_cache_pool_bytes(300000, 40, 128) == 300000 * 40 * 72 * 128
    assert lib.vsa_cache_pool_bytes(10, 8, 96) == 0
    assert lib.vsa_cache_pool_bytes(0, 8, 128) == 0
    assert lib.vsa_cache_attn_workspace_bytes(8, 128, 1, 40) > 0
    assert lib.vsa_cache_attn_workspace_bytes(8, 128, 1, 41) == 0
    assert lib.vsa_cache_attn_workspace_bytes(8, 96, 1, 40) == 0


def cache(**kw):
    a = dict(pages=4, kv_heads=2, D=64, B=1, width=3, pool=A, table=A, kv_lens=A, kv_scale=None)
    a.update(kw)
    return ctypes.byref(vsa.VsaCache(*a.values()))


BAD_CACHES = [(dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(kv_lens=None), INVALID),
              (dict(pages=0), INVALID), (dict(kv_heads=0), INVALID), (dict(B=-1), INVALID), (dict(width=0), INVALID),
              (dict(D=96), UNSUPPORTED), (dict(B=70000), UNSUPPORTED), (dict(kv_heads=70000), UNSUPPORTED),
              (dict(pages=1 << 30, kv_heads=4), UNSUPPORTED), (dict(width=1 << 25), UNSUPPORTED),
              (dict(pool=MIS16), ALIGNMENT), (dict(table=MIS4), ALIGNMENT), (dict(kv_scale=MIS4), ALIGNMENT)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, kw, status):
    c = cache(**kw)
    assert lib.vsa_cache_append(c, None, A, A, 1, 0, None, None, 0, 0, 0, None, None, None) == status
    assert lib.vsa_cache_read(c, 1, A, A, None) == status
    assert lib.vsa_cache_attn(c, A, 1, 4, None, 1, None, 0, 0.0, A, A, None, None) == status
    assert lib.vsa_cache_append(None, None, A, A, 1, 0, None, None, 0, 0, 0, None, None, None) == INVALID


def test_append_refusals(lib):
    def call(q=None, k=A, v=A, S=1, heads=0, new=None, rope=None, rows=0, R=0, pos=None, qo=None):
        return lib.vsa_cache_append(cache(), q, k, v, S, heads, new, rope, rows, R, 0, pos, qo, None)
    assert call(k=None) == INVALID and call(v=None) == INVALID and call(S=0) == INVALID
    assert call(q=A, heads=2) == INVALID and call(qo=A, heads=2) == INVALID  # q and q_out go together
    assert call(q=A, qo=A, heads=0) == INVALID
    assert call(rope=A, rows=4, R=0) == INVALID and call(R=32) == INVALID and call(rope=A, rows=0, R=32) == INVALID
    assert call(rope=A, rows=4, R=48) == UNSUPPORTED and call(rope=A, rows=4, R=96) == UNSUPPORTED
    assert call(q=A, qo=A, heads=70000) == UNSUPPORTED
    assert call(k=MIS16) == ALIGNMENT and call(rope=MIS16, rows=4, R=32) == ALIGNMENT and call(new=MIS4) == ALIGNMENT


def test_attn_and_read_refusals(lib):
    def call(q=A, Sq=1, heads=4, ql=None, sel=None, nsel=0, scale=0.0, ws=A, out=A, lse=None):
        return lib.vsa_cache_attn(cache(), q, Sq, heads, ql, 1, sel, nsel, scale, ws, out, lse, None)
    assert call(q=None) == INVALID and call(ws=None) == INVALID and call(out=None) == INVALID
    assert call(heads=3) == INVALID and call(heads=0) == INVALID and call(Sq=0) == INVALID
    assert call(nsel=2) == INVALID and call(sel=A) == INVALID and call(scale=float("nan")) == INVALID
    assert call(heads=70000) == UNSUPPORTED and call(Sq=1 << 23) == UNSUPPORTED
    assert call(q=MIS16) == ALIGNMENT and call(ws=MIS16) == ALIGNMENT and call(lse=MIS4) == ALIGNMENT
    assert lib.vsa_cache_read(cache(), 0, A, A, None) == INVALID
    assert lib.vsa_cache_read(cache(), 1, None, A, None) == INVALID
    assert lib.vsa_cache_read(cache(), 1, A, MIS16, None) == ALIGNMENT


def test_binding_refuses_cpu_tensors_and_bad_sizes():
    pool = vsa.cache_pool(2, 2, 64, device="cpu")
    assert pool.shape == (2, 2, 72 * 64) and pool.dtype == torch.uint8
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: vsa.cache_append(pool, k, k, table, lens), lambda: vsa.cache_read(pool, table, lens, 64),
                 lambda: vsa.cache_attn(k, pool, table, lens)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        vsa.cache_pool(2, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        vsa.cache_pool(0, 2, 64, device="cpu")


def test_attn_refuses_an_infinite_scale_and_a_selection_beyond_any_table(lib):
    def call(sel=None, nsel=0, scale=0.0):
        return lib.vsa_cache_attn(cache(), A, 1, 4, None, 1, sel, nsel, scale, A, A, None, None)
    assert call(scale=float("inf")) == INVALID
    assert call(sel=A, nsel=1 << 25) == UNSUPPORTED


def test_native_front_leaves_what_it_does_not_take(lib):
    """Built beside the library; CPU tensors, wrong counts of arguments and anything else go to the Python path."""
    front = vsa._front()
    assert front
    pool = vsa.cache_pool(2, 2, 64, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    assert front.append(pool, k, k, table, lens, None, None, None, False, None, None, None) is False
    assert front.read(pool, table, lens, 64, None, None, None) is False
    assert front.attn(k, pool, table, lens, None, True, None, None, 0.0, None, None, None, True) is False
    assert front.attn() is False and front.read(1, 2, 3, 4, 5, 6, 7) is False
    with pytest.raises(TypeError):
        front.bind(1)


def test_cache_kernels_read_nothing_as_read_only_data():
    """They are launched before the kernel ahead of them has ended, which may write what they read: a
    non-coherent load asks for memory that nobody writes during the reading kernel's life, and the
    compiler may move it before the wait for that end."""
    csrc = os.path.dirname(vbuild.FRONT_SRC)
    names = [n for n in sorted(os.listdir(csrc)) if n.startswith("cache") and n.endswith((".cu", ".cuh"))]
    assert names == ["cache.cuh", "cache_attn.cu", "cache_chunk.cu", "cache_store.cu"]
    for name in names:
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for word in ("__ldg", ".nc.", "ld.global.nc", "__restrict__", "__ldca", "tex1D"):
            assert word not in text, (name, word)


def test_chunk_rows_are_stored_only_after_the_wait_for_their_last_product():
    """The rows that the epilogue stores are chosen after that wait: one that runs out stores none."""
    with open(os.path.join(os.path.dirname(vbuild.FRONT_SRC), "cache_chunk.cu")) as f:
        text = f.read()
    wait, stored = "cache_wait<kSleepShort>(smem_u32(&ms.unit_done)", "const bool real = ok && x.real;"
    assert text.count(wait) == 1 and text.count(stored) == 1
    assert text.index(wait) < text.index(stored) < text.index("__ballot_sync(0xffffffffu, real)")


def test_attn_refuses_a_scale_of_minus_infinity(lib):
    """The scale is finite; below zero it selects the default, at minus infinity it is an error."""
    assert lib.vsa_cache_attn(cache(), A, 1, 4, None, 1, None, 0, float("-inf"), A, A, None, None) == INVALID
