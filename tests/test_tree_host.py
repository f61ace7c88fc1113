"""Host-only checks of drafted trees, attention weights and eviction: the tests' plain statements against hand
values, and the refusals of the C ABI and the Python binding (nothing here launches a kernel)."""
import os

import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import tree_ref as tref
from block_sparse_video_vsa_gb300 import build as vbuild
from test_cache_host import A, ALIGNMENT, BAD_CACHES, INVALID, MIS4, MIS16, UNSUPPORTED, cache

B_ = 0x20000  # another address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    vbuild.build()
    return vsa.library()


def test_masks_by_hand():
    # 0 -> 1 -> 3, 0 -> 2, 4 alone
    bits, depth = tref.masks(np.array([[-1, 0, 0, 1, -1]]), [5])
    assert bits[0, :, 0].tolist() == [1, 3, 5, 11, 16] and depth[0].tolist() == [0, 1, 1, 2, 0]
    assert tref.seen_by_bits(bits[0], 7, 5).tolist()[3] == [True, True, True, True, False, True, False]
    wide, _ = tref.masks(np.arange(-1, 69)[None], [70])
    assert wide.shape == (1, 70, 2) and wide[0, 69].tolist() == [-1, 63]


def test_choice_by_hand():
    w = np.array([5, 1, 3, 3, np.nan, 3, 9, 0, -1], np.float32)
    assert tref.choose(w, 9, 4, 0, 0).tolist() == [0, 2, 3, 6]   # of three alike the lowest two
    assert tref.choose(w, 9, 4, 2, 1).tolist() == [0, 1, 6, 8]
    assert tref.choose(w, 9, 8, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7, 8]  # NaN goes first
    assert tref.choose(w, 5, 5, 1, 1).tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, kw, status):
    c = cache(**kw)
    assert lib.vsa_cache_attn_tree(c, A, 1, 4, None, A, None, 0, 0.0, A, A, None, None) == status
    assert lib.vsa_cache_accept(c, A, A, A, 1, B_, None) == status
    assert lib.vsa_cache_weigh(c, A, A, 1, 4, None, 1, 0.0, None, A, None) == status
    assert lib.vsa_cache_evict(c, A, 4, 0, 0, None, 0, A, B_, None, None) == status


def test_tree_refusals(lib):
    def tree(parents=A, B=1, S=4, lens=None, new=None, starts=None, mask=A, pos=A):
        return lib.vsa_cache_tree(parents, B, S, lens, new, starts, mask, pos, None)
    assert tree(parents=None) == INVALID and tree(mask=None) == INVALID and tree(B=0) == INVALID and tree(S=0) == INVALID
    assert tree(S=1025) == UNSUPPORTED and tree(B=65536) == UNSUPPORTED
    assert tree(parents=MIS4) == ALIGNMENT and tree(starts=MIS4) == ALIGNMENT and tree(mask=A + 4) == ALIGNMENT

    def attn(q=A, Sq=1, heads=4, mask=A, sel=None, nsel=0, scale=0.0, ws=A, out=A, lse=None):
        return lib.vsa_cache_attn_tree(cache(), q, Sq, heads, None, mask, sel, nsel, scale, ws, out, lse, None)
    assert attn(mask=None) == INVALID and attn(q=None) == INVALID and attn(heads=3) == INVALID
    assert attn(nsel=2) == INVALID and attn(scale=float("inf")) == INVALID and attn(Sq=0) == INVALID
    assert attn(Sq=1025) == UNSUPPORTED and attn(mask=A + 4) == ALIGNMENT and attn(out=MIS16) == ALIGNMENT

    def accept(new=A, path=A, plens=A, n=4, lens=B_):
        return lib.vsa_cache_accept(cache(), new, path, plens, n, lens, None)
    assert accept(new=None) == INVALID and accept(path=None) == INVALID and accept(plens=None) == INVALID
    assert accept(lens=None) == INVALID and accept(lens=A) == INVALID and accept(n=0) == INVALID
    assert accept(n=1025) == UNSUPPORTED and accept(path=MIS4) == ALIGNMENT and accept(lens=B_ + 2) == ALIGNMENT


def test_weigh_refusals(lib):
    def weigh(q=A, lse=A, Sq=1, heads=4, ql=None, scale=0.0, w=None, out=A):
        return lib.vsa_cache_weigh(cache(), q, lse, Sq, heads, ql, 1, scale, w, out, None)
    assert weigh(q=None) == INVALID and weigh(lse=None) == INVALID and weigh(out=None) == INVALID
    assert weigh(heads=3) == INVALID and weigh(heads=0) == INVALID and weigh(Sq=0) == INVALID
    for x in ("nan", "inf", "-inf"):
        assert weigh(scale=float(x)) == INVALID
    assert weigh(heads=70000) == UNSUPPORTED and weigh(Sq=1 << 23) == UNSUPPORTED
    assert weigh(q=MIS16) == ALIGNMENT and weigh(out=MIS16) == ALIGNMENT and weigh(w=MIS16) == ALIGNMENT
    assert weigh(lse=MIS4) == ALIGNMENT and weigh(ql=MIS4) == ALIGNMENT


def test_evict_refusals(lib):
    def evict(w=A, budget=64, first=0, recent=0, to=None, tw=0, kept=A, lens=B_, moved=None, **kw):
        return lib.vsa_cache_evict(cache(**kw), w, budget, first, recent, to, tw, kept, lens, moved, None)
    assert evict(w=None) == INVALID and evict(kept=None) == INVALID and evict(lens=None) == INVALID
    assert evict(lens=A) == INVALID  # kv_lens
    assert evict(budget=0) == INVALID and evict(first=-1) == INVALID and evict(recent=-1) == INVALID
    assert evict(first=40, recent=25) == INVALID and evict(first=2 ** 31 - 1, recent=2 ** 31 - 1) == INVALID
    assert evict(to=A) == INVALID and evict(to=A, tw=1) == INVALID and evict(tw=1) == INVALID
    assert evict(moved=B_) == INVALID and evict(to=A, tw=1, moved=A) == INVALID
    assert evict(to=A, tw=1, moved=B_, budget=65) == INVALID  # no room
    assert evict(B=60000, kv_heads=3000) == UNSUPPORTED and evict(budget=(1 << 30) + 1) == UNSUPPORTED
    assert evict(to=A, tw=1 << 25, moved=B_) == UNSUPPORTED
    assert evict(w=MIS4) == ALIGNMENT and evict(to=MIS4, tw=1, moved=B_) == ALIGNMENT and evict(lens=B_ + 2) == ALIGNMENT


def test_binding_refuses_cpu_tensors():
    pool = vsa.cache_pool(2, 2, 64, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q, lse = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 1))
    w = torch.zeros((1, 2, 128))
    for call in (lambda: vsa.cache_tree(torch.zeros((1, 3), dtype=torch.int32)),
                 lambda: vsa.cache_attn(q, pool, table, lens, tree=torch.ones((1, 1, 1), dtype=torch.int64)),
                 lambda: vsa.cache_accept(pool, table, lens, lens, torch.zeros((1, 3), dtype=torch.int32), lens),
                 lambda: vsa.cache_weigh(q, lse, pool, table, lens), lambda: vsa.cache_evict(pool, table, lens, w, 64)):
        with pytest.raises(ValueError):
            call()


def test_native_front_leaves_what_it_does_not_take(lib):
    front = vsa._front()
    assert front
    pool = vsa.cache_pool(2, 2, 64, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q, lse, w = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 1)), torch.zeros((1, 2, 128))
    path = torch.zeros((1, 3), dtype=torch.int32)
    mask = torch.ones((1, 1, 1), dtype=torch.int64)
    assert front.attn(q, pool, table, lens, None, True, None, None, 0.0, None, None, None, True, mask) is False
    assert front.tree(path, None, None, None, None, None) is False and front.tree(1, 2, 3, 4, 5, 6) is False
    assert front.accept(pool, table, lens, lens, path, lens, None) is False
    assert front.weigh(q, lse, pool, table, lens, None, True, None, None, None, 0.0) is False
    assert front.evict(pool, table, lens, w, 64, 0, 0, None, None, None, None) is False
    assert front.tree() is False and front.accept(1) is False and front.weigh(1) is False and front.evict(1) is False


def test_these_kernels_read_nothing_as_read_only_data():
    """As the other kernels of the cache: they are launched before the kernel ahead of them has ended."""
    csrc = os.path.dirname(vbuild.FRONT_SRC)
    for name in ("tree.cu", "move.cuh", "evict.cu", "weigh.cu", "weigh.cuh", "weigh_chunk.cu"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for word in ("__ldg", ".nc.", "ld.global.nc", "__restrict__", "__ldca", "tex1D"):
            assert word not in text, (name, word)
