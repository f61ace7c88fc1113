"""GPU: the 4-bit paged cache (append, attention, read back) against the plain
statement in cache_ref: stored bytes exactly, attention within bounds derived
from its roundings (cache_ref.attention_bounds)."""
import threading

import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import cache_ref as ref

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(r, *shape, gain=1.0):
    """Random bf16 numbers as (cuda tensor, float32 array of the same values)."""
    t = torch.from_numpy((gain * r.standard_normal(shape)).astype(np.float32)).bfloat16()
    return t.cuda(), t.float().numpy()


def table_for(r, lens, width, pages):
    """Distinct random pages for every sequence; unused entries hold what must not be read."""
    order = iter(r.permutation(pages).tolist())
    table = np.full((len(lens), width), 2 ** 31 - 1, np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            table[b, i] = next(order)
    return table


def filled(r, lens, width, kv, D, kv_scale, gain=1.0, extra=3):
    """A pool of garbage (NaN scales among it) with the sequences' tokens stored in it."""
    pages = sum(-(-n // 64) for n in lens) + extra
    pool = r.integers(0, 256, (pages, kv, 72 * D), dtype=np.uint8)
    pool[..., 64 * D:] |= np.uint8(0x7F)  # every scale byte of an unused slot is NaN
    table = table_for(r, lens, width, pages)
    for b, n in enumerate(lens):
        for side in (0, 1):
            x = (gain * r.standard_normal((n, kv, D))).astype(np.float32)
            codes, scales = ref.quantise(x, kv_scale[side])
            for t in range(n):
                for h in range(kv):
                    ref.put(pool, table[b, t // 64], t % 64, h, D, side, codes[t, h], scales[t, h])
    return pool, table


def rope_table(rows, R):
    a = np.arange(rows)[:, None] * 1e4 ** (-2.0 * np.arange(R // 2) / R)
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("D,kv,heads,S,lens,new,R,pairs,own_pos", [
    (128, 2, 4, 1, [1, 64, 65, 200], [1, 1, 1, 1], 128, True, False),
    (64, 3, 3, 1, [5, 0, 130], [1, 0, 1], 64, False, False),
    (128, 1, 5, 7, [7, 70, 3], [7, 6, 0], 32, False, True),
    (64, 2, 2, 9, [9, 73, 64], [9, 8, 5], 32, True, True),
    (128, 5, 0, 70, [70, 131], [70, 3], 96, True, False),
    (64, 1, 2, 65, [65], None, 0, False, False),
])
def test_append_stores_the_rule_bytes(D, kv, heads, S, lens, new, R, pairs, own_pos):
    r = np.random.default_rng(D + S + kv)
    B, width = len(lens), 4
    kv_scale = (0.25 + r.random((2, kv))).astype(np.float32)
    pool, table = filled(r, lens, width, kv, D, kv_scale)
    k, k_np = bf16(r, B, S, kv, D)
    v, v_np = bf16(r, B, S, kv, D, gain=0.3)
    rope = rope_table(width * 64, R) if R else None
    pos = r.integers(0, width * 64, (B, S)).astype(np.int32) if own_pos else None
    q = q_np = None
    if heads:
        q, q_np = bf16(r, B, S, heads, D)
    fresh = [S] * B if new is None else new
    want = ref.append(pool, table, k_np, v_np, lens, fresh, kv_scale, rope, pos, pairs)
    got = dev(pool)
    q_out = vsa.cache_append(got, k, v, dev(table), dev(np.array(lens, np.int32)),
                             new_lens=None if new is None else dev(np.array(new, np.int32)),
                             rope=None if rope is None else dev(rope), positions=None if pos is None else dev(pos),
                             interleaved=pairs, q=q, kv_scale=dev(kv_scale))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    # A zero's sign (-0 of a small negative number) is not a value: compare codes with it taken off.
    a, b = got.cpu().numpy(), want
    codes = slice(0, 64 * D)
    plain = lambda x: np.where((x & 7) == 0, x & 0xF0, x)  # noqa: E731  low nibble
    high = lambda x: np.where((x & 0x70) == 0, x & 0x0F, x)  # noqa: E731
    assert np.array_equal(high(plain(a[..., codes])), high(plain(b[..., codes])))
    assert np.array_equal(a[..., 64 * D:], b[..., 64 * D:])
    if heads:
        want_q = np.zeros_like(q_np)
        for s in range(B):
            for i in range(fresh[s]):
                at = lens[s] - fresh[s] + i if pos is None else pos[s, i]
                want_q[s, i] = ref.rotate32(q_np[s, i], rope[at] if R else None, R, pairs)
        assert torch.equal(q_out.cpu(), torch.from_numpy(want_q).bfloat16())
    else:
        assert q_out is None


def test_append_special_values_and_unit_head_scale():
    r = np.random.default_rng(3)
    D, kv = 64, 1
    pool, table = filled(r, [4], 1, kv, D, np.ones((2, kv), np.float32))
    k, k_np = bf16(r, 1, 4, kv, D)
    for t, (at, x) in enumerate([(3, np.nan), (17, np.inf), (40, -np.inf)]):
        k[0, t, 0, at] = x
        k_np[0, t, 0, at] = x
    k[0, 3] = 0
    k_np[0, 3] = 0
    got = dev(pool)
    vsa.cache_append(got, k, k, dev(table), dev(np.array([4], np.int32)))
    want = ref.append(pool, table, k_np, k_np, [4], [4], np.ones((2, kv), np.float32))
    kk, vv = vsa.cache_read(got, dev(table), dev(np.array([4], np.int32)), 4)
    a, b = ref.sequence(want, table[0], 4, D, np.ones((2, kv)))
    assert np.array_equal(kk.double().cpu().numpy()[0], a) and np.array_equal(vv.double().cpu().numpy()[0], b)
    assert np.isfinite(a).all() and a[0, 0, 3] == 0 and a[1, 0, 17] == 2688 and a[2, 0, 40] == -2688


def test_append_and_attention_report_bad_pages_and_positions():
    r = np.random.default_rng(4)
    D, kv, lens = 64, 2, [130]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 3, kv, D, one)
    n = dev(np.array(lens, np.int32))
    k, k_np = bf16(r, 1, 2, kv, D)
    bad = table.copy()
    bad[0, 2] = pool.shape[0]  # one past the pool: the new tokens' page
    got = dev(pool)
    vsa.device_error(reset=True)
    vsa.cache_append(got, k, k, dev(bad), n)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2 and np.array_equal(got.cpu().numpy(), pool)
    # A position outside the table: a zero rotation, and the bit.
    rope = dev(rope_table(100, 64))
    vsa.cache_append(got, k, k, dev(table), n, rope=rope)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    kk, _ = vsa.cache_read(got, dev(table), n, 130)
    assert not kk[0, 128:].any()
    assert vsa.device_error(reset=True) == 0
    # Attention and reading pass a bad page over.
    bad = table.copy()
    bad[0, 1] = -5
    q, q_np = bf16(r, 1, 1, 2, D)
    out, lse = vsa.cache_attn(q, dev(pool), dev(bad), n)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    sel = np.array([[[0, 2], [0, 2]]], np.int32)
    check(q_np, pool, table, lens, [1], False, one, out, lse, sel)
    kk, vv = vsa.cache_read(dev(pool), dev(bad), n, 130)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    assert not kk[0, 64:128].any() and not vv[0, 64:128].any() and kk[0, 128:].any()
    # A length the table cannot hold is cut to it.
    kk, vv = vsa.cache_read(dev(pool), dev(table), dev(np.array([1000], np.int32)), 256)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2 and not kk[0, 192:].any()


# --------------------------------------------------------------------- read
@pytest.mark.parametrize("D,kv,lens,S", [(64, 2, [1, 64, 0, 130], 192), (128, 3, [65, 200], 130), (128, 1, [40], 256)])
def test_read_back(D, kv, lens, S):
    r = np.random.default_rng(S)
    width = 4
    for kv_scale in (np.ones((2, kv), np.float32), (0.1 + r.random((2, kv))).astype(np.float32)):
        pool, table = filled(r, lens, width, kv, D, kv_scale)
        k, v = vsa.cache_read(dev(pool), dev(table), dev(np.array(lens, np.int32)), S, kv_scale=dev(kv_scale))
        torch.cuda.synchronize()
        assert vsa.device_error(reset=True) == 0
        for b, n in enumerate(lens):
            m = min(n, S)
            for got, want in zip((k, v), ref.sequence(pool, table[b], n, D, kv_scale)):
                x = got[b].double().cpu().numpy()
                assert not x[m:].any()
                # fp32 product (2^-24) rounded to bf16 (2^-8); exact for head scales of 1
                lim = 0.0 if (kv_scale == 1).all() else (2.0 ** -8 + 2.0 ** -23) * np.abs(want[:m])
                assert (np.abs(x[:m] - want[:m]) <= lim).all()


# ---------------------------------------------------------------- attention
def check(q_np, pool, table, lens, q_lens, causal, kv_scale, out, lse, sel=None, sm_scale=None):
    D = q_np.shape[-1]
    sm = 1 / np.sqrt(D) if sm_scale is None else sm_scale
    want, want_lse, info = ref.attention(q_np.astype(np.float64), pool, table, lens, q_lens, causal, sm, kv_scale, sel)
    lim, lim_lse = ref.attention_bounds(want, want_lse, info, D)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    err = np.abs(got - want)
    assert (err <= lim).all(), (err - lim).max()
    fin = np.isfinite(want_lse)
    err = np.abs(got_lse[fin] - want_lse[fin])
    assert (err <= lim_lse[fin]).all(), (err - lim_lse[fin]).max()


CASES = [
    # D, kv, heads, Sq, lens, q_lens, causal
    (128, 2, 2, 1, [1, 64, 65, 0, 300], None, True),
    (64, 2, 2, 1, [300], None, True),
    (64, 1, 8, 1, [63, 700], None, False),
    (128, 2, 16, 1, [129, 33], None, True),
    (128, 1, 12, 1, [200], None, True),          # more than 8 rows
    (64, 2, 10, 2, [150, 2, 64], [2, 1, 0], True),
    (128, 1, 3, 4, [70, 3], [4, 4], True),       # a sequence shorter than its queries
    (128, 2, 2, 16, [16, 90], None, True),
    (64, 1, 5, 7, [130, 40], [7, 2], False),     # 35 rows: several tiles
    (128, 1, 2, 40, [100, 61], [40, 33], True),
    (128, 3, 3, 130, [130, 400], [130, 64], True),
    (64, 1, 1, 300, [310], None, True),
    (64, 2, 6, 50, [513, 64], [50, 1], False),
]


@pytest.mark.parametrize("D,kv,heads,Sq,lens,q_lens,causal", CASES)
def test_attention(D, kv, heads, Sq, lens, q_lens, causal):
    r = np.random.default_rng(D + heads + Sq)
    kv_scale = (0.25 + r.random((2, kv))).astype(np.float32)
    pool, table = filled(r, lens, 12, kv, D, kv_scale)
    q, q_np = bf16(r, len(lens), Sq, heads, D, gain=1.5)
    ql = [Sq] * len(lens) if q_lens is None else q_lens
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), dev(np.array(lens, np.int32)),
                              q_lens=None if q_lens is None else dev(np.array(q_lens, np.int32)), causal=causal,
                              kv_scale=dev(kv_scale))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    check(q_np, pool, table, lens, ql, causal, kv_scale, out, lse)


@pytest.mark.parametrize("D,kv,heads,Sq,causal", [(128, 2, 4, 1, False), (64, 1, 12, 1, True), (128, 2, 2, 70, True),
                                                  (64, 3, 3, 20, False)])
def test_attention_over_selected_pages(D, kv, heads, Sq, causal):
    r = np.random.default_rng(Sq + D)
    lens = [700, 64, 640]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 11, kv, D, one)
    sel = np.full((3, kv, 9), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(kv):
            pages = r.permutation(-(-n // 64))[:r.integers(0, 9)]
            sel[b, h, r.permutation(9)[:len(pages)]] = pages
    sel[1, 0, 0] = 40  # past the sequence: passed over
    sel[1, 0, 1:] = -1
    q, q_np = bf16(r, 3, Sq, heads, D)
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), dev(np.array(lens, np.int32)), causal=causal,
                              page_sel=dev(sel))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    seen = np.where(sel >= np.array([-(-n // 64) for n in lens])[:, None, None], -1, sel)
    check(q_np, pool, table, lens, [Sq] * 3, causal, one, out, lse, seen)


@pytest.mark.parametrize("Sq,heads", [(1, 4), (33, 4)])
def test_attention_large_and_small_magnitudes(Sq, heads):
    """Logits near 1e3, queries of 1e30 and 1e-30 (scaled back through sm_scale would overflow fp16 as they are)."""
    r = np.random.default_rng(8)
    D, kv, lens = 128, 2, [333]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 6, kv, D, one)
    for gain, sm in ((120.0, 0.2), (2.0 ** 100, 2.0 ** -104), (2.0 ** -110, 2.0 ** 100)):
        q, q_np = bf16(r, 1, Sq, heads, D, gain=gain)
        out, lse = vsa.cache_attn(q, dev(pool), dev(table), dev(np.array(lens, np.int32)), sm_scale=sm)
        check(q_np, pool, table, lens, [Sq], True, one, out, lse, sm_scale=np.float32(sm))


def test_long_sequence_split_over_the_grid():
    """One sequence of 20000 tokens: its pages are cut over all CTAs; the joined rows match a float64
    softmax of the values read back."""
    g = torch.Generator(device="cuda").manual_seed(0)
    for D, kv, heads, Sq in ((128, 1, 8, 1), (64, 2, 32, 1), (128, 1, 1, 5)):
        n = 20000
        pages = -(-n // 64)
        pool = vsa.cache_pool(pages, kv, D)
        table = torch.randperm(pages, generator=g, device="cuda").int()[None]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        k, v = (torch.randn((1, n, kv, D), generator=g, device="cuda").bfloat16() for _ in "kv")
        vsa.cache_append(pool, k, v, table, lens)
        q = (2 * torch.randn((1, Sq, heads, D), generator=g, device="cuda")).bfloat16()
        out, lse = vsa.cache_attn(q, pool, table, lens)
        kk, vv = (x.double() for x in vsa.cache_read(pool, table, lens, n))
        rep = heads // kv
        s = torch.einsum("qhd,khd->hqk", q[0].double(), kk[0].repeat_interleave(rep, 1)) / D ** 0.5
        at = torch.arange(n, device="cuda")
        s = s.masked_fill(at > n - Sq + torch.arange(Sq, device="cuda")[:, None], -torch.inf)
        want = torch.einsum("hqk,khd->qhd", s.softmax(-1), vv[0].repeat_interleave(rep, 1))
        wabs = torch.einsum("hqk,khd->qhd", s.softmax(-1), vv[0].abs().repeat_interleave(rep, 1))
        # P to fp16 2^-11, logits and sums 2^-12 in all (|s| < 16, 128 terms), the result to bf16 2^-8;
        # weights under fp16's smallest normal: 2^-25 of the largest, n of them, over the sum of weights
        top = (s.amax(-1, keepdim=True) - torch.logsumexp(s, -1, keepdim=True)).exp().movedim(0, 1)
        lim = (2.0 ** -11 + 2.0 ** -12) * wabs + n * 2.0 ** -25 * top * vv.abs().max() + 2.0 ** -8 * want.abs()
        assert ((out[0].double() - want).abs() <= lim).all()
        assert (lse[0].double() - torch.logsumexp(s, -1)).abs().max() <= 2.0 ** -17
    assert vsa.device_error(reset=True) == 0


def dense_reference(q, kk, vv, n, m, causal, pages=None):
    """float64 attention of one sequence: q [Sq, heads, D] (its first m rows live) over kk, vv [>= n, kv, D];
    pages [kv, P] bool: the pages each kv head may see.  -> out, lse, and the error bound of out."""
    Sq, heads, D = q.shape
    kv, rep = kk.shape[1], heads // kk.shape[1]
    k, v = (x[:n].double().repeat_interleave(rep, 1) for x in (kk, vv))
    s = torch.einsum("qhd,khd->hqk", q.double(), k) / D ** 0.5
    at, row = torch.arange(n, device="cuda"), torch.arange(Sq, device="cuda")[:, None]
    keep = (row < m) & ((at <= n - m + row) if causal else torch.ones_like(at, dtype=torch.bool))
    keep = keep.expand(heads, Sq, n)
    if pages is not None:
        keep = keep & pages.repeat_interleave(rep, 0)[:, at // 64][:, None]
    s = s.masked_fill(~keep, -torch.inf)
    lse = torch.logsumexp(s, -1)
    w = (s - lse.clamp(min=-1e300)[..., None]).exp()
    want, wabs = (torch.einsum("hqk,khd->qhd", w, x) for x in (v, v.abs()))
    top = w.amax(-1, keepdim=True).movedim(0, 1) if n else torch.zeros((Sq, heads, 1), device="cuda")
    big = v.abs().max() if n else 0.0
    # P to fp16 2^-11; logits of |s| < 16 as fp32 sums of 128 terms, numerator and denominator: 2^-12;
    # weights under fp16's smallest normal: 2^-25 of the largest, n of them; the result to bf16 2^-8
    return want, lse, (2.0 ** -11 + 2.0 ** -12) * wabs + n * 2.0 ** -25 * top * big + 2.0 ** -8 * want.abs() + 1e-30


@pytest.mark.parametrize("B,kv,heads,D,Sq,most,causal,sel", [
    (33, 2, 6, 128, 1, 1500, True, 0),      # more sequences than a warp's lanes
    (700, 1, 4, 64, 1, 300, True, 0),       # more than a block's threads
    (3, 8, 8, 128, 3, 400, True, 0),        # short walks: units are not cut
    (40, 1, 5, 64, 2, 2500, False, 7),      # selected pages, more than 32 sequences
    (2, 2, 32, 128, 1, 9000, True, 0),      # 16 rows a kv head, cut over the grid
    (5, 3, 9, 128, 60, 1200, True, 0),      # chunks of two tiles a kv head
    (37, 1, 2, 64, 200, 700, True, 0),      # chunks, more than 32 sequences
    (2, 1, 8, 128, 400, 6000, True, 0),     # long chunks, cut over the grid
    (6, 2, 4, 128, 33, 4000, False, 20),    # chunks over selected pages
    (1, 1, 1, 64, 900, 900, True, 0),       # a sequence of its queries alone
])
def test_ragged_batches_of_every_size(B, kv, heads, D, Sq, most, causal, sel):
    r = np.random.default_rng(B + Sq)
    g = torch.Generator(device="cuda").manual_seed(B + Sq)
    lens = [0 if b % 11 == 5 else int(r.integers(1, most + 1)) for b in range(B)]
    lens[0] = most
    q_lens = [int(r.integers(0, Sq + 1)) for _ in range(B)]
    q_lens[0] = Sq
    width = -(-most // 64)
    counts = [-(-n // 64) for n in lens]
    pool = vsa.cache_pool(sum(counts) + 1, kv, D)
    pool.random_(0, 255, generator=g)
    table = dev(table_for(r, lens, width, sum(counts) + 1))
    n = dev(np.array(lens, np.int32))
    k, v = (torch.randn((B, most, kv, D), generator=g, device="cuda").bfloat16() for _ in "kv")
    vsa.cache_append(pool, k, v, table, n, new_lens=n)
    kk, vv = vsa.cache_read(pool, table, n, most)
    q = (1.5 * torch.randn((B, Sq, heads, D), generator=g, device="cuda")).bfloat16()
    page_sel = allowed = None
    if sel:
        pick = np.stack([[r.permutation(width)[:sel] for _ in range(kv)] for _ in range(B)]).astype(np.int32)
        page_sel = dev(pick)
        allowed = torch.zeros((B, kv, width), dtype=torch.bool, device="cuda").scatter_(2, page_sel.long(), True)
    out, lse = vsa.cache_attn(q, pool, table, n, q_lens=dev(np.array(q_lens, np.int32)), causal=causal,
                              page_sel=page_sel)
    again = vsa.cache_attn(q, pool, table, n, q_lens=dev(np.array(q_lens, np.int32)), causal=causal,
                           page_sel=page_sel)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert vsa.device_error(reset=True) == 0
    for b in range(B):
        want, want_lse, lim = dense_reference(q[b], kk[b], vv[b], lens[b], q_lens[b], causal,
                                              None if allowed is None else allowed[b])
        assert ((out[b].double() - want).abs() <= lim).all(), b
        dead = torch.isneginf(want_lse)
        assert torch.equal(dead, torch.isneginf(lse[b])), b
        assert not dead.all() or not out[b].any()
        if not dead.all():
            assert (lse[b].double() - want_lse)[~dead].abs().max() <= 2.0 ** -12, b


@pytest.mark.parametrize("pages", [140000, 280000])  # 2.6 and 5.2 GB
def test_pool_beyond_32_bit_offsets(pages):
    """Pages whose byte offset passes 2^31 and 2^32 are written and read where they are."""
    D, kv = 128, 2
    pool = vsa.cache_pool(pages, kv, D)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, 150, kv, D), generator=g, device="cuda").bfloat16() for _ in "kv")
    vsa.cache_append(pool, k, v, table, lens)
    small = vsa.cache_pool(3, kv, D)
    t2 = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    vsa.cache_append(small, k, v, t2, lens)
    assert torch.equal(pool[table[0].long()], small[t2[0].long()])
    assert int((pool.view(torch.int64) != 0).any(-1).any(-1).sum()) == 3
    for Sq in (1, 40):
        q = torch.randn((1, Sq, 4, D), generator=g, device="cuda").bfloat16()
        for a, b in zip(vsa.cache_attn(q, pool, table, lens), vsa.cache_attn(q, small, t2, lens)):
            assert torch.equal(a, b)
    assert torch.equal(vsa.cache_read(pool, table, lens, 150)[0], vsa.cache_read(small, t2, lens, 150)[0])


# ------------------------------------------------------ as they are used together
def chunked_session(D=128, kv=2, heads=4, chunk=70, steps=3, tokens=5):
    """Chunks, then single tokens, of two ragged sequences: (inputs, final pool, table, lens, outputs)."""
    g = torch.Generator(device="cuda").manual_seed(7)
    B, width = 2, 6
    pool = vsa.cache_pool(B * width + 1, kv, D)
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    rope = dev(rope_table(width * 64, D))
    scale = torch.full((2, kv), 0.5, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    seen = []
    for s in range(steps + tokens):
        S = chunk if s < steps else 1
        new = torch.tensor([S, max(1, S - 13)], dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn((B, S, h, D), generator=g, device="cuda").bfloat16() for h in (heads, kv, kv))
        lens = lens + new
        qr = vsa.cache_append(pool, k, v, table, lens, new_lens=new, rope=rope, q=q, kv_scale=scale)
        seen.append((qr, lens, new, *vsa.cache_attn(qr, pool, table, lens, q_lens=new, kv_scale=scale)))
    torch.cuda.synchronize()
    return pool, table, scale, seen


def test_session_of_chunks_and_tokens():
    pool, table, scale, seen = chunked_session()
    assert vsa.device_error(reset=True) == 0
    p, t, s = pool.cpu().numpy(), table.cpu().numpy(), scale.cpu().numpy()
    for qr, lens, new, out, lse in seen:  # the cache only grows: every step can be checked on the final pool
        check(qr.float().cpu().numpy(), p, t, lens.tolist(), new.tolist(), True, s, out, lse)
    assert not pool[-1].any()  # a page of no sequence stays as it was


def test_cache_feeds_the_fine_stage():
    """cache_read's tiled rows through sparse_attn_fwd over all cubes equal the cache's own attention."""
    g = torch.Generator(device="cuda").manual_seed(2)
    B, heads, D, N = 1, 3, 128, 5
    n = 64 * N - 20
    pool, table = vsa.cache_pool(N, heads, D), torch.arange(N, dtype=torch.int32, device="cuda").flip(0)[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn((B, 64 * N, heads, D), generator=g, device="cuda").bfloat16() for _ in "qkv")
    vsa.cache_append(pool, k[:, :n].contiguous(), v[:, :n].contiguous(), table, lens)
    kt, vt = vsa.cache_read(pool, table, lens, 64 * N)
    vbs = torch.tensor([64] * (N - 1) + [44], dtype=torch.int32, device="cuda")
    a, la = vsa.sparse_attn_fwd(q, kt, vt, vsa.all_cubes(B, heads, N, "cuda"), vbs)
    b, lb = vsa.cache_attn(q, pool, table, lens, causal=False)
    # Both round to bf16 once (2^-8 each of |out| < 1) and P to 2^-9 or 2^-11 of weights over |v| < 4.
    assert (a.float() - b.float()).abs().max() < 2 * 2.0 ** -8 + 4 * (2.0 ** -9 + 2.0 ** -11)
    assert (la - lb).abs().max() < 1e-5
    # One selected page of each kv head is the fine stage with that cube alone.
    sel = torch.tensor([[[1], [4], [0]]], dtype=torch.int32, device="cuda")
    a, _ = vsa.sparse_attn_fwd(q, kt, vt, sel[:, :, None].expand(B, heads, N, 1).contiguous(), vbs)
    b, _ = vsa.cache_attn(q, pool, table, lens, causal=False, page_sel=sel)
    assert (a.float() - b.float()).abs().max() < 2 * 2.0 ** -8 * 4 + 4 * (2.0 ** -9 + 2.0 ** -11)


@pytest.mark.parametrize("Sq", [1, 100])
def test_captured_step_replays_with_new_lengths(Sq):
    """Append and attention captured once; replays on longer caches equal the eager calls bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, kv, heads, D, width = 3, 2, 6, 64, 24
    pool = vsa.cache_pool(B * width, kv, D)
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    rope = dev(rope_table(width * 64, D))
    lens = torch.tensor([Sq, Sq + 500, Sq + 63], dtype=torch.int32, device="cuda")
    fill, fv = (torch.randn((B, width * 64 - 64, kv, D), generator=g, device="cuda").bfloat16() for _ in "kv")
    full = torch.full((B,), width * 64 - 64, dtype=torch.int32, device="cuda")
    vsa.cache_append(pool, fill, fv, table, full, rope=rope)
    q, k, v = (torch.randn((B, Sq, h, D), generator=g, device="cuda").bfloat16() for h in (heads, kv, kv))

    def step():
        return vsa.cache_attn(vsa.cache_append(pool, k, v, table, lens, rope=rope, q=q), pool, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for extra in (0, 7, 64, 700):
        lens += extra
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        graph.replay()
        replayed = [x.clone() for x in got]
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b)
    assert vsa.device_error(reset=True) == 0


def test_two_streams_and_repeated_runs_give_the_same_bits():
    r = np.random.default_rng(11)
    lens, kv, D, heads = [900, 64, 333], 2, 128, 8
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 15, kv, D, one)
    p, t, n = dev(pool), dev(table), dev(np.array(lens, np.int32))
    q, _ = bf16(r, 3, 2, heads, D)
    base = vsa.cache_attn(q, p, t, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:  # each call takes a workspace of its own
            with torch.cuda.stream(s):
                got.append(vsa.cache_attn(q, p, t, n))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, base[0]) and torch.equal(lse, base[1])
    # A stream given to the call, its tensors made by the call and dropped at once by the caller.
    side = streams[0]
    side.wait_stream(torch.cuda.current_stream())
    kept = []
    for i in range(20):
        res = vsa.cache_attn(q, p, t, n, stream=side)
        if i % 7 == 6:
            kept.append(res)
        del res
        torch.full((3, 2, heads, D), float(i), device="cuda")  # whatever the allocator hands out next
    side.synchronize()
    for out, lse in kept:
        assert torch.equal(out, base[0]) and torch.equal(lse, base[1])


def test_calls_between_copies_other_kernels_and_streams_captured_and_not():
    """A call starts its blocks while the kernel before it runs: what copies, other kernels, a join of two
    streams or the call before wrote is seen all the same, in a graph too."""
    r = np.random.default_rng(33)
    lens, kv, D, heads, S = [700, 1500], 2, 128, 4, 70
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 24, kv, D, one)
    t, n = dev(table), dev(np.array(lens, np.int32))
    sets = [[bf16(r, 2, S, h, D)[0] for h in (heads, kv, kv)] for _ in range(4)]
    p, q, k, v = dev(pool), *(torch.zeros_like(x) for x in sets[0])
    side = torch.cuda.Stream()

    def step(src):
        q.copy_(src[0])  # a copy before
        k.copy_(src[1])
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            v.copy_(src[2])
            v.mul_(2.0)
        here.wait_stream(side)  # a join before
        vsa.cache_append(p, k, v, t, n)
        a = vsa.cache_attn(q, p, t, n)  # straight after a call that wrote what it reads
        b = vsa.cache_attn(q[:, -1:].contiguous(), p, t, n)
        kb, vb = vsa.cache_read(p, t, n, 1536)
        return [*a, *b, kb, vb, kb + vb]  # another kernel straight after

    slow = []
    for src in sets:
        p.copy_(dev(pool))
        out = []
        for x in (q.copy_, k.copy_, v.copy_):
            x(src[len(out)]), out.append(0)
        v.mul_(2.0)
        torch.cuda.synchronize()
        vsa.cache_append(p, k, v, t, n)
        torch.cuda.synchronize()
        a = vsa.cache_attn(q, p, t, n)
        torch.cuda.synchronize()
        b = vsa.cache_attn(q[:, -1:].contiguous(), p, t, n)
        torch.cuda.synchronize()
        kb, vb = vsa.cache_read(p, t, n, 1536)
        torch.cuda.synchronize()
        slow.append([*a, *b, kb, vb, kb + vb])
    for _ in range(10):
        fast = [step(src) for src in sets]
        for x, y in zip(slow, fast):
            for c, d in zip(x, y):
                assert torch.equal(c, d)
    now = [x.clone() for x in sets[0]]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        res = step(now)
    for _ in range(5):
        for src, want in zip(sets, slow):
            for x, y in zip(now, src):
                x.copy_(y)
            g.replay()
            for c, d in zip(want, res):
                assert torch.equal(c, d)


def test_threads_call_at_once():
    """Four host threads, each on a stream of its own, append to sequences of their own and attend over them."""
    r = np.random.default_rng(21)
    lens, kv, D, heads = [130, 700, 64, 5], 2, 128, 6
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 24, kv, D, one)
    p = dev(pool)
    t = [dev(table[i:i + 1]) for i in range(4)]
    n = [dev(np.array([x], np.int32)) for x in lens]
    q, k, v = (bf16(r, 4, 5, h, D)[0] for h in (heads, kv, kv))

    def work(i, pool):
        vsa.cache_append(pool, k[i:i + 1], v[i:i + 1], t[i], n[i])
        return (*vsa.cache_attn(q[i:i + 1], pool, t[i], n[i]), *vsa.cache_read(pool, t[i], n[i], 700))

    alone = p.clone()
    want = [work(i, alone) for i in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def thread(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got[i] = work(i, p)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join(60)
    torch.cuda.synchronize()
    assert torch.equal(p, alone)
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_native_front_and_python_path_agree(monkeypatch):
    """The same bits, tensors of the same kind, and the same refusals by either path."""
    r = np.random.default_rng(3)
    lens, kv, D, heads = [90, 200], 2, 64, 6
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 8, kv, D, one)
    t, n = dev(table), dev(np.array(lens, np.int32))
    q, k, v = (bf16(r, 2, 3, h, D)[0] for h in (heads, kv, kv))
    rope = dev(rope_table(256, 32))
    new = dev(np.array([3, 2], np.int32))
    scale = torch.ones(2, kv, device="cuda")
    sel = dev(np.array([[[0, 1], [1, -1]], [[3, 0], [2, 1]]], np.int32))

    def calls():
        p = dev(pool)
        qr = vsa.cache_append(p, k, v, t, n, new_lens=new, rope=rope, q=q, kv_scale=scale, interleaved=True)
        assert vsa.cache_append(p, k, v, t, n, positions=torch.zeros(2, 3, dtype=torch.int32, device="cuda")) is None
        out, lse = torch.empty_like(q), torch.empty((2, heads, 3), device="cuda")
        ws = torch.empty(vsa.cache_attn_workspace_bytes(kv, D, 3, heads), dtype=torch.uint8, device="cuda")
        res = [p, qr, *vsa.cache_attn(qr, p, t, n, q_lens=new, kv_scale=scale, sm_scale=0.25),
               *vsa.cache_attn(qr, p, t, n, causal=False, page_sel=sel, workspace=ws, out=out, lse=lse),
               vsa.cache_attn(qr, p, t, n, want_lse=False)[0], *vsa.cache_read(p, t, n, 130, kv_scale=scale)]
        assert vsa.cache_attn(qr, p, t, n, want_lse=False)[1] is None
        a, b = vsa.cache_attn(qr, p, t, n, out=out, lse=lse)
        assert a is out and b is lse
        mine = torch.empty_like(q)
        assert vsa.cache_append(p, k, v, t, n, q=q, q_out=mine) is mine
        said = []
        for call in (lambda: vsa.cache_attn(q[:, :, :5], p, t, n), lambda: vsa.cache_attn(q, p, t, n, q_lens=new[:1]),
                     lambda: vsa.cache_attn(q, p, t, n, workspace=ws[:16]), lambda: vsa.cache_attn(q, p, t.long(), n),
                     lambda: vsa.cache_attn(q, p, t, n, page_sel=sel[0]), lambda: vsa.cache_attn(q.float(), p, t, n),
                     lambda: vsa.cache_append(p, k, v[:, :2], t, n), lambda: vsa.cache_append(p, k, v, t, n, q_out=mine),
                     lambda: vsa.cache_append(p, k, v, t, n, rope=rope[0]), lambda: vsa.cache_read(p, t, n, 64, k=k)):
            with pytest.raises((TypeError, ValueError)) as e:
                call()
            said.append(str(e.value))
        for call in (lambda: vsa.cache_append(p, k, v, t, n, rope=rope[:, :16].contiguous()),
                     lambda: vsa.cache_attn(q, p, t, n, sm_scale=float("nan")), lambda: vsa.cache_read(p, t, n, 0)):
            with pytest.raises(vsa.VsaError) as e:
                call()
            said.append(str(e.value))
        return res, said

    assert vsa._front()
    native, said_native = calls()
    monkeypatch.setattr(vsa, "_front_module", False)
    assert not vsa._front()
    python, said_python = calls()
    assert said_native == said_python
    for a, b in zip(native, python):
        assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous() and torch.equal(a, b)


def test_binding_refusals():
    D, kv = 64, 2
    pool = vsa.cache_pool(3, kv, D)
    table = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    k = torch.zeros((2, 1, kv, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 1, 4, D), dtype=torch.bfloat16, device="cuda")
    for bad, err in ((dict(pool=pool[:, :, :100].contiguous()), ValueError), (dict(table=table[0]), ValueError),
                     (dict(table=table.long()), TypeError), (dict(kv_lens=lens[:1]), ValueError),
                     (dict(kv_scale=torch.ones(2, device="cuda")), ValueError)):
        a = dict(pool=pool, table=table, kv_lens=lens)
        a.update(bad)
        with pytest.raises(err):
            vsa.cache_attn(q, **a)
        with pytest.raises(err):
            vsa.cache_read(a.pop("pool"), a.pop("table"), a.pop("kv_lens"), 64, **a)
    with pytest.raises(ValueError):
        vsa.cache_attn(q[:, :, :3].contiguous(), pool, table, lens)
    with pytest.raises(ValueError):
        vsa.cache_attn(q.transpose(1, 2), pool, table, lens)
    with pytest.raises(TypeError):
        vsa.cache_attn(q.half(), pool, table, lens)
    with pytest.raises(ValueError):
        vsa.cache_attn(q, pool, table, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        vsa.cache_attn(q, pool, table, lens, page_sel=torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        vsa.cache_append(pool, k, k[:1], table, lens)
    with pytest.raises(ValueError):
        vsa.cache_append(pool, k, k, table, lens, q_out=q)
    with pytest.raises(vsa.VsaError) as e:
        vsa.cache_append(pool, k, k, table, lens, rope=torch.zeros((4, 48), device="cuda"))
    assert e.value.status == 2
    with pytest.raises(vsa.VsaError):
        vsa.cache_read(pool, table, lens, 0)
