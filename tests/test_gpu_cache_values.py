"""GPU: values at the edges of what the 4-bit cache's attention takes: NaN in
queries, scales so small that they leave fp32, weights far below the largest,
queries whose channels are far apart."""
import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import cache_ref as ref

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def random_cache(seed, lens, kv, D):
    """(pool, table, lens on the GPU, k and v as read back) of sequences of `lens` random tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    counts = [-(-n // 64) for n in lens]
    width, most = max(counts), max(lens)
    pool = vsa.cache_pool(sum(counts), kv, D)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(counts), generator=g, device="cuda").int()
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((len(lens), most, kv, D), generator=g, device="cuda").bfloat16() for _ in "kv")
    vsa.cache_append(pool, k, v, table, n, new_lens=n)
    return pool, table, n, *vsa.cache_read(pool, table, n, most), g


@pytest.mark.parametrize("D,kv,heads,Sq,lens", [
    (128, 1, 1, 1, [300]),         # a unit that is not cut
    (128, 1, 8, 1, [20000]),       # one row a head, cut over the grid
    (64, 2, 32, 1, [20000, 70]),   # 16 rows a kv head, cut
    (128, 1, 4, 40, [20000]),      # chunks, cut
    (64, 2, 6, 50, [513, 64]),     # chunks, whole
])
def test_a_nan_query_gives_nan_however_the_work_is_cut(D, kv, heads, Sq, lens):
    """By the definition a NaN in a query makes every logit of its row NaN; the other rows keep their bits."""
    pool, table, n, _, _, g = random_cache(Sq + D, lens, kv, D)
    q = torch.randn((len(lens), Sq, heads, D), generator=g, device="cuda").bfloat16()
    base = vsa.cache_attn(q, pool, table, n, causal=False)
    sick = q.clone()
    rows = {(0, 0, heads - 1), (len(lens) - 1, Sq - 1, 0), (0, Sq // 2, heads // 2)}
    for j, (b, i, h) in enumerate(sorted(rows)):  # (an infinity's products with keys of both signs and 0 too)
        sick[b, i, h, (7 * i + h) % D] = float("inf" if j == 1 else "nan")
    out, lse = vsa.cache_attn(sick, pool, table, n, causal=False)
    for b in range(len(lens)):
        for i in range(Sq):
            for h in range(heads):
                if (b, i, h) in rows:
                    assert out[b, i, h].isnan().all() and lse[b, h, i].isnan(), (b, i, h)
                else:
                    assert torch.equal(out[b, i, h], base[0][b, i, h]), (b, i, h)
                    assert torch.equal(lse[b, h, i], base[1][b, h, i]), (b, i, h)
    # Rows from a sequence's query count on have no key, whatever they hold.
    out, lse = vsa.cache_attn(torch.full_like(q, float("nan")), pool, table, n,
                              q_lens=torch.zeros_like(n), causal=False)
    assert not out.any() and torch.isneginf(lse).all()
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("Sq", [1, 40])
def test_a_scale_below_fp32_leaves_masked_keys_out(Sq):
    """Queries of 1e-34 on a head scale of 1e-10: every logit is 0 to fp32, and the slots past the length
    stay out of the sum."""
    D, kv, heads, n = 128, 2, 4, 100
    pool, table, lens, _, vv, g = random_cache(5, [n], kv, D)
    scale = torch.tensor([[1e-10] * kv, [1.0] * kv], device="cuda")
    q = (1e-34 * torch.randn((1, Sq, heads, D), generator=g, device="cuda")).bfloat16()
    for causal in (False, True):
        out, lse = vsa.cache_attn(q, pool, table, lens, causal=causal, kv_scale=scale)
        for i in range(Sq):
            seen = n - Sq + i + 1 if causal else n
            want = vv[0, :seen].double().mean(0).repeat_interleave(heads // kv, 0)
            mag = vv[0, :seen].double().abs().mean(0).repeat_interleave(heads // kv, 0)
            # equal weights: P and the sum are exact up to 2^-21; the result to bf16 2^-8
            assert ((out[0, i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * mag).all()
            assert (lse[0, :, i].double() - np.log(seen)).abs().max() <= 2.0 ** -20 * (1 + np.log(seen))
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("D,Sq", [(64, 1), (128, 1), (64, 17), (128, 17)])
def test_many_small_weights_count_beside_a_large_one(D, Sq):
    """One key of weight 1 and n - 1 of weight 2^-26: together they are 2^-8 of the sum, and with v = 0 at
    the first and 1 at the others all of the output.  The pages of the small keys are one page, shared."""
    B, kv, pages = 8, 40, 4096
    n = 64 * pages
    pool = np.zeros((2, kv, 72 * D), np.uint8)
    one, zero = np.full(D, 2, np.uint8), np.zeros(D, np.uint8)  # codes of 1 and 0
    unit = np.full(D // 16, 0x38, np.uint8)                      # scales of 1
    six = zero.copy()
    six[0] = 7                                                   # a 6 in channel 0
    for h in range(kv):
        for page in (0, 1):
            for t in range(64):
                first = page == 0 and t == 0
                ref.put(pool, page, t, h, D, 0, six if first else zero, unit)
                ref.put(pool, page, t, h, D, 1, zero if first else one, unit)
    table = np.ones((B, pages), np.int32)
    table[:, 0] = 0
    lens = np.full(B, n, np.int32)
    q = torch.zeros((B, Sq, kv, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    sm = 26 * np.log(2.0) / 6
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), dev(lens), causal=False, sm_scale=float(sm))
    small = (n - 1) * 2.0 ** -26
    want = small / (1 + small)
    # A weight of 2^-26 is a whole number of fp16's smallest steps once the largest is 2^7, so what is left
    # is exp2 and the fp32 sums (the logit is off by 26 * 2^-23, exp2 by 2^-21, sums of 2^12 terms a lane
    # by 2^-12 at most) and the result's rounding to bf16, 2^-8 of it.
    assert ((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want).all(), out.double().mean().item() / want
    assert ((lse.double() - (26 * np.log(2.0) + np.log1p(small))).abs() <= 2.0 ** -11).all()
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("D,heads,Sq", [(128, 2, 1), (64, 16, 1), (128, 2, 40), (64, 3, 20)])
def test_queries_with_channels_far_apart(D, heads, Sq):
    """A channel of 2^20 whose keys are 0 beside channels of 2^-12 to 1 (2^-32 to 2^-20 of the largest): the
    small ones make the logits, and lose at most 2^-39 of the row's largest each on their way to fp16."""
    n, kv = 700, 1
    r = np.random.default_rng(D)
    k = r.standard_normal((1, n, kv, D)).astype(np.float32) * 2.0
    k[..., 0] = 0
    g = torch.Generator(device="cuda").manual_seed(1)
    pool, table, lens, _, _, _ = random_cache(2, [n], kv, D)
    v = torch.randn((1, n, kv, D), generator=g, device="cuda").bfloat16()
    vsa.cache_append(pool, dev(k).bfloat16(), v, table, lens)
    kk, vv = (x[0, :, 0].double() for x in vsa.cache_read(pool, table, lens, n))
    q = torch.randn((1, Sq, heads, D), generator=g, device="cuda") * torch.exp2(
        torch.randint(-12, 1, (1, Sq, heads, D), generator=g, device="cuda").float())
    q[..., 0] = 2.0 ** 20
    q = q.bfloat16()
    out, lse = vsa.cache_attn(q, pool, table, lens, causal=False, sm_scale=0.5)
    s = 0.5 * torch.einsum("qhd,kd->qhk", q[0].double(), kk)
    w = s.softmax(-1)
    want, wabs = w @ vv, w @ vv.abs()
    # logits: 2^-39 * 2^20 a channel from fp16, fp32 sums of D products (D + 4 roundings of 2^-24)
    absk = 0.5 * kk.abs().sum(-1).max()
    d = 2.0 ** -19 * absk + (D + 4) * 2.0 ** -24 * 0.5 * torch.einsum("qhd,kd->qhk", q[0].double().abs(), kk.abs()).amax()
    lim = (2.0 ** -11 + 2.0 ** -21 + 2 * d) * wabs + n * 2.0 ** -25 * vv.abs().max() * w.amax(-1, keepdim=True)
    assert ((out[0].double() - want).abs() <= lim + 2.0 ** -8 * (want.abs() + lim)).all()
    assert (lse[0].T.double() - torch.logsumexp(s, -1)).abs().max() <= d + 2.0 ** -19
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("D,heads,Sq", [(128, 2, 1), (64, 12, 1), (128, 2, 40)])
def test_logits_near_their_limit_stay_finite(D, heads, Sq):
    """Logits of up to 2^22: weights may pass 2^15 by what fp32 rounds off a logit, and still fit fp16."""
    n, kv = 2000, 2 if heads == 2 else 1
    pool, table, lens, kk, vv, g = random_cache(9, [n], kv, D)
    rep = heads // kv
    k, v = (x[0].double().repeat_interleave(rep, 1) for x in (kk, vv))
    q = torch.randn((1, Sq, heads, D), generator=g, device="cuda")
    s = torch.einsum("qhd,khd->qhk", q[0].double(), k) / D ** 0.5
    q = (q * (4.0e6 / s.abs().amax(-1)[None, ..., None])).bfloat16()  # (bf16 moves a logit by 2^-9 of 2^22 or so)
    s = torch.einsum("qhd,khd->qhk", q[0].double(), k) / D ** 0.5
    assert 2.0 ** 21 < s.abs().max() < 2.0 ** 22
    out, lse = vsa.cache_attn(q, pool, table, lens, causal=False)
    assert out.isfinite().all() and lse.isfinite().all()
    # Each logit is off by at most (D + 4) roundings of 2^-24 of sum |q k|, and so is the log of their sum.
    d = (D + 4) * 2.0 ** -24 * torch.einsum("qhd,khd->qhk", q[0].double().abs(), k.abs()).amax(-1) / D ** 0.5
    assert ((lse[0].T.double() - torch.logsumexp(s, -1)).abs() <= d + 2.0 ** -22 * lse[0].T.abs()).all()
    # Where the largest logit leads by more than both can be off, the row is its value (bf16: exact for a head scale of 1).
    top2 = s.topk(2, -1)
    sure = top2.values[..., 0] - top2.values[..., 1] > 2 * d + 20
    assert sure.any()
    pick = v[top2.indices[..., 0], torch.arange(heads, device="cuda")[None, :]]
    assert ((out[0].double() - pick).abs() <= 2.0 ** -8 * pick.abs() + 1e-6)[sure].all()
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("Sq", [1, 40])
def test_a_nan_head_scale_is_not_hidden(Sq):
    """Head scales are finite by contract; a NaN one gives NaN in its head's rows and leaves the others alone."""
    kv, D = 2, 64
    pool, table, lens, _, _, g = random_cache(3, [700], kv, D)
    q = torch.randn((1, Sq, 4, D), generator=g, device="cuda").bfloat16()
    scale = torch.ones(2, kv, device="cuda")
    base = vsa.cache_attn(q, pool, table, lens, kv_scale=scale)
    for side in (0, 1):
        bad = scale.clone()
        bad[side, 1] = float("nan")
        out, lse = vsa.cache_attn(q, pool, table, lens, kv_scale=bad)
        assert out[:, :, 2:].isnan().all() and (side == 1 or lse[:, 2:].isnan().all())
        assert torch.equal(out[:, :, :2], base[0][:, :, :2]) and torch.equal(lse[:, :2], base[1][:, :2])
    assert vsa.device_error(reset=True) == 0
