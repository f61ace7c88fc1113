"""GPU: attention weights of cached keys and eviction by them, against plain statements in 64 bits (tree_ref)."""
import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import cache_ref as ref
import tree_ref as tref
from test_gpu_cache import bf16, dev, filled

pytestmark = pytest.mark.gpu


def i32(a):
    return dev(np.ascontiguousarray(np.asarray(a, np.int32)))


# --------------------------------------------------------------- weights
def weigh_case(D, kv, group, S, lens, new, causal, add, gain=1.5, width=None, seed=0):
    r = np.random.default_rng(D + kv * 7 + S + seed)
    B = len(lens)
    width = width or -(-max(max(lens), 1) // 64) + 1
    kv_scale = (0.5 + r.random((2, kv))).astype(np.float32)
    pool, table = filled(r, lens, width, kv, D, kv_scale)
    fresh = [S] * B if new is None else new
    q, q_np = bf16(r, B, S, kv * group, D, gain=gain)
    lse = ref.attention(q_np.astype(np.float64), pool, table, lens, fresh, causal, D ** -0.5, kv_scale)[1]
    lse = lse.astype(np.float32)
    before = r.random((B, kv, 64 * width)).astype(np.float32) if add else np.zeros((B, kv, 64 * width), np.float32)
    for b in range(B):
        q[b, fresh[b]:] = float("nan")
        lse[b, :, fresh[b]:] = float("nan")
    want, lim = tref.weigh(q_np.astype(np.float64), lse.astype(np.float64), pool, table, lens, fresh, causal,
                           D ** -0.5, kv_scale, before)
    call = dict(q_lens=None if new is None else i32(new), causal=causal, kv_scale=dev(kv_scale))
    return q, dev(lse), dev(pool), dev(table), i32(lens), call, before, want, lim


CASES = [
    (128, 2, 1, 1, [1, 63, 64, 65, 300], None, True),
    (64, 1, 8, 1, [33, 0, 500], None, True),
    (128, 1, 5, 1, [31, 130], [1, 0], False),
    (64, 3, 4, 2, [2, 100, 1, 257], [2, 1, 2, 2], True),       # a sequence shorter than its queries
    (128, 2, 12, 1, [40, 200], None, True),
    (64, 2, 5, 3, [3, 90, 31], [3, 2, 0], False),
    (128, 2, 1, 17, [17, 260, 600], [17, 9, 17], True),        # tcgen05 from here on
    (64, 1, 3, 40, [40, 129, 255], [40, 33, 0], True),
    (128, 1, 5, 30, [30, 31, 300], [30, 7, 29], False),
    (64, 2, 1, 200, [200, 70, 333], [200, 130, 1], True),      # several tiles of rows, more queries than tokens
    (128, 1, 12, 50, [50, 513], [50, 41], True),
    (64, 1, 130, 2, [70, 300], [2, 1], True),                  # more heads a kv head than a tile has rows
    (128, 1, 300, 1, [129], None, False),
    (64, 1, 128, 3, [200], None, True),
]


@pytest.mark.parametrize("D,kv,group,S,lens,new,causal", CASES)
@pytest.mark.parametrize("add", [False, True])
def test_weights_against_the_definition(D, kv, group, S, lens, new, causal, add):
    q, lse, pool, table, lens_t, call, before, want, lim = weigh_case(D, kv, group, S, lens, new, causal, add)
    vsa.device_error(reset=True)
    if add:
        kept = dev(before)
        out = torch.full_like(kept, float("nan"))
        got = vsa.cache_weigh(q, lse, pool, table, lens_t, weights=kept, out=out, **call)
        assert got is out and torch.equal(kept.cpu(), torch.from_numpy(before))
        inplace = vsa.cache_weigh(q, lse, pool, table, lens_t, weights=kept, **call)
        assert inplace is kept and torch.equal(kept, out)
    else:
        got = vsa.cache_weigh(q, lse, pool, table, lens_t, **call)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    x = got.double().cpu().numpy()
    assert (np.abs(x - want) <= lim).all(), np.nanmax(np.abs(x - want) / np.maximum(lim, 1e-45))
    again = vsa.cache_weigh(q, lse, pool, table, lens_t, weights=dev(before) if add else None, **call)
    assert torch.equal(again, got)
    for b, n in enumerate(lens):  # behind the last token: as it was, or zero
        assert np.array_equal(x[b, :, n:], before[b, :, n:])


@pytest.mark.parametrize("S,group", [(1, 2), (9, 4)])
def test_many_sequences(S, group):
    r = np.random.default_rng(S)
    lens = [int(x) for x in r.integers(0, 140, 70)]
    new = [min(S, n) for n in lens]
    q, lse, pool, table, lens_t, call, _, want, lim = weigh_case(64, 1, group, S, lens, new, True, False, width=6)
    x = vsa.cache_weigh(q, lse, pool, table, lens_t, **call).double().cpu().numpy()
    assert (np.abs(x - want) <= lim).all()


@pytest.mark.parametrize("S,group", [(1, 4), (6, 8)])
def test_weights_of_a_long_cache_sum_to_the_rows(S, group):
    """Each row's softmax weights sum to one: over all keys a kv head's come to its number of rows."""
    r = np.random.default_rng(8)
    D, kv, n = 128, 2, 40000
    gen = torch.Generator(device="cuda").manual_seed(1)
    width = -(-n // 64)
    pool = vsa.cache_pool(width, kv, D)
    table = torch.arange(width, device="cuda", dtype=torch.int32)[None].contiguous()
    lens = i32([n])
    k = torch.randn((1, n, kv, D), generator=gen, device="cuda").bfloat16()
    vsa.cache_append(pool, k, k, table, lens)
    q, _ = bf16(r, 1, S, kv * group, D)
    _, lse = vsa.cache_attn(q, pool, table, lens)
    w = vsa.cache_weigh(q, lse, pool, table, lens).double().sum(-1)
    assert (w - S * group).abs().max() < 1e-4 * S * group


@pytest.mark.parametrize("S,group", [(1, 3), (1, 12), (5, 8), (40, 5)])
def test_rows_without_a_finite_sum_add_nothing(S, group):
    """Whatever their queries hold: NaN, infinities."""
    q, lse, pool, table, lens_t, call, _, _, _ = weigh_case(64, 2, group, S, [300, 90], None, True, False)
    heads = 2 * group
    bad_q, bad_lse = q.clone(), lse.clone()
    for j, x in ((0, float("nan")), (heads - 1, float("inf")), (group, -float("inf"))):
        bad_q[:, S - 1, j] = x
        bad_lse[:, j, S - 1] = x
    zero_lse = lse.clone()
    for j in (0, heads - 1, group):
        zero_lse[:, j, S - 1] = float("inf")
    got = vsa.cache_weigh(bad_q, bad_lse, pool, table, lens_t, **call)
    want = vsa.cache_weigh(q, zero_lse, pool, table, lens_t, **call)
    assert torch.isfinite(got).all() and torch.equal(got, want)
    every = vsa.cache_weigh(q, lse, pool, table, lens_t, **call)
    assert every.sum() > got.sum() + 1  # (the rows taken out had weights of one each)


@pytest.mark.parametrize("S,group", [(1, 2), (30, 3)])
def test_bad_pages_and_lengths_have_no_weight(S, group):
    q, lse, pool, table, lens_t, call, _, _, _ = weigh_case(128, 2, group, S, [700, 200], None, True, False)
    good = vsa.cache_weigh(q, lse, pool, table, lens_t, **call)
    bad = table.clone()
    bad[0, 3], bad[1, 0] = pool.shape[0], -1
    vsa.device_error(reset=True)
    got = vsa.cache_weigh(q, lse, pool, bad, lens_t, **call)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    good[0, :, 192:256] = 0
    good[1, :, :64] = 0
    assert torch.equal(got, good)
    got = vsa.cache_weigh(q, lse, pool, table, i32([-5, 200]), **call)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2 and (got[0] == 0).all()


# -------------------------------------------------------------- eviction
def weights_like(r, kind, shape):
    if kind == "spread":
        w = np.exp(3 * r.standard_normal(shape))
    elif kind == "ties":
        w = r.integers(0, 4, shape) * 0.25
    elif kind == "alike":
        w = np.ones(shape)
    elif kind == "signed":
        w = r.standard_normal(shape) * 10.0 ** r.integers(-38, 38, shape)
        w[..., ::7] = -0.0
        w[..., 3::7] = 0.0
    else:  # special values
        w = r.standard_normal(shape)
        w[..., ::5] = np.nan
        w[..., 1::11] = np.inf
        w[..., 2::13] = -np.inf
        w[..., 4::17] = 1e-42
    return w.astype(np.float32)


@pytest.mark.parametrize("D,kv,lens,budget,first,recent", [
    (64, 2, [1, 64, 65, 200, 0], 64, 0, 0),
    (128, 1, [300, 129], 100, 4, 32),
    (64, 3, [500, 70], 70, 70, 0),
    (128, 2, [500, 130], 129, 0, 129),
    (64, 1, [190, 333], 1, 0, 0),
    (64, 1, [190, 333], 3, 1, 1),
    (128, 2, [700, 640], 639, 3, 500),
    (64, 2, [40, 60], 4000, 5, 10),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "alike", "signed", "special"])
@pytest.mark.parametrize("inplace", [True, False])
def test_evict_keeps_and_moves_what_the_definition_says(D, kv, lens, budget, first, recent, kind, inplace):
    r = np.random.default_rng(budget + D)
    B, width = len(lens), -(-max(lens) // 64) + 1
    to_width = -(-min(budget, 64 * width) // 64) + 1
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, width, kv, D, one, extra=3 + B * to_width)
    free = np.setdiff1d(np.arange(pool.shape[0]), table)
    to_table = r.permutation(free)[:B * to_width].reshape(B, to_width).astype(np.int32)
    w = weights_like(r, kind, (B, kv, 64 * width))
    for b, n in enumerate(lens):
        w[b, :, n:] = 0 if inplace else np.nan
    want = tref.evict(pool, table, w, lens, budget, first, recent, D, None if inplace else to_table)
    got, w_t = dev(pool), dev(w)
    vsa.device_error(reset=True)
    new_lens, kept, moved = vsa.cache_evict(got, dev(table), i32(lens), w_t, budget, first, recent,
                                            to_table=None if inplace else dev(to_table))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    assert np.array_equal(kept.cpu().numpy(), want[1])
    assert np.array_equal(new_lens.cpu().numpy(), want[2])
    bits = lambda x: np.ascontiguousarray(x).view(np.uint32)  # noqa: E731
    assert np.array_equal(bits(moved.cpu().numpy()), bits(want[3]))
    if not inplace:
        assert np.array_equal(bits(w_t.cpu().numpy()), bits(w))
    a, b = got.cpu().numpy(), want[0]
    assert np.array_equal(a, b)


@pytest.mark.parametrize("kind", ["spread", "ties", "alike", "signed", "special"])
@pytest.mark.parametrize("D,kv,lens,budget", [(64, 2, [13000, 300, 33000], 400), (64, 1, [16500, 8100], 8000),
                                              (64, 40, [12400], 65)])
def test_rows_shared_by_blocks_choose_the_same(D, kv, lens, budget, kind):
    """Widths at which a row is a cluster's, with lengths that leave blocks of it few places or none."""
    test_evict_keeps_and_moves_what_the_definition_says(D, kv, lens, budget, 2, 30, kind, False)


def big_case(D, kv, n, budget, seed, B=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-n // 64)
    pool = torch.randint(0, 256, (2 * B * width, kv, 72 * D), generator=gen, device="cuda", dtype=torch.uint8)
    order = torch.randperm(2 * B * width, generator=gen, device="cuda").int()
    w = torch.exp(2 * torch.randn((B, kv, width * 64), generator=gen, device="cuda"))
    w = (w * 64).round() / 64
    return pool, order[:B * width].view(B, width).contiguous(), order[B * width:].view(B, width).contiguous(), w


def rows_of(pool, table, at, D):
    """Bytes of tokens `at` [B, kv, m] (places): K and V codes and scales, [B, kv, m, 9 D / 8]."""
    kv = pool.shape[1]
    page = table.long()[torch.arange(table.shape[0], device=at.device)[:, None, None], at // 64]
    raw = pool[page, torch.arange(kv, device=at.device)[None, :, None]]
    slot = (at % 64)[..., None]
    cut = [raw.gather(3, base + slot * size + torch.arange(size, device=at.device))
           for base, size in ((0, D // 2), (32 * D, D // 2), (64 * D, D // 16), (68 * D, D // 16))]
    return torch.cat(cut, 3)


@pytest.mark.parametrize("D,kv,n,budget,first,recent", [
    (128, 8, 32760, 8190, 0, 1560), (64, 2, 115200, 50001, 4, 1000), (128, 1, 400000, 399000, 7, 0),
    (64, 40, 5000, 2048, 4, 256)])
@pytest.mark.parametrize("inplace", [True, False])
def test_evict_of_long_sequences(D, kv, n, budget, first, recent, inplace):
    """Rows that take a whole cluster, whose keys do or do not fit its shared memory."""
    pool, table, to, w = big_case(D, kv, n, budget, budget)
    lens = i32([n])
    place = torch.arange(w.shape[2], device="cuda")
    key = torch.where((place < first) | (place >= n - recent), torch.inf, w).masked_fill_(place >= n, -torch.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    at = best.sort(-1).values
    want, want_w = rows_of(pool, table, at, D), w.gather(2, at)
    to = to[:, :-(-budget // 64)].contiguous()
    before = pool.clone()
    new_lens, kept, moved = vsa.cache_evict(pool, table, lens, w, budget, first, recent, to_table=None if inplace else to)
    assert new_lens.tolist() == [budget] and torch.equal(kept.long(), at)
    assert torch.equal(moved[..., :budget], want_w) and (moved[..., budget:n] == 0).all()
    now = torch.arange(budget, device="cuda").expand(1, kv, budget)
    assert torch.equal(rows_of(pool, table if inplace else to, now, D), want)
    untouched = torch.ones(pool.shape[0], dtype=torch.bool, device="cuda")
    untouched[(table[:, :-(-budget // 64)] if inplace else to).flatten().long()] = False
    assert torch.equal(pool[untouched], before[untouched])
    assert vsa.device_error(reset=True) == 0


def test_evict_reports_bad_pages():
    pool, table, to, w = big_case(64, 2, 500, 100, 3)
    bad = table.clone()
    bad[0, 5] = pool.shape[0]
    before = pool.clone()
    w[..., :320] = 0
    w[..., 320:384] = 9  # tokens of the bad page are kept: nothing is written to their places
    vsa.device_error(reset=True)
    lens, kept, moved = vsa.cache_evict(pool, bad, i32([500]), w, 64, to_table=to[:, :1].contiguous())
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    want = before.cpu().numpy().copy()
    for h in range(2):
        at = tref.choose(w[0, h].cpu().numpy(), 500, 64, 0, 0)
        assert kept[0, h].tolist() == at.tolist() and (at // 64 == 5).sum() > 10
        there = at // 64 != 5
        tref.move(before.cpu().numpy(), want, table[0].cpu().numpy(), to[0].cpu().numpy(), at[there],
                  np.arange(64)[there], h, 64)
    assert lens.tolist() == [64] and np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("budget", [200, 320])
@pytest.mark.parametrize("inplace", [True, False])
def test_bad_pages_among_those_moved(budget, inplace):
    """Few tokens kept and more: those of a bad page leave their new places as they were."""
    pool, table, to, w = big_case(128, 3, 700, 400, 5)
    bad = table.clone()
    bad[0, 7] = -1
    w[..., 448:512] += 100
    before, want = pool.cpu().numpy(), pool.cpu().numpy().copy()
    weights = w[0].cpu().numpy().copy()
    vsa.device_error(reset=True)
    _, kept, _ = vsa.cache_evict(pool, bad, i32([700]), w, budget, 1, 9,
                                 to_table=None if inplace else to[:, :-(-budget // 64)].contiguous())
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    for h in range(3):
        at = tref.choose(weights[h], 700, budget, 1, 9)
        assert kept[0, h].tolist() == at.tolist()
        there = at // 64 != 7
        assert (~there).sum() == 64
        tref.move(before, want, table[0].cpu().numpy(), (table if inplace else to)[0].cpu().numpy(), at[there],
                  np.arange(budget)[there], h, 128)
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("D,kv,lens,budget,first,recent", [
    (128, 2, [4160, 256, 257, 0], 256, 0, 0), (64, 2, [4160, 255], 255, 3, 100), (64, 1, [4224, 100], 256, 0, 7),
    (128, 1, [600, 258], 257, 1, 1), (128, 2, [300, 129, 64], 128, 64, 64), (64, 3, [193, 4000], 193, 0, 192)])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("inplace", [True, False])
def test_few_kept_tokens_and_one_more(D, kv, lens, budget, first, recent, kind, inplace):
    """Both sides of the lengths and budgets up to which choice and move are one kernel."""
    test_evict_keeps_and_moves_what_the_definition_says(D, kv, lens, budget, first, recent, kind, inplace)


# ----------------------------------------------------- together, as they are used
def test_a_decoder_that_evicts():
    """A prompt, then tokens one by one with weights summed up and an eviction whenever the cache passes its
    mark, against the same steps in 64 bits on the stored bytes."""
    r = np.random.default_rng(9)
    D, kv, heads, B, width, mark, budget = 64, 2, 4, 2, 3, 120, 90
    kv_scale = (0.5 + r.random((2, kv))).astype(np.float32)
    pool, table = filled(r, [0, 0], width, kv, D, kv_scale, extra=2 * B * width)
    table = r.permutation(pool.shape[0])[:B * width].reshape(B, width).astype(np.int32)
    pool_t, table_t, ks = dev(pool), dev(table), dev(kv_scale)
    lens = np.array([110, 70], np.int32)
    position = lens.copy()
    q, q_np = bf16(r, B, 110, heads, D)
    k, _ = bf16(r, B, 110, kv, D)
    rope = torch.from_numpy(np.concatenate((np.cos(np.arange(400)[:, None] * [1, 0.1] * 8), np.sin(
        np.arange(400)[:, None] * [1, 0.1] * 8)), 1).astype(np.float32)).cuda().repeat_interleave(8, 1)
    qr = vsa.cache_append(pool_t, k, k, table_t, i32(lens), new_lens=i32(lens), rope=rope, q=q, kv_scale=ks)
    _, lse = vsa.cache_attn(qr, pool_t, table_t, i32(lens), q_lens=i32(lens), kv_scale=ks)
    w_t = vsa.cache_weigh(qr, lse, pool_t, table_t, i32(lens), q_lens=i32(lens), kv_scale=ks)
    w, lim = tref.weigh(qr.double().cpu().numpy(), lse.double().cpu().numpy(), pool_t.cpu().numpy(), table, lens, lens, True,
                        D ** -0.5, kv_scale, np.zeros((B, kv, 64 * width)))
    assert (np.abs(w_t.double().cpu().numpy() - w) <= lim).all()
    evictions = 0
    for step in range(40):
        lens, position = lens + 1, position + 1
        q, _ = bf16(r, B, 1, heads, D)
        k, _ = bf16(r, B, 1, kv, D)
        qr = vsa.cache_append(pool_t, k, k, table_t, i32(lens), rope=rope, positions=i32(position[:, None] - 1), q=q,
                              kv_scale=ks)
        _, lse = vsa.cache_attn(qr, pool_t, table_t, i32(lens), kv_scale=ks)
        vsa.cache_weigh(qr, lse, pool_t, table_t, i32(lens), weights=w_t, kv_scale=ks)
        now = pool_t.cpu().numpy()
        w, more = tref.weigh(qr.double().cpu().numpy(), lse.double().cpu().numpy(), now, table, lens, [1, 1], True,
                             D ** -0.5, kv_scale, w)
        lim = lim + more
        assert (np.abs(w_t.double().cpu().numpy() - w) <= lim).all()
        if lens.max() > mark:
            was = w_t.cpu().numpy()
            want = tref.evict(now, table, was, lens, budget, 4, 30, D)
            new_lens, kept, _ = vsa.cache_evict(pool_t, table_t, i32(lens), w_t, budget, 4, 30)
            assert np.array_equal(kept.cpu().numpy(), want[1]) and np.array_equal(pool_t.cpu().numpy(), want[0])
            assert np.array_equal(w_t.cpu().numpy(), want[3])
            for b in range(B):
                for h in range(kv):
                    at = want[1][b, h][want[1][b, h] >= 0]
                    for x in (w, lim):
                        rest = x[b, h, at]
                        if lens[b] > budget:
                            x[b, h] = 0
                        x[b, h, :len(at)] = rest
            lens = new_lens.cpu().numpy()
            evictions += 1
    torch.cuda.synchronize()
    assert evictions >= 1 and vsa.device_error(reset=True) == 0


def test_weigh_and_evict_on_other_streams_through_both_paths_and_in_a_graph():
    q, lse, pool, table, lens_t, call, _, _, _ = weigh_case(128, 2, 5, 6, [700, 320], [6, 5], True, False)
    to = torch.arange(pool.shape[0], pool.shape[0] + 8, device="cuda", dtype=torch.int32).view(2, 4).contiguous()
    big = torch.cat((pool, torch.zeros_like(pool[:8])))
    q1, lse1 = q[:, :1].contiguous(), lse[:, :, :1].contiguous()

    def step(pool_t, **kw):
        w = vsa.cache_weigh(q, lse, pool_t, table, lens_t, **call, **kw)
        w2 = vsa.cache_weigh(q1, lse1, pool_t, table, lens_t, causal=False, weights=w, kv_scale=call["kv_scale"], **kw)
        lens, kept, moved = vsa.cache_evict(pool_t, table, lens_t, w2, 200, 2, 50, to_table=to, **kw)
        _, kept2, _ = vsa.cache_evict(pool_t, table, lens_t, w2, 250, 2, 50, **kw)
        return w, lens, kept, moved, kept2

    a_pool, b_pool, c_pool = big.clone(), big.clone(), big.clone()
    a = step(a_pool)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = step(b_pool, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = step(c_pool)
    c_pool.copy_(big)
    g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)
    assert torch.equal(a_pool, b_pool) and torch.equal(a_pool, c_pool)
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("D,group,S,n,new", [(64, 5, 200, 300, 199), (128, 8, 150, 500, 150), (64, 300, 4, 200, 3)])
def test_few_units_are_shared_by_clusters(D, group, S, n, new):
    """One kv head, few keys and many tiles of rows: up to 8 blocks share a unit's rows."""
    q, lse, pool, table, lens_t, call, before, want, lim = weigh_case(D, 1, group, S, [n], [new], True, True)
    got = vsa.cache_weigh(q, lse, pool, table, lens_t, weights=dev(before), **call)
    assert (np.abs(got.double().cpu().numpy() - want) <= lim).all()
    assert torch.equal(got, vsa.cache_weigh(q, lse, pool, table, lens_t, weights=dev(before), **call))
    assert vsa.device_error(reset=True) == 0


def test_pages_beyond_four_gib():
    """The same few tokens at the pool's start and at its end give the same weights, choice and moves."""
    D, kv = 128, 40
    r = np.random.default_rng(11)
    pages = 2 ** 32 // (kv * 72 * D) + 60
    lens = [500, 130]
    small, table = filled(r, lens, 8, kv, D, np.ones((2, kv), np.float32))
    pool = torch.zeros((pages, kv, 72 * D), dtype=torch.uint8, device="cuda")
    shift = pages - small.shape[0]
    pool[shift:] = dev(small)
    far = np.where(table < small.shape[0], table + shift, table).astype(np.int32)
    parents = i32(np.stack([np.arange(9) - 1, np.full(9, -1)]))
    new = i32([9, 7])
    mask, _ = vsa.cache_tree(parents, i32(lens), new)
    results = []
    for p, t in ((dev(small), table), (pool, far)):
        t = dev(t)
        for S in (1, 9):  # both kernels of each
            q, _ = bf16(np.random.default_rng(S), 2, S, kv * 4, D)
            m = new if S == 9 else None
            out, lse = vsa.cache_attn(q, p, t, i32(lens), q_lens=m, tree=mask if S == 9 else None)
            w = vsa.cache_weigh(q, lse, p, t, i32(lens), q_lens=m)
            results.append((out, lse, w))
        ends = vsa.cache_accept(p, t, i32(lens), new, i32([[0, 3, 4], [1, 2, -1]]), i32([3, 2]))
        _, kept, moved = vsa.cache_evict(p, t, ends, w, 100, 2, 30)
        results.append((ends, kept, moved, *vsa.cache_read(p, t, i32([100, 100]), 100)))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    for a, b in zip(results[:3], results[3:]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_refusals_say_what_is_wrong():
    q, lse, pool, table, lens_t, call, _, _, _ = weigh_case(64, 2, 2, 3, [100, 40], [3, 2], True, False)
    w = vsa.cache_weigh(q, lse, pool, table, lens_t, **call)
    places = w.shape[2]
    bad = [
        lambda: vsa.cache_weigh(q.float(), lse, pool, table, lens_t),
        lambda: vsa.cache_weigh(q, lse[:, :2], pool, table, lens_t),
        lambda: vsa.cache_weigh(q, lse.transpose(1, 2), pool, table, lens_t),
        lambda: vsa.cache_weigh(q[:, :, :3].contiguous(), lse, pool, table, lens_t),
        lambda: vsa.cache_weigh(q, lse, pool, table, lens_t, q_lens=lens_t[:1]),
        lambda: vsa.cache_weigh(q, lse, pool, table, lens_t, weights=w[..., :64]),
        lambda: vsa.cache_weigh(q, lse, pool, table, lens_t, out=w.double()),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 0),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 10, 6, 5),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 10, -1, 0),
        lambda: vsa.cache_evict(pool, table, lens_t, w[:, :1], 10),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 10, moved=w),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 10, to_table=table[:1]),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 10, to_table=table.float()),
        lambda: vsa.cache_evict(pool, table, lens_t, w, 10, kept=torch.zeros((2, 2, 9), dtype=torch.int32, device="cuda")),
        lambda: vsa.cache_tree(lens_t),
        lambda: vsa.cache_tree(table, new_lens=lens_t[:1]),
        lambda: vsa.cache_tree(table, mask=torch.zeros((2, 2, 1), dtype=torch.int64, device="cuda")),
        lambda: vsa.cache_accept(pool, table, lens_t, None, table, lens_t),
        lambda: vsa.cache_accept(pool, table, lens_t, lens_t, lens_t, lens_t),
        lambda: vsa.cache_attn(q, pool, table, lens_t, tree=torch.zeros((2, 3, 2), dtype=torch.int64, device="cuda")),
        lambda: vsa.cache_attn(q, pool, table, lens_t, tree=torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda")),
    ]
    for call_ in bad:
        with pytest.raises((ValueError, TypeError)):
            call_()
    for call_, status in ((lambda: vsa.cache_weigh(q, lse, pool, table, lens_t, sm_scale=float("nan")), 1),
                          (lambda: vsa.cache_evict(pool, table, lens_t, w, 10, lens=lens_t), 1),
                          (lambda: vsa.cache_evict(pool, table, lens_t, w, places, to_table=table[:, :1].contiguous()), 1),
                          (lambda: vsa.cache_accept(pool, table, lens_t, lens_t, table, lens_t, lens=lens_t), 1)):
        with pytest.raises(vsa.VsaError) as e:
            call_()
        assert e.value.status == status
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0


def test_four_host_threads_at_once():
    """Each with its own stream and cache: the same answers as alone."""
    import threading
    cases = [weigh_case(128 if i % 2 else 64, 2, 3 + i, 1 + 9 * (i % 2), [700 + i, 90], None, True, False, seed=i)
             for i in range(4)]

    def steps(c):
        q, lse, pool, table, lens_t, call = c[:6]
        pool = pool.clone()
        w = vsa.cache_weigh(q, lse, pool, table, lens_t, **call)
        lens, kept, _ = vsa.cache_evict(pool, table, lens_t, w, 300, 2, 20)
        return w, lens, kept, pool

    alone = [steps(c) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = steps(cases[i])
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
