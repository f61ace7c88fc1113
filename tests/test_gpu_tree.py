"""GPU: drafted trees over the 4-bit cache (masks and positions, attention, the accepted path) against plain
statements in 64 bits (tree_ref, cache_ref)."""
import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import cache_ref as ref
import tree_ref as tref
from test_gpu_cache import bf16, dev, filled, rope_table

pytestmark = pytest.mark.gpu


def i32(a):
    return dev(np.ascontiguousarray(np.asarray(a, np.int32)))


def random_parents(r, B, S, kind="any"):
    if kind == "chain":
        return np.tile(np.arange(S) - 1, (B, 1)).astype(np.int32)
    if kind == "roots":
        return np.full((B, S), -1, np.int32)
    return np.stack([[r.integers(-1, i) if i else -1 for i in range(S)] for _ in range(B)]).astype(np.int32)


# -------------------------------------------------------------- masks
@pytest.mark.parametrize("B,S,new,kind", [
    (1, 1, [1], "any"), (3, 7, [7, 0, 4], "any"), (2, 64, [64, 63], "any"), (2, 65, [65, 1], "any"),
    (2, 200, [200, 129], "any"), (1, 1024, [1024], "chain"), (1, 1000, [1000], "any"), (2, 130, None, "roots"),
])
def test_masks_and_positions(B, S, new, kind):
    r = np.random.default_rng(S + B)
    parents = random_parents(r, B, S, kind)
    fresh = [S] * B if new is None else new
    lens = np.array([m + 10 * (b + 1) for b, m in enumerate(fresh)], np.int32)
    want, depth = tref.masks(parents, fresh)
    live = np.arange(S) < np.array(fresh)[:, None]
    new_t = None if new is None else i32(new)
    mask, pos = vsa.cache_tree(i32(parents), i32(lens), new_t)
    assert np.array_equal(mask.cpu().numpy(), want)
    start = lens - np.array(fresh)
    assert np.array_equal(pos.cpu().numpy(), np.where(live, start[:, None] + depth, 0))
    starts = np.arange(B) * 1000 + 7
    _, pos = vsa.cache_tree(i32(parents), i32(lens), new_t, starts=i32(starts))
    assert np.array_equal(pos.cpu().numpy(), np.where(live, starts[:, None] + depth, 0))
    _, pos = vsa.cache_tree(i32(parents), None, new_t)
    assert np.array_equal(pos.cpu().numpy(), np.where(live, depth, 0))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0


def test_bad_parents_become_roots_and_are_reported():
    parents = np.array([[-1, 0, 2, 7, -2, 1]], np.int32)  # 2 is itself, 7 comes later, -2 is none
    want, depth = tref.masks(np.array([[-1, 0, -1, -1, -1, 1]]), [6])
    mask, pos = vsa.cache_tree(i32(parents))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2
    assert np.array_equal(mask.cpu().numpy(), want) and np.array_equal(pos.cpu().numpy(), depth)
    vsa.cache_tree(i32([[-1, 5, 9]]), new_lens=i32([1]))  # what lies behind the nodes is not looked at
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0


# ---------------------------------------------------------- attention
def compare(out, lse, q_np, pool, table, lens, new, bits, kv_scale, scale, pages=None):
    D = q_np.shape[-1]
    seen = [tref.seen_by_bits(bits[b], int(n), int(m)) for b, (n, m) in enumerate(zip(lens, new))]
    want, want_lse, info = tref.attention(q_np.astype(np.float64), pool, table, lens, new, seen, scale, kv_scale, pages)
    lim, lim_lse = ref.attention_bounds(want, want_lse, info, D)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = ~np.isfinite(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert (np.abs(got - want) <= lim).all(), (np.abs(got - want) / lim).max()
    assert (np.abs(got_lse[~empty] - want_lse[~empty]) <= lim_lse[~empty]).all()


@pytest.mark.parametrize("D,kv,group,S,lens,new", [
    (64, 2, 1, 1, [1, 65, 200], [1, 1, 0]),                  # one node
    (128, 1, 2, 4, [4, 64, 70, 300], [4, 4, 3, 2]),          # up to 8 rows
    (64, 2, 1, 8, [8, 72, 64, 131], [8, 8, 5, 8]),
    (128, 2, 3, 5, [5, 66, 190], [5, 4, 5]),                 # up to 16
    (64, 1, 5, 3, [3, 40, 600], [3, 3, 3]),
    (128, 2, 5, 12, [12, 130, 75], [12, 11, 12]),            # tcgen05
    (64, 1, 1, 70, [70, 200, 133], [70, 64, 70]),
    (128, 1, 4, 65, [65, 300], [65, 33]),
    (64, 2, 3, 130, [130, 400], [129, 130]),                 # several tiles, three words
])
def test_tree_attention(D, kv, group, S, lens, new):
    r = np.random.default_rng(D + kv + S)
    B, width = len(lens), -(-max(lens) // 64) + 1
    kv_scale = (0.5 + r.random((2, kv))).astype(np.float32)
    pool, table = filled(r, lens, width, kv, D, kv_scale)
    parents = random_parents(r, B, S)
    mask, _ = vsa.cache_tree(i32(parents), new_lens=i32(new))
    q, q_np = bf16(r, B, S, kv * group, D, gain=1.5)
    for b in range(B):
        q[b, new[b]:] = float("nan")  # rows behind the last node hold anything
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), i32(lens), q_lens=i32(new), tree=mask, kv_scale=dev(kv_scale))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    compare(out, lse, q_np, pool, table, lens, new, mask.cpu().numpy(), kv_scale, D ** -0.5)


@pytest.mark.parametrize("D,kv,group,S,lens,new", [
    (64, 1, 5, 12, [20000], [12]),                           # one unit in all CTAs
    (128, 1, 4, 65, [9000], [65]),                           # three
    (64, 3, 2, 70, [8000, 130, 0, 3000], [70, 33, 0, 5]),    # units of 40 parts, of two and of one
    (128, 2, 1, 17, [1500, 90, 700, 2500, 64, 1000], [17, 17, 3, 16, 17, 0]),
    (64, 4, 3, 40, [900] * 12, [40, 1] * 6),                 # as many units as CTAs, nearly
])
def test_units_cut_into_many_parts(D, kv, group, S, lens, new):
    test_tree_attention(D, kv, group, S, lens, new)


@pytest.mark.parametrize("D,group,S,lens,new", [
    (64, 1, 6, [6, 40, 70, 6], [6, 6, 6, 4]), (128, 3, 30, [30, 95, 64], [30, 30, 12]),
    (64, 2, 90, [90, 154, 60], [90, 90, 60])])
def test_any_mask_rows_without_a_key_and_fewer_tokens_than_queries(D, group, S, lens, new):
    """Masks that are no trees: random bits, rows of none (with a context and without one), bits of tokens
    that are not there; and a sequence that is shorter than its queries."""
    r = np.random.default_rng(S)
    B, kv, width = len(lens), 2, 3
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, width, kv, D, one)
    bits = r.integers(-2 ** 63, 2 ** 63 - 1, (B, S, -(-S // 64)), dtype=np.int64)
    bits[:, ::3] = 0
    q, q_np = bf16(r, B, S, kv * group, D)
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), i32(lens), q_lens=i32(new), tree=dev(bits), sm_scale=0.3)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    compare(out, lse, q_np, pool, table, lens, new, bits, one, 0.3)
    # More queries than tokens: the first nodes have no place, the others' bits count from the first node on.
    short = [max(1, m // 2) for m in new]
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), i32(short), q_lens=i32(new), tree=dev(bits), sm_scale=0.3)
    D_ = D
    words = bits.view(np.uint64)
    seen = []
    for b, (n, m) in enumerate(zip(short, new)):
        row = np.zeros((m, n), bool)
        for i in range(m):
            for x in range(n):
                j = x - (n - m)
                row[i, x] = bool((words[b, i, j // 64] >> np.uint64(j % 64)) & np.uint64(1))
        seen.append(row)
    want, want_lse, info = tref.attention(q_np.astype(np.float64), pool, table, short, new, seen, 0.3, one)
    lim, _ = ref.attention_bounds(want, want_lse, info, D_)
    assert (np.abs(out.double().cpu().numpy() - want) <= lim).all()
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), np.isneginf(want_lse))


@pytest.mark.parametrize("group,S", [(1, 5), (4, 40)])
def test_tree_with_selected_pages(group, S):
    r = np.random.default_rng(group)
    D, kv, lens, new = 64, 2, [64 * 7 + 20, 300], [S, S - 2]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 8, kv, D, one)
    parents = random_parents(r, 2, S)
    mask, _ = vsa.cache_tree(i32(parents), new_lens=i32(new))
    sel = np.array([[[7, 0, 3, -1], [6, 7, 1, 2]], [[4, 3, 0, -1], [1, -1, 4, 9]]], np.int32)
    q, q_np = bf16(r, 2, S, kv * group, D)
    out, lse = vsa.cache_attn(q, dev(pool), dev(table), i32(lens), q_lens=i32(new), tree=mask, page_sel=dev(sel))
    compare(out, lse, q_np, pool, table, lens, new, mask.cpu().numpy(), one, D ** -0.5, pages=sel)


@pytest.mark.parametrize("D,group,S", [(128, 1, 4), (64, 4, 4), (128, 8, 40), (64, 1, 200)])
def test_a_chain_is_causal_attention_bit_by_bit(D, group, S):
    r = np.random.default_rng(S)
    kv, lens = 2, [S, S + 64, 700]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 12, kv, D, one)
    mask, pos = vsa.cache_tree(i32(random_parents(r, 3, S, "chain")), i32(lens))
    q, _ = bf16(r, 3, S, kv * group, D)
    args = (q, dev(pool), dev(table), i32(lens))
    a, b = vsa.cache_attn(*args, tree=mask), vsa.cache_attn(*args, causal=True)
    if S * group <= 128:  # (tiles of one unit: the line is cut at the same places)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    else:
        assert (a[0].float() - b[0].float()).abs().max() <= 2 ** -7 * a[0].float().abs().max()
    assert torch.equal(pos.cpu(), torch.tensor(lens)[:, None] - S + torch.arange(S))


# -------------------------------------------------------------- accept
def path_of(r, parents, m):
    """A random node's path."""
    return tref.lines(parents, m)[int(r.integers(0, m))] if m else []


@pytest.mark.parametrize("D,kv,S,lens,new", [
    (64, 1, 1, [1, 64], [1, 1]), (128, 3, 9, [9, 64, 65, 200], [9, 9, 2, 0]), (64, 2, 70, [70, 130, 191], [70, 66, 70]),
    (128, 1, 300, [300, 333], [300, 290])])
def test_accept_moves_the_path(D, kv, S, lens, new):
    r = np.random.default_rng(S + kv)
    B, width = len(lens), -(-max(lens) // 64)
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, width, kv, D, one)
    for case in range(3):
        if case == 0:
            parents = random_parents(r, B, S)
            paths = [path_of(r, parents[b], new[b]) for b in range(B)]
        elif case == 1:  # long paths: every other node, all nodes
            paths = [list(range(b % 2, new[b], 1 + b % 2)) for b in range(B)]
        else:
            paths = [[] for _ in range(B)]
        n = max(1, max(len(p) for p in paths))
        path = np.full((B, n), 2 ** 31 - 1, np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        want = pool.copy()
        for b, p in enumerate(paths):
            base = lens[b] - new[b]
            for h in range(kv):
                tref.move(pool, want, table[b], table[b], [base + x for x in p], range(base, base + len(p)), h, D)
        got = dev(pool)
        out = vsa.cache_accept(got, dev(table), i32(lens), i32(new), dev(path), i32([len(p) for p in paths]))
        torch.cuda.synchronize()
        assert vsa.device_error(reset=True) == 0
        assert out.tolist() == [lens[b] - new[b] + len(p) for b, p in enumerate(paths)]
        assert np.array_equal(got.cpu().numpy(), want)


def test_accept_reports_bad_paths_and_pages():
    r = np.random.default_rng(5)
    D, kv, lens, new = 64, 2, [100], [8]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 2, kv, D, one)
    # Node 9 is not there, 1 does not ascend; the others move.
    path = np.array([[1, 3, 9, 1, 6]], np.int32)
    want = pool.copy()
    for h in range(kv):
        tref.move(pool, want, table[0], table[0], [93, 95], [92, 93], h, D)
        tref.move(pool, want, table[0], table[0], [98], [96], h, D)
    got = dev(pool)
    vsa.device_error(reset=True)
    out = vsa.cache_accept(got, dev(table), i32(lens), i32(new), dev(path), i32([5]))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2 and out.tolist() == [97]
    assert np.array_equal(got.cpu().numpy(), want)
    # More nodes than there are, a page outside the pool: cut, and nothing moved.
    bad = table.copy()
    bad[0, 1] = pool.shape[0]
    got = dev(pool)
    out = vsa.cache_accept(got, dev(bad), i32(lens), i32(new), dev(np.arange(20, dtype=np.int32)[None]), i32([20]))
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 2 and out.tolist() == [100]
    assert np.array_equal(got.cpu().numpy(), pool)


# ------------------------------------------------------- a draft's whole step
@pytest.mark.parametrize("interleaved", [False, True])
def test_steps_of_a_drafting_decoder(interleaved):
    """Three steps: masks, append at the tree's positions, attention, accept.  At the end the cache holds what
    appending the accepted tokens one after another at their positions would have stored."""
    r = np.random.default_rng(6)
    D, kv, heads, S, R = 64, 2, 6, 11, 32
    B, width = 3, 3
    start = np.array([0, 60, 100], np.int32)
    kv_scale = (0.5 + r.random((2, kv))).astype(np.float32)
    pool, table = filled(r, [160, 160, 160], width, kv, D, kv_scale)
    rope = rope_table(width * 64, R)
    got, want, lens = dev(pool), pool.copy(), start.copy()
    for step in range(3):
        new = np.array([11, 5 + step, 8], np.int32)
        parents = random_parents(r, B, S)
        held = i32(lens + new)
        mask, pos = vsa.cache_tree(i32(parents), held, i32(new))
        k, k_np = bf16(r, B, S, kv, D)
        v, v_np = bf16(r, B, S, kv, D, gain=0.5)
        q, q_np = bf16(r, B, S, heads, D)
        qr = vsa.cache_append(got, k, v, dev(table), held, new_lens=i32(new), rope=dev(rope), positions=pos,
                              interleaved=interleaved, q=q, kv_scale=dev(kv_scale))
        out, lse = vsa.cache_attn(qr, got, dev(table), held, q_lens=i32(new), tree=mask, kv_scale=dev(kv_scale))
        compare(out, lse, qr.float().cpu().numpy(), got.cpu().numpy(), table, lens + new, new, mask.cpu().numpy(),
                kv_scale, D ** -0.5)
        paths = [path_of(r, parents[b], int(new[b])) for b in range(B)]
        path = np.full((B, S), -1, np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        after = vsa.cache_accept(got, dev(table), held, i32(new), dev(path), i32([len(p) for p in paths]))
        for b, p in enumerate(paths):  # the same tokens, appended alone
            one = np.array(p)
            want = ref.append(want, table[b:b + 1], k_np[b:b + 1, one], v_np[b:b + 1, one], [lens[b] + len(p)], [len(p)],
                              kv_scale, rope, interleaved=interleaved)
            lens[b] += len(p)
        assert after.tolist() == lens.tolist()
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    kk, vv = vsa.cache_read(got, dev(table), i32(lens), width * 64, kv_scale=dev(kv_scale))
    wk, wv = vsa.cache_read(dev(want), dev(table), i32(lens), width * 64, kv_scale=dev(kv_scale))
    assert torch.equal(kk, wk) and torch.equal(vv, wv)


def test_trees_on_other_streams_through_both_paths_and_in_a_graph():
    r = np.random.default_rng(7)
    D, kv, heads, S, lens, new = 128, 2, 10, 9, [300, 77], [9, 6]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 5, kv, D, one)
    parents, lens_t, new_t = i32(random_parents(r, 2, S)), i32(lens), i32(new)
    q, _ = bf16(r, 2, S, heads, D)
    path, path_lens = i32([[0, 2], [1, 3]]), i32([2, 1])
    table_t = dev(table)

    def step(pool_t, **kw):
        mask, pos = vsa.cache_tree(parents, lens_t, new_t, **kw)
        out, lse = vsa.cache_attn(q, pool_t, table_t, lens_t, q_lens=new_t, tree=mask, **kw)
        return mask, pos, out, lse, vsa.cache_accept(pool_t, table_t, lens_t, new_t, path, path_lens, **kw)

    a_pool, b_pool, c_pool = dev(pool), dev(pool), dev(pool)
    a = step(a_pool)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = step(b_pool, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    step(c_pool)
    c_pool.copy_(dev(pool))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = step(c_pool)
    c_pool.copy_(dev(pool))
    g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)
    assert torch.equal(a_pool, b_pool) and torch.equal(a_pool, c_pool)
    assert vsa.device_error(reset=True) == 0
