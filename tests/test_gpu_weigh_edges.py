"""GPU: attention weights of cached keys where rows, heads or log-sums are out of the ordinary, against the
definition in 64 bits (tree_ref) and against calls that leave those rows out."""
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
from test_gpu_evict import weigh_case

pytestmark = pytest.mark.gpu


# A kv head's last tile of 128 query heads ends inside what one load brings: behind its last head lie the next
# kv head's.
@pytest.mark.parametrize("D,kv,group,S,lens,new", [
    (64, 2, 130, 1, [200], None), (128, 2, 200, 2, [70, 300], [2, 2]), (64, 3, 300, 1, [129], None),
    (128, 2, 200, 3, [90, 150], [3, 1])])
@pytest.mark.parametrize("causal", [True, False])
def test_more_heads_than_a_tile_has_rows_on_several_kv_heads(D, kv, group, S, lens, new, causal):
    q, lse, pool, table, lens_t, call, _, want, lim = weigh_case(D, kv, group, S, lens, new, causal, False)
    got = vsa.cache_weigh(q, lse, pool, table, lens_t, **call)
    x = got.double().cpu().numpy()
    assert (abs(x - want) <= lim).all()
    # The next kv head's first heads hold anything, and have no finite log-sums.
    bad_q, bad_lse, no_lse = q.clone(), lse.clone(), lse.clone()
    for j, v in ((0, float("nan")), (1, float("inf")), (5, -float("inf")), (group - 1, float("nan"))):
        bad_q[:, :, group + j] = v
        bad_lse[:, group + j] = v
        no_lse[:, group + j] = float("inf")
    got_bad = vsa.cache_weigh(bad_q, bad_lse, pool, table, lens_t, **call)
    assert torch.isfinite(got_bad).all()
    assert torch.equal(got_bad[:, 0], got[:, 0])
    assert torch.equal(got_bad, vsa.cache_weigh(q, no_lse, pool, table, lens_t, **call))
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("causal", [False, True])
def test_the_last_rows_of_the_widest_groups(causal):
    """65408 heads (511 tiles of 128) of 64 queries on one kv head: only the last two queries' log-sums are
    finite, and all their rows count.

    A sum of the N rows' positive weights, a fp32 sum in any order, is N 2^-24 off; a weight by what the bound of
    tree_ref.weigh says of logits."""
    D, heads, S, n, live = 64, 511 * 128, 64, 130, 2
    gen = torch.Generator(device="cuda").manual_seed(5)
    pool = vsa.cache_pool(3, 1, D)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    k = torch.randn((1, n, 1, D), generator=gen, device="cuda").bfloat16()
    vsa.cache_append(pool, k, k, table, lens)
    q = torch.randn((1, S, heads, D), generator=gen, device="cuda").bfloat16()
    lse = torch.full((1, heads, S), float("inf"), device="cuda")
    lse[:, :, S - live:] = 4 + torch.rand((1, heads, live), generator=gen, device="cuda")
    got = vsa.cache_weigh(q, lse, pool, table, lens, causal=causal)
    stored = vsa.cache_read(pool, table, lens, n)[0][0, :, 0].double()  # (exact in bf16: no head scale)
    want, lim = torch.zeros(2, 192, dtype=torch.float64, device="cuda")
    for i in range(S - live, S):
        rows = q[0, i].double()
        sums = lse[0, :, i].double()[:, None]
        s = rows @ stored.T / 8
        d = (D + 4) * 2.0 ** -24 * (rows.abs() @ stored.abs().T / 8) + 4 * 2.0 ** -24 * (s.abs() + sums.abs())
        w = torch.exp(s - sums)
        if causal:
            w[:, n - S + i + 1:] = 0
        want[:n] += w.sum(0)
        lim[:n] += (w * (torch.expm1(d) + 2.0 ** -22 + (heads * live + 8) * 2.0 ** -24)).sum(0)
    assert want[:n - 1].min() > heads / 100 and lim[:n].max() < 0.02 * want[:n].max()
    assert ((got[0, 0].double() - want).abs() <= 1.01 * lim).all()
    assert vsa.device_error(reset=True) == 0


@pytest.mark.parametrize("S,group", [(4, 4), (9, 1), (20, 1), (60, 2), (3, 130)])
def test_rows_without_a_key_add_nothing_whatever_their_log_sum(S, group):
    """Rows that see no key (more queries than tokens), their log-sums marked with the type's lowest value."""
    q, lse, pool, table, lens_t, call, _, want, lim = weigh_case(64, 2, group, S, [2, 90], None, True, False)
    marked = lse.clone()
    marked[0, :, :S - 2] = torch.finfo(torch.float32).min
    got = vsa.cache_weigh(q, marked, pool, table, lens_t, **call)
    assert torch.equal(got, vsa.cache_weigh(q, lse, pool, table, lens_t, **call))
    assert (abs(got.double().cpu().numpy() - want) <= lim).all()


@pytest.mark.parametrize("S,group", [(1, 3), (20, 2), (40, 5), (2, 130)])
@pytest.mark.parametrize("bits", [0x7FFFDEAD, 0x7FC00000, 0x7F800001, -1])
def test_no_bits_of_a_nan_log_sum_let_its_row_in(S, group, bits):
    q, lse, pool, table, lens_t, call, _, _, _ = weigh_case(64, 2, group, S, [300, 90], None, False, False)
    heads = 2 * group
    bad_q, bad_lse, no_lse = q.clone(), lse.clone(), lse.clone()
    for j in (0, group, heads - 1):
        bad_q[:, S - 1, j] = float("nan")
        bad_lse.view(torch.int32)[:, j, S - 1] = bits
        no_lse[:, j, S - 1] = float("inf")
    got = vsa.cache_weigh(bad_q, bad_lse, pool, table, lens_t, **call)
    assert torch.isfinite(got).all()
    assert torch.equal(got, vsa.cache_weigh(q, no_lse, pool, table, lens_t, **call))
