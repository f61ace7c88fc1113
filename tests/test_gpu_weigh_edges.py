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
