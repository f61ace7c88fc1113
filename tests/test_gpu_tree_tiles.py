"""GPU: a chain of drafted tokens in several tiles of rows, where a causal call cuts its work at other places:
both within the derived bounds of the definition (cache_ref.attention_bounds)."""
import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
from test_gpu_cache import bf16, dev, filled
from test_gpu_tree import compare, i32, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,group,S", [(128, 4, 40), (64, 1, 200), (64, 3, 90)])
def test_a_chain_of_several_tiles_and_its_causal_form(D, group, S):
    r = np.random.default_rng(S)
    kv, lens, new = 2, [S, S + 64, 500], [S, S, S - 7]
    one = np.ones((2, kv), np.float32)
    pool, table = filled(r, lens, 9, kv, D, one)
    mask, _ = vsa.cache_tree(i32(random_parents(r, 3, S, "chain")), i32(lens), i32(new))
    q, q_np = bf16(r, 3, S, kv * group, D)
    for b, m in enumerate(new):
        q_np[b, m:] = 0
    bits = mask.cpu().numpy()
    args = (q, dev(pool), dev(table), i32(lens), i32(new))
    for form in (dict(tree=mask), dict(causal=True)):
        out, lse = vsa.cache_attn(*args, **form)
        compare(out, lse, q_np, pool, table, lens, new, bits, one, D ** -0.5)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
