"""GPU: drafts, the accepted path, weights and eviction one after another, as the readme's lines for them run."""
import os

import numpy as np
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa
import cache_ref as ref
import tree_ref as tref
from test_gpu_cache import bf16, dev, filled, rope_table
from test_gpu_tree import i32, path_of, random_parents

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "README.md")


def readme_lines(first, last):
    """The readme's lines of code from the one that begins with `first` to the one that holds `last`."""
    with open(README) as f:
        lines = f.read().split("\n")
    at = next(i for i, line in enumerate(lines) if line.startswith(first))
    end = next(i for i, line in enumerate(lines) if i >= at and last in line)
    return "\n".join(lines[at:end + 1])


@pytest.mark.parametrize("S,group,kind", [(9, 2, "any"), (40, 2, "chain"), (30, 6, "any")])
def test_weights_after_an_accepted_path_as_the_readme_has_them(S, group, kind):
    """Only the path's rows leave weights, each of them one in all, on the keys that it attended.

    The weights' bound is tree_ref.weigh's, with log-sums in 64 bits: the kernel's are off by what
    cache_ref.attention_bounds says, which a weight is by as a factor."""
    r = np.random.default_rng(S)
    B, kv, D, width, R = 3, 2, 64, 4, 32
    one = np.ones((2, kv), np.float32)
    lens = np.array([0, 70, 130])
    new = np.array([S, S - 3, S])
    pool, table = filled(r, lens + new, width, kv, D, one)
    parents = random_parents(r, B, S, kind)
    paths = [path_of(r, parents[0], S), [], max((path_of(r, parents[2], S) for _ in range(20)), key=len)]
    path = np.full((B, S), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    ends = np.array([len(p) for p in paths])
    q, _ = bf16(r, B, S, kv * group, D)
    k, _ = bf16(r, B, S, kv, D)
    v, _ = bf16(r, B, S, kv, D)
    weights = torch.zeros((B, kv, 64 * width), device="cuda")
    vsa.device_error(reset=True)
    names = dict(vsa=vsa, torch=torch, pool=dev(pool), table=dev(table), kv_lens=i32(lens + new), new_lens=i32(new),
                 parents=i32(parents), rope=dev(rope_table(64 * width, R)), q=q, k=k, v=v, path=dev(path),
                 path_lens=i32(ends), weights=weights)
    exec(readme_lines("mask, pos = vsa.cache_tree(", "vsa.cache_evict("), names)
    torch.cuda.synchronize()
    assert vsa.device_error(reset=True) == 0
    now = lens + ends
    assert names["kv_lens"].tolist() == now.tolist()
    pos = names["pos"].cpu().numpy()
    # The rows as they were rotated, the keys as they lie there now.
    qr = vsa.cache_append(dev(pool), k, v, dev(table), i32(lens + new), new_lens=i32(new), rope=names["rope"],
                          positions=dev(pos), q=q).float().cpu().numpy()
    rows = np.zeros((B, S, kv * group, D))
    for b, p in enumerate(paths):
        rows[b, :len(p)] = qr[b, p]
    held = names["pool"].cpu().numpy()
    out, lse, info = ref.attention(rows, held, table, now, ends, True, D ** -0.5, one)
    want, lim = tref.weigh(rows, lse, held, table, now, ends, True, D ** -0.5, one, np.zeros(weights.shape))
    lim_lse = ref.attention_bounds(out, lse, info, D)[1].max()
    got = names["weights"].double().cpu().numpy()
    assert (np.abs(got - want) <= lim + want * np.expm1(lim_lse)).all()
    assert np.allclose(want.sum(-1), group * ends[:, None], rtol=1e-12)
