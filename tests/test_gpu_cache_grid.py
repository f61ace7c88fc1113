"""GPU: the 4-bit cache and the cubes of a grid.  Raster tokens are attended by
cache_attn on any grid; tiled rows, padding slots among them, are read back for
the fine stage, which masks them by vbs; on a grid of full cubes a page is a cube."""
import pytest
import torch

import block_sparse_video_vsa_gb300 as vsa

pytestmark = pytest.mark.gpu


def clip(grid, heads, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T, H, W = grid
    return [torch.randn((B, T * H * W, heads, D), generator=g, device="cuda").bfloat16() for _ in "qkv"]


def cached(k, v):
    """A cache that holds k, v's rows in their order -> (pool, table, lens)."""
    B, S, heads, D = k.shape
    width = -(-S // 64)
    pool = vsa.cache_pool(B * width, heads, D)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").flip(0).view(B, width).contiguous()
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    vsa.cache_append(pool, k, v, table, lens)
    return pool, table, lens


# Both sides round to bf16 once (2^-8 each of |out| < 2) and P to 2^-9 or 2^-11 of weights over |v| < 6.
LIMIT = 2 * 2 * 2.0 ** -8 + 6 * (2.0 ** -9 + 2.0 ** -11)


@pytest.mark.parametrize("grid", [(1, 5, 6, 7), (2, 3, 9, 4), (1, 4, 8, 12)])
def test_raster_tokens_and_tiled_rows_give_the_same_attention(grid):
    heads, D = 2, 64
    q, k, v = clip(grid, heads, D, sum(grid))
    a, la = vsa.cache_attn(q, *cached(k, v), causal=False)  # raster: every place is a token
    (qt, vbs), (kt, _), (vt, _) = (vsa.tile(x, grid) for x in (q, k, v))
    B, N = q.shape[0], vsa.num_cubes(grid)
    kr, vr = vsa.cache_read(*cached(kt, vt), 64 * N)
    b, lb = vsa.sparse_attn_fwd(qt, kr, vr, vsa.all_cubes(B, heads, N, "cuda"), vbs)
    assert (a.float() - vsa.untile(b, grid).float()).abs().max() < LIMIT
    lb = vsa.untile(lb.transpose(1, 2)[..., None].repeat(1, 1, 1, D).bfloat16(), grid)[..., 0]  # (bf16: 2^-8 of |lse| < 8)
    assert (la.transpose(1, 2) - lb.float()).abs().max() < 8 * 2.0 ** -8 + 1e-4
    assert vsa.device_error(reset=True) == 0


def test_on_full_cubes_a_page_selection_is_a_cube_selection():
    grid, heads, D = (1, 4, 8, 12), 3, 128
    q, k, v = clip(grid, heads, D, 1)
    (qt, vbs), (kt, _), (vt, _) = (vsa.tile(x, grid) for x in (q, k, v))
    N = vsa.num_cubes(grid)
    assert bool((vbs == 64).all())
    pool, table, lens = cached(kt, vt)
    kr, vr = vsa.cache_read(pool, table, lens, 64 * N)
    sel = torch.tensor([[[1, 4], [5, 0], [2, 3]]], dtype=torch.int32, device="cuda")
    a, _ = vsa.cache_attn(qt, pool, table, lens, causal=False, page_sel=sel)
    b, _ = vsa.sparse_attn_fwd(qt, kr, vr, sel[:, :, None].expand(1, heads, N, 2).contiguous(), vbs)
    assert (a.float() - b.float()).abs().max() < 2 * LIMIT  # (|out| < 4 over fewer keys)
    assert vsa.device_error(reset=True) == 0
