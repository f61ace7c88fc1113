"""Drafted trees over the 4-bit paged cache, and eviction from it, as measured: attention for a tree of drafted
tokens, a draft's step (masks, append, the accepted path kept), attention weights summed for every cached key, and
eviction by them.

A cache pool is uint8 [pages, kv_heads, 72 * D]; a page of one head holds 64 tokens:
    K codes [64][D / 2] | V codes [64][D / 2] | K scales [64][D / 16] | V scales [64][D / 16]
A code is 4 bits (sign, two exponent bits, one mantissa bit; the low nibble is the even channel), a scale
is an 8-bit e4m3 number shared by 16 channels, and kv_scale [2, kv_heads] is fp32 per head (0: K, 1: V).
"""
import math

import torch

own = False

PAGE = 64
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # --- attention of a tree: 8 nodes on the 5 x 6 x 10 grid, 2 heads (latency)
        dict(name="tree_tiny", op="tree", B=1, S=8, heads=2, kv=2, D=64, most=308, ragged=False),
        # 60 nodes on a 21 x 30 x 52 clip, 40 query heads on 8 cached heads
        dict(name="tree_clip", op="tree", B=1, S=60, heads=40, kv=8, D=128, most=32760, ragged=False),
        # a serving batch: trees of up to 26 nodes, ragged contexts
        dict(name="tree_batch", op="tree", B=16, S=26, heads=32, kv=8, D=128, most=12000, ragged=True),
        # --- a draft's step around that attention (masks and positions, append, accept, the tail read back):
        # one session (latency), and a serving batch
        dict(name="draft_one", op="draft", B=1, S=12, heads=40, kv=8, D=128, most=2000, R=128, pairs=True, ragged=False),
        dict(name="draft_batch", op="draft", B=61, S=48, heads=32, kv=8, D=128, most=4000, R=128, pairs=False,
             ragged=True),
        # --- weights of the cached keys: one new token on a clip, added to those so far
        dict(name="weigh_token", op="weigh", B=1, S=1, heads=40, kv=8, D=128, most=32760, causal=True, add=True,
             ragged=False),
        # a serving batch's step, ragged lengths
        dict(name="weigh_batch", op="weigh", B=61, S=1, heads=32, kv=8, D=128, most=12000, causal=True, add=True,
             ragged=True),
        # the last 64 tokens of a prompt as the window that decides what is kept, whole heads
        dict(name="weigh_window", op="weigh", B=1, S=64, heads=40, kv=40, D=128, most=32760, causal=True, add=False,
             ragged=False),
        # one latent frame's queries on the clip so far (the largest)
        dict(name="weigh_frame", op="weigh", B=1, S=1560, heads=40, kv=40, D=128, most=32760, causal=False, add=False,
             ragged=False),
        # --- eviction to other pages, read back: a small grid (latency), a clip cut to a quarter, a ragged batch
        dict(name="evict_small", op="evict", B=2, kv=2, D=64, most=300, budget=128, first=4, recent=32, ragged=True),
        dict(name="evict_clip", op="evict", B=1, kv=40, D=128, most=32760, budget=8190, first=0, recent=1560,
             ragged=False),
        dict(name="evict_batch", op="evict", B=24, kv=8, D=64, most=12000, budget=2048, first=4, recent=256,
             ragged=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "draft", "token", "chunk", "chunk", "evict", "evict"))
    D = rng.choice((64, 128, 128))
    kv = rng.choice((1, 2, 5, 8, 24, 40))
    if op == "evict":
        most = _spread(rng, 1, 32760)
        B = _spread(rng, 1, max(1, min(24, 32760 * 40 // (most * kv))))
        budget = _spread(rng, 1, most + most // 8)
        first = rng.choice((0, 0, _spread(rng, 1, 8)))
        first = min(first, budget)
        recent = rng.choice((0, budget // 8, budget // 3, budget - first))
        return dict(op="evict", B=B, kv=kv, D=D, most=most, budget=budget, first=first,
                    recent=min(recent, budget - first), ragged=rng.random() < 0.7)
    group = rng.choice((1, 2, 3, 4, 5, 8, 12))
    if op == "draft":
        S = _spread(rng, 1, 200)
        B = _spread(rng, 1, max(1, min(61, 120000 // (S * kv * (2 + group)))))
        return dict(op="draft", B=B, S=S, heads=kv * group, kv=kv, D=D, most=S + _spread(rng, 1, 4000),
                    R=rng.choice((0, 32, 64, D)), pairs=rng.random() < 0.5, ragged=rng.random() < 0.7)
    if op == "tree":
        S = _spread(rng, 1, 200)
        most = S + _spread(rng, 1, 32560)
        B = _spread(rng, 1, max(1, min(32, 5000000 // (most * kv), 400000000 // (S * most * kv * group))))
        return dict(op="tree", B=B, S=S, heads=kv * group, kv=kv, D=D, most=most, ragged=rng.random() < 0.6)
    if op == "token":
        S = rng.choice((1, 1, 1, 2, 4))
        most = _spread(rng, S, 65536)
        B = _spread(rng, 1, max(1, min(128, 5000000 // (most * kv))))
    else:
        S = _spread(rng, 5, 2048)
        most = _spread(rng, S, 32760)
        while S * most * kv * group > 2000000000 and group > 1:
            group -= 1
        while S * most * kv * group > 2000000000:
            most = max(S, most // 2)
            S = max(5, S // 2)
        B = _spread(rng, 1, max(1, min(16, 1000000000 // (S * most * kv * group))))
    return dict(op="weigh", B=B, S=S, heads=kv * group, kv=kv, D=D, most=most, causal=rng.random() < 0.7,
                add=rng.random() < 0.5, ragged=rng.random() < 0.6)


def _lens(case):
    """Tokens of each sequence in the cache, and those of this step among them (made from the case alone)."""
    B, most = case["B"], case["most"]
    step = case.get("S", 0)
    kv, new = [], []
    for b in range(B):
        share = 1.0 if not case["ragged"] or b == 0 else 0.05 + 0.95 * ((b * 0.6180339887) % 1.0)
        n = max(1, round(step * share)) if step else 0
        kv.append(max(n, round(most * share), 1))
        new.append(n)
    return kv, new


# ----------------------------------------------------------------- inputs
def _e2m1(y):
    """Codes 0..15 of the nearest 4-bit values, ties to the even code, saturating."""
    below = lambda edge: float(torch.nextafter(torch.tensor(edge), torch.tensor(0.0)))  # noqa: E731
    edges = torch.tensor((0.25, below(0.75), 1.25, below(1.75), 2.5, below(3.5), 5.0), device=y.device)
    return torch.bucketize(y.abs(), edges).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)


def _quantise(x, head_scale):
    """fp32 [..., kv, D] -> (codes uint8 [..., kv, D], scales e4m3 [..., kv, D / 16]) for fp32 head_scale [kv]."""
    y = x * torch.reciprocal(head_scale)[:, None]
    y = y.unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    code = _e2m1(y * torch.where(sf > 0, torch.reciprocal(sf), torch.zeros_like(sf))[..., None])
    return code.flatten(-2), s


def _dequantise(code, scale, head_scale):
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=code.device)
    y = grid[code.int()].unflatten(-1, (-1, 16)) * scale.float()[..., None]
    return y.flatten(-2) * head_scale[:, None]


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(byte):
    return torch.stack((byte & 15, byte >> 4), -1).flatten(-2)


def _filled_pool(gen, pages, kv, D, kv_scale, dev):
    """A pool whose pages hold quantised keys and values; a few key channels run larger, as they do in models."""
    pool = torch.empty((pages, kv, 72 * D), dtype=torch.uint8, device=dev)
    loud = 1.0 + 3.0 * (torch.rand((kv, D), generator=gen, device=dev) < 0.03).float()
    per = max(1, 50000000 // (PAGE * kv * D))
    for p in range(0, pages, per):
        n = min(per, pages - p)
        part = pool[p:p + n]
        for row, (c0, s0, gain) in enumerate(((0, 64 * D, loud), (32 * D, 68 * D, 0.5))):
            x = torch.randn((n, PAGE, kv, D), generator=gen, device=dev) * gain
            code, scale = _quantise(x, kv_scale[row])
            part[:, :, c0:c0 + 32 * D] = _pack(code).permute(0, 2, 1, 3).flatten(2)
            part[:, :, s0:s0 + 4 * D] = scale.view(torch.uint8).permute(0, 2, 1, 3).flatten(2)
    return pool


def _trees(case, seed, new):
    """Parents [B, S] of random trees (-1: the context), and the path from a root to some node: [B, longest], lengths."""
    gen = torch.Generator().manual_seed(seed)
    B, S = case["B"], case["S"]
    u = torch.rand((B, S), generator=gen)
    parents = (u * (torch.arange(S) + 1)).floor().int().clamp(max=S - 1) - 1
    ends = [int(x * n) for x, n in zip(torch.rand(B, generator=gen).tolist(), new)]
    paths = []
    for row, end in zip(parents.tolist(), ends):
        path = [end]
        while row[path[0]] >= 0:
            path.insert(0, row[path[0]])
        paths.append(path)
    path = torch.full((B, min(S, 32)), -1, dtype=torch.int32)
    lens = [min(len(p), path.shape[1]) for p in paths]
    for b, p in enumerate(paths):
        path[b, :lens[b]] = torch.tensor(p[:lens[b]], dtype=torch.int32)
    return parents, path, lens


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, kv, D, op = case["B"], case["kv"], case["D"], case["op"]
    kv_lens, new = _lens(case)
    width = -(-max(kv_lens) // PAGE)
    counts = [-(-n // PAGE) for n in kv_lens]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    to_width = -(-min(case["budget"], max(kv_lens)) // PAGE) if op == "evict" else 0
    pages = sum(counts) + B * to_width + 3
    order = torch.randperm(pages, generator=gen, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    kv_scale = 0.25 + 0.5 * torch.rand((2, kv), generator=gen, device=dev)
    st = dict(case=case, kv_lens=i32(kv_lens), new=i32(new), table=table, width=width, kv_scale=kv_scale,
              pool=_filled_pool(gen, pages, kv, D, kv_scale, dev))
    if op == "evict":
        # Sums of softmax weights: spread over many orders of magnitude, some of them zero, some alike.
        w = torch.exp(2.5 * torch.randn((B, kv, width * PAGE), generator=gen, device=dev))
        w = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.1, torch.zeros_like(w), w)
        st["weights"] = torch.where(w > 3.0, (w * 8.0).round() / 8.0, w)
        st["to_table"] = order[at:at + B * to_width].view(B, to_width).contiguous()
        return st
    S, heads = case["S"], case["heads"]
    if op == "draft":
        R = case["R"]
        bf = lambda h: torch.randn((B, S, h, D), generator=gen, device=dev).bfloat16()  # noqa: E731
        st.update(q=bf(heads), k=bf(kv), v=bf(kv))
        if R:
            angle = torch.arange(width * PAGE, device=dev, dtype=torch.float64)[:, None] * torch.exp(
                torch.arange(R // 2, device=dev, dtype=torch.float64) * (-2.0 * math.log(1e4) / R))
            st["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        # The pages from the first that the draft touches on: what a step may have changed.
        skip = torch.tensor([(n - m) // PAGE for n, m in zip(kv_lens, new)], device=dev)
        tail = max(c - int(s) for c, s in zip(counts, skip.tolist()))
        column = skip[:, None] + torch.arange(tail, device=dev)
        st["tail"] = torch.where(column < i32(counts)[:, None], table.gather(1, column.clamp(max=width - 1)), -1).int()
        st["skipped"] = (skip * PAGE).int()
    else:
        st["q"] = (1.5 * torch.randn((B, S, heads, D), generator=gen, device=dev)).bfloat16()
    if op in ("tree", "draft"):
        parents, path, lens = _trees(case, seed, new)
        st.update(parents=parents.to(dev), path=path.to(dev), path_lens=i32(lens))
        if op == "tree":
            st["mask"] = _mask_plain(st)[0]
    if op == "weigh":
        s, _ = _logits_plain(st)
        lse = torch.logsumexp(s.double() if s.numel() < 50000000 else s, -1).float()
        st["lse"] = _by_head(lse, case).contiguous()
        if case["add"]:
            st["weights"] = 4.0 * torch.rand((B, kv, width * PAGE), generator=gen, device=dev)
    return st


# -------------------------------------------------------------- plain forms
def _read_plain(st, table=None):
    """All pages of a table as fp32 K, V [B, kv, n, 64, D]."""
    D, kv = st["case"]["D"], st["case"]["kv"]
    table = st["table"] if table is None else table
    page = table.long().clamp(min=0)[:, None, :].expand(table.shape[0], kv, table.shape[1])
    raw = st["pool"][page, torch.arange(kv, device=page.device)[:, None]]
    half = lambda c0, s0, scale: _dequantise(  # noqa: E731
        _unpack(raw[..., c0:c0 + 32 * D].unflatten(-1, (PAGE, D // 2))).movedim(1, -2),
        raw[..., s0:s0 + 4 * D].view(torch.float8_e4m3fn).unflatten(-1, (PAGE, D // 16)).movedim(1, -2),
        scale).movedim(-2, 1)
    return half(0, 64 * D, st["kv_scale"][0]), half(32 * D, 68 * D, st["kv_scale"][1])


def _rows(x, keep):
    """[B, kv, n, 64, D] pages as token rows [B, n * 64, kv, D], zero where keep [B, n * 64] is false."""
    x = x.flatten(2, 3).transpose(1, 2)
    return torch.where(keep[:, :, None, None], x, torch.zeros_like(x))


def _by_head(x, case):
    """[B, kv, S * group] rows as [B, heads, S]."""
    B, kv = x.shape[:2]
    return x.view(B, kv, case["S"], -1).permute(0, 1, 3, 2).reshape(B, case["heads"], case["S"])


def _mask_plain(st):
    """Ancestors (and itself) of every node as bits, int64 [B, S, words], and its position, int32 [B, S]."""
    B, S = st["parents"].shape
    node = torch.arange(S, device=st["parents"].device)
    fresh = node < st["new"][:, None]
    reach = (((st["parents"][..., None] == node) | (node[:, None] == node)) & fresh[..., None]).float()
    for _ in range(S.bit_length()):
        reach = (torch.matmul(reach, reach) > 0).float()
    reach = reach > 0
    start = (st["kv_lens"] - st["new"])[:, None]
    position = torch.where(fresh, start + reach.sum(-1) - 1, torch.zeros_like(start)).int()
    words = -(-S // PAGE)
    bits = torch.zeros((B, S, words * PAGE), dtype=torch.int64, device=node.device)
    bits[..., :S] = reach.long()
    return (bits.unflatten(-1, (words, PAGE)) << torch.arange(PAGE, device=node.device)).sum(-1), position


def _seen(st):
    """Which keys [B, S, n * 64] each query sees."""
    case = st["case"]
    pos = torch.arange(st["width"] * PAGE, device=st["kv_lens"].device)
    step = torch.arange(case["S"], device=pos.device)
    n, m = st["kv_lens"][:, None, None], st["new"][:, None, None]
    seen = (pos < n).expand(case["B"], case["S"], -1)
    if case["op"] == "tree":
        node = (pos - (n - m)).clamp(min=0, max=case["S"] - 1)  # [B, 1, keys]
        word = st["mask"].gather(2, (node // PAGE).expand(-1, case["S"], -1))
        seen = seen & ((pos < n - m) | ((word >> (node % PAGE)) & 1).bool())
    elif case["causal"]:
        seen = seen & (pos <= n - m + step[:, None])
    return seen & (step[:, None] < m)


def _logits_plain(st):
    """fp32 logits [B, kv, S * group, keys], -inf where a row does not see a key, and V [B, kv, keys, D]."""
    case = st["case"]
    B, S, heads, D = st["q"].shape
    kv = case["kv"]
    k, v = _read_plain(st)
    q = st["q"].float().view(B, S, kv, heads // kv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, k.flatten(2, 3).transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    hidden = ~_seen(st)[:, None, :, None, :]
    s.view(B, kv, S, heads // kv, -1).masked_fill_(hidden, -math.inf)
    return s, v.flatten(2, 3)


def _tree_plain(st):
    case = st["case"]
    B, S, heads, D = st["q"].shape
    kv = case["kv"]
    s, v = _logits_plain(st)
    here = torch.arange(v.shape[2], device=v.device) < st["kv_lens"][:, None]
    v = torch.where(here[:, None, :, None], v, torch.zeros_like(v))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.clamp(min=1e-30)
    o = o.view(B, kv, S, heads // kv, D).permute(0, 2, 1, 3, 4).reshape(B, S, heads, D)
    return {"out": o.bfloat16(), "lse": _by_head((m + total.log()).squeeze(-1), case)}


def _weigh_plain(st):
    case = st["case"]
    s, _ = _logits_plain(st)
    B, kv = s.shape[:2]
    lse = st["lse"].view(B, kv, -1, case["S"]).transpose(2, 3).flatten(2)
    off = torch.where(torch.isfinite(lse), lse, torch.full_like(lse, math.inf))
    w = s.sub_(off[..., None]).exp_().sum(2)
    return {"weights": st["weights"] + w if case["add"] else w}


def _rotate(x, st, at):
    """x fp32 [B, S, h, D] rotated by the rows of positions `at` [B, S]."""
    R = st["case"]["R"]
    if not R:
        return x
    row = st["rope"][at.long().clamp(0, st["rope"].shape[0] - 1)][:, :, None, :]
    c, s = row[..., :R // 2], row[..., R // 2:]
    if st["case"]["pairs"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., R:]), -1)


def _draft_plain(st):
    S, scale = st["case"]["S"], st["kv_scale"]
    mask, position = _mask_plain(st)
    step = torch.arange(S, device=mask.device)
    fresh = step < st["new"][:, None]
    q = _rotate(st["q"].float(), st, position)
    q = torch.where(fresh[:, :, None, None], q, torch.zeros_like(q)).bfloat16()
    base = st["kv_lens"] - st["new"]
    lens = base + st["path_lens"]
    local = (base - st["skipped"]).long()  # where the draft begins among the tail's pages
    keep = torch.arange(st["tail"].shape[1] * PAGE, device=mask.device) < local[:, None]
    seq, i = torch.nonzero(torch.arange(st["path"].shape[1], device=mask.device) < st["path_lens"][:, None],
                           as_tuple=True)
    node = st["path"][seq, i].long()

    def joined(x, old, head):
        rows = _rows(old, keep)
        rows[seq, local[seq] + i] = _dequantise(*_quantise(x, head), head)[seq, node]
        return rows.bfloat16()

    k, v = _read_plain(st, st["tail"])
    return {"mask": mask, "position": position, "lens": lens, "q": q,
            "k": joined(_rotate(st["k"].float(), st, position), k, scale[0]),
            "v": joined(st["v"].float(), v, scale[1])}


def _evict_plain(st):
    case = st["case"]
    B, kv, budget = case["B"], case["kv"], case["budget"]
    w, n = st["weights"], st["kv_lens"][:, None, None]
    place = torch.arange(w.shape[2], device=w.device)
    held = (place < case["first"]) | (place >= n - case["recent"])
    key = torch.where(held, torch.full_like(w, math.inf), w)
    key = torch.where(place < n, key, torch.full_like(w, -math.inf))
    most = st["to_table"].shape[1] * PAGE
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :min(budget, w.shape[2])]
    lens = torch.minimum(st["kv_lens"], torch.full_like(st["kv_lens"], budget))
    live = torch.arange(best.shape[2], device=w.device) < lens[:, None, None]
    best = torch.sort(torch.where(live, best, torch.full_like(best, w.shape[2])), dim=-1).values
    kept = torch.full((B, kv, budget), -1, dtype=torch.int32, device=w.device)
    kept[..., :best.shape[2]] = torch.where(live, best, torch.full_like(best, -1)).int()
    source = torch.where(live, best, torch.zeros_like(best))
    moved = torch.zeros((B, kv, most), device=w.device)
    moved[..., :best.shape[2]] = torch.where(live, w.gather(2, source), torch.zeros_like(moved[..., :best.shape[2]]))

    def rows(x):
        x = x.flatten(2, 3).gather(2, source[..., None].expand(-1, -1, -1, case["D"]))
        x = torch.where(live[..., None], x, torch.zeros_like(x))
        y = torch.zeros((B, kv, most, case["D"]), device=x.device)
        y[:, :, :x.shape[2]] = x
        return y.transpose(1, 2).contiguous().bfloat16()

    k, v = _read_plain(st)
    return {"kept": kept, "lens": lens, "weights": moved, "k": rows(k), "v": rows(v)}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import block_sparse_video_vsa_gb300 as vsa
        pool, table, kv_lens, scale = state["pool"], state["table"], state["kv_lens"], state["kv_scale"]
        if op == "tree":
            out, lse = vsa.cache_attn(state["q"], pool, table, kv_lens, q_lens=state["new"], tree=state["mask"],
                                      kv_scale=scale)
            return {"out": out, "lse": lse}
        if op == "weigh":
            before = state.get("weights")
            after = None if before is None else torch.empty_like(before)
            return {"weights": vsa.cache_weigh(state["q"], state["lse"], pool, table, kv_lens, q_lens=state["new"],
                                               causal=case["causal"], weights=before, out=after, kv_scale=scale)}
        if op == "evict":
            lens, kept, moved = vsa.cache_evict(pool, table, kv_lens, state["weights"], case["budget"],
                                                first=case["first"], recent=case["recent"],
                                                to_table=state["to_table"])
            k, v = vsa.cache_read(pool, state["to_table"], lens, state["to_table"].shape[1] * PAGE, kv_scale=scale)
            return {"kept": kept, "lens": lens, "weights": moved, "k": k, "v": v}
        mask, position = vsa.cache_tree(state["parents"], kv_lens, new_lens=state["new"])
        q = vsa.cache_append(pool, state["k"], state["v"], table, kv_lens, new_lens=state["new"],
                             rope=state.get("rope"), positions=position, interleaved=case["pairs"], q=state["q"],
                             kv_scale=scale)
        lens = vsa.cache_accept(pool, table, kv_lens, state["new"], state["path"], state["path_lens"])
        k, v = vsa.cache_read(pool, state["tail"], lens - state["skipped"], state["tail"].shape[1] * PAGE,
                              kv_scale=scale)
        return {"mask": mask, "position": position, "lens": lens, "q": q, "k": k, "v": v}
    if op == "tree":
        return _tree_plain(state)
    if op == "weigh":
        return _weigh_plain(state)
    return _evict_plain(state) if op == "evict" else _draft_plain(state)


def work(case):
    B, kv, D, op = case["B"], case["kv"], case["D"], case["op"]
    kv_lens, new = _lens(case)
    token = 2 * kv * D * 9 // 16  # one token's codes and scales
    width = -(-max(kv_lens) // PAGE)
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in kv_lens)
        back = B * (-(-min(case["budget"], max(kv_lens)) // PAGE)) * PAGE * kv
        return {"bytes": sum(kv_lens) * kv * 4 + B * kv * case["budget"] * 4 + back * 4 + 2 * kept * token
                + kept * token + 2 * back * D * 2, "flops": 2 * kept * kv * D}
    rows = sum(new) * case["heads"]
    if op == "draft":
        tail = max(-(-n // PAGE) - (n - m) // PAGE for n, m in zip(kv_lens, new))
        words = -(-case["S"] // PAGE)
        put = sum(new) * ((case["heads"] + 2 * kv) * D * 2 + token) + B * case["S"] * case["heads"] * D * 2
        return {"bytes": put + 2 * B * tail * PAGE * kv * D * 2 + B * case["S"] * (8 + 8 * words)
                + max(new) * case["R"] * 4,
                "flops": sum(new) * (3 * (case["heads"] + kv) * case["R"] + 2 * kv * D * 2)}
    if op == "tree":
        pairs = sum(m * (n - m + 1) for n, m in zip(kv_lens, new))
        return {"bytes": sum(kv_lens) * token + rows * D * 2 + B * case["S"] * case["heads"] * (D * 2 + 4)
                + sum(m * (-(-m // PAGE)) * 8 for m in new), "flops": 4 * pairs * case["heads"] * D}
    pairs = sum(m * n - (m * (m - 1) // 2 if case["causal"] else 0) for n, m in zip(kv_lens, new))
    places = B * kv * width * PAGE * 4
    return {"bytes": sum(kv_lens) * token // 2 + rows * (D * 2 + 4) + places * (2 if case["add"] else 1),
            "flops": 2 * pairs * case["heads"] * D}


# ------------------------------------------------- the definitions in 64 bits
def _nearest(y, values):
    """The nearest of the ascending `values` (index parity = even/odd code), ties to the even index."""
    at = torch.searchsorted(values, y.contiguous()).clamp(1, len(values) - 1)
    lo, hi = values[at - 1], values[at]
    up = (y - lo > hi - y) | ((y - lo == hi - y) & (at % 2 == 0))
    return torch.where(up, hi, lo)


def _stored(x, head):
    """What the cache holds of float64 x [..., kv, D]."""
    dev = x.device
    small = [m * 2.0 ** -9 for m in range(8)]
    e4m3 = torch.tensor(small + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=dev)
    y = (x / head[:, None]).reshape(*x.shape[:-1], -1, 16)
    s = _nearest((y.abs().amax(-1) / 6).clamp(max=448.0), e4m3)[..., None]
    z = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    grid = torch.tensor(_GRID, dtype=torch.float64, device=dev)
    return (torch.sign(z) * _nearest(z.abs().clamp(max=6.0), grid) * s).reshape(x.shape) * head[:, None]


def _token_rows(st, b):
    """Sequence b's cached K and V as float64 [kv_len, kv, D], read byte by byte position."""
    D, n = st["case"]["D"], int(st["kv_lens"][b])
    t = torch.arange(n, device=st["pool"].device)
    raw = st["pool"][st["table"][b].long()[t // PAGE]]
    e4m3 = torch.arange(256, dtype=torch.uint8, device=raw.device).view(torch.float8_e4m3fn).double()
    grid = torch.tensor(_GRID, dtype=torch.float64, device=raw.device)
    ch = torch.arange(D, device=raw.device)
    got = []
    for c0, s0, head in ((0, 64 * D, st["kv_scale"][0]), (32 * D, 68 * D, st["kv_scale"][1])):
        slot = (t % PAGE)[:, None, None]
        byte = raw.gather(2, (c0 + slot * (D // 2) + (ch // 2)).expand(n, raw.shape[1], D)).int()
        code = torch.where(ch % 2 == 1, byte >> 4, byte & 15)
        scale = e4m3[raw.gather(2, (s0 + slot * (D // 16) + ch // 16).expand(n, raw.shape[1], D)).int()]
        got.append(grid[code & 7] * torch.where(code > 7, -1.0, 1.0) * scale * head.double()[:, None])
    return got


def _lines(parents, m):
    """For each of m nodes the nodes from its root down to itself."""
    lines = []
    for i in range(m):
        lines.append((lines[parents[i]] if parents[i] >= 0 else []) + [i])
    return lines


def _exact_draft(st, case):
    B, S, kv, D, R = case["B"], case["S"], case["kv"], case["D"], case["R"]
    dev, half = st["pool"].device, case["R"] // 2
    words = -(-S // PAGE)
    mask = [[[0] * words for _ in range(S)] for _ in range(B)]
    position = torch.zeros((B, S), dtype=torch.int32, device=dev)
    q = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    shape = (B, st["tail"].shape[1] * PAGE, kv, D)
    k, v = torch.zeros(shape, dtype=torch.float64, device=dev), torch.zeros(shape, dtype=torch.float64, device=dev)
    left = torch.arange(half, device=dev) * (2 if case["pairs"] else 1)
    right = left + (1 if case["pairs"] else half)
    lens = []
    for b in range(B):
        n, m = int(st["kv_lens"][b]), int(st["new"][b])
        lines = _lines(st["parents"][b].tolist(), m)
        for i, line in enumerate(lines):
            for j in line:
                bit = 1 << (j % PAGE)
                mask[b][i][j // PAGE] += bit - (1 << PAGE if j % PAGE == PAGE - 1 else 0)
        depth = torch.tensor([len(line) - 1 for line in lines], device=dev)
        position[b, :m] = n - m + depth
        turned = {}
        for x in "qk":
            y = st[x][b, :m].double()
            if R:
                z = torch.complex(y[..., left], y[..., right])
                f = st["rope"][n - m + depth].double()
                z = z * torch.complex(f[:, :half], f[:, half:])[:, None]
                y[..., left], y[..., right] = z.real, z.imag
            turned[x] = y
        q[b, :m] = turned["q"]
        a = int(st["path_lens"][b])
        path = st["path"][b, :a].long()
        first = int(st["skipped"][b])
        rows = _token_rows(st, b)
        here = n - m - first
        for to, old, fresh, head in ((k, rows[0], turned["k"], st["kv_scale"][0]),
                                     (v, rows[1], st["v"][b, :m].double(), st["kv_scale"][1])):
            to[b, :here] = old[first:n - m]
            to[b, here:here + a] = _stored(fresh[path], head.double())
        lens.append(n - m + a)
    return {"mask": torch.tensor(mask, dtype=torch.int64, device=dev), "position": position,
            "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "q": q, "k": k, "v": v}


def _exact_evict(st, case):
    B, kv, D, budget = case["B"], case["kv"], case["D"], case["budget"]
    dev = st["pool"].device
    most = st["to_table"].shape[1] * PAGE
    kept = torch.full((B, kv, budget), -1, dtype=torch.int32, device=dev)
    moved = torch.zeros((B, kv, most), dtype=torch.float64, device=dev)
    k, v = (torch.zeros((B, most, kv, D), dtype=torch.float64, device=dev) for _ in range(2))
    lens = []
    for b in range(B):
        n = int(st["kv_lens"][b])
        rows = _token_rows(st, b)
        size = min(n, budget)
        lens.append(size)
        for h in range(kv):
            w = st["weights"][b, h, :n].double()
            chosen = torch.ones(n, dtype=torch.bool, device=dev)
            if n > budget:
                a, z = case["first"], n - case["recent"]
                chosen[a:z] = False
                want = budget - case["first"] - case["recent"]
                if want:
                    middle = w[a:z]
                    edge = middle.sort().values[len(middle) - want]
                    over = middle > edge
                    same = middle == edge
                    chosen[a:z] = over | (same & (same.cumsum(0) <= want - over.sum()))
            at = torch.nonzero(chosen)[:, 0]
            kept[b, h, :size] = at.int()
            moved[b, h, :size] = w[at]
            k[b, :size, h], v[b, :size, h] = rows[0][at, h], rows[1][at, h]
    return {"kept": kept, "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "weights": moved, "k": k, "v": v}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "draft":
        return _exact_draft(st, case)
    if case["op"] == "evict":
        return _exact_evict(st, case)
    B, kv, S, heads, D = case["B"], case["kv"], case["S"], case["heads"], case["D"]
    dev = st["pool"].device
    out = torch.zeros((B, S, heads, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, heads, S), -math.inf, dtype=torch.float64, device=dev)
    total = torch.zeros((B, kv, st["width"] * PAGE), dtype=torch.float64, device=dev)
    if "weights" in st:
        total += st["weights"]
    for b in range(B):
        n, m = int(st["kv_lens"][b]), int(st["new"][b])
        k, v = _token_rows(st, b)
        t = torch.arange(n, device=dev)
        if case["op"] == "tree":
            mask = (t < n - m).repeat(m, 1)
            for i, line in enumerate(_lines(st["parents"][b].tolist(), m)):
                mask[i, [n - m + j for j in line]] = True
        else:
            mask = t <= torch.arange(m, device=dev)[:, None] + (n - m if case["causal"] else n)
        for h in range(kv):
            for j in range(h * heads // kv, (h + 1) * heads // kv):
                s = (st["q"][b, :m, j].double() @ k[:, h].T) / math.sqrt(D)
                s = torch.where(mask, s, -math.inf)
                if case["op"] == "weigh":
                    off = st["lse"][b, j, :m].double()
                    w = torch.exp(s - off[:, None])
                    total[b, h, :n] += torch.where(torch.isfinite(off)[:, None], w, 0.0).sum(0)
                else:
                    lse[b, j, :m] = torch.logsumexp(s, -1)
                    out[b, :m, j] = torch.softmax(s, -1).nan_to_num(0.0) @ v[:, h]
    return {"weights": total} if case["op"] == "weigh" else {"out": out, "lse": lse}
