"""Plain statements in 64 bits of drafted trees over the 4-bit cache, of attention weights and of eviction,
for the tests (imported, not collected).  Builds on cache_ref; nothing here is shared with the package."""
import numpy as np

import cache_ref as ref


def lines(parents, m):
    """For each of m nodes the nodes from its root down to itself."""
    got = []
    for i in range(m):
        p = int(parents[i])
        got.append((got[p] if 0 <= p < i else []) + [i])
    return got


def masks(parents, new_lens):
    """(uint64 [B, S, words] as int64, depths int32 [B, S]) of parents [B, S]."""
    B, S = parents.shape
    bits = np.zeros((B, S, -(-S // 64)), np.uint64)
    depth = np.zeros((B, S), np.int32)
    for b in range(B):
        for i, line in enumerate(lines(parents[b], int(new_lens[b]))):
            for j in line:
                bits[b, i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
            depth[b, i] = len(line) - 1
    return bits.view(np.int64), depth


def seen_by_bits(bits, n, m):
    """bool [m, n]: the context, and of the last m tokens those of each row's bits (int64 [S, words])."""
    seen = np.zeros((m, n), bool)
    words = bits.view(np.uint64)
    for i in range(m):
        for x in range(n):
            j = x - (n - m)
            seen[i, x] = j < 0 or bool((words[i, j // 64] >> np.uint64(j % 64)) & np.uint64(1))
    return seen


def attention(q, pool, table, kv_lens, q_lens, seen, sm_scale, kv_scale, pages=None):
    """As cache_ref.attention, the keys of row i of sequence b given by seen[b][i] (bool [m, n]); with pages
    (per sequence and head) only tokens of those pages."""
    B, Sq, heads, D = q.shape
    kv = pool.shape[1]
    G = heads // kv
    out, wabs = np.zeros((2, B, Sq, heads, D))
    lse = np.full((B, heads, Sq), -np.inf)
    mag, inv, count = np.zeros((3, B, heads, Sq))
    for b in range(B):
        n, m = int(kv_lens[b]), int(q_lens[b])
        k, v = ref.sequence(pool, table[b], n, D, kv_scale)
        for h in range(kv):
            inside = np.ones(n, bool) if pages is None else np.isin(np.arange(n) // 64, pages[b, h])
            for j in range(h * G, (h + 1) * G):
                for i in range(m):
                    x = np.flatnonzero(seen[b][i] & inside)
                    if not len(x):
                        continue
                    s = k[x, h] @ q[b, i, j] * sm_scale
                    p = np.exp(s - s.max())
                    w = p / p.sum()
                    out[b, i, j] = w @ v[x, h]
                    wabs[b, i, j] = w @ np.abs(v[x, h])
                    lse[b, j, i] = s.max() + np.log(p.sum())
                    mag[b, j, i] = (np.abs(k[x, h]) @ np.abs(q[b, i, j])).max() * sm_scale
                    inv[b, j, i] = np.abs(v[x, h]).max() / p.sum()
                    count[b, j, i] = len(x)
    return out, lse, dict(wabs=wabs, mag=mag, inv=inv, seen=count)


def weigh(q, lse, pool, table, kv_lens, q_lens, causal, sm_scale, kv_scale, before):
    """float64 (weights [B, kv, places], bound on a kernel's error).

    A logit is a fp32 sum of D exact products, (D + 4) 2^-24 of sum |q k| off; its argument of the
    exponential takes four more roundings, of the scale's factors, the log-sum and their sum: 4 2^-24 (|s| +
    |lse|).  The exponential is 2^-22 off, and a sum of N positive numbers N 2^-24.  What underflows is below
    2^-126 a row."""
    B, Sq, heads, D = q.shape
    kv = pool.shape[1]
    G = heads // kv
    out = np.array(before, np.float64)
    off = np.zeros_like(out)
    for b in range(B):
        n, m = int(kv_lens[b]), int(q_lens[b])
        k, _ = ref.sequence(pool, table[b], n, D, kv_scale)
        x = np.arange(n)
        for h in range(kv):
            for j in range(h * G, (h + 1) * G):
                for i in range(m):
                    if not np.isfinite(lse[b, j, i]):
                        continue
                    see = x <= (n - m + i if causal else n)
                    s = k[:, h] @ q[b, i, j] * sm_scale
                    w = np.where(see, np.exp(np.where(see, s - lse[b, j, i], 0)), 0)
                    d = (D + 4) * 2.0 ** -24 * (np.abs(k[:, h]) @ np.abs(q[b, i, j])) * sm_scale
                    d = d + 4 * 2.0 ** -24 * (np.abs(s) + abs(lse[b, j, i]))
                    out[b, h, :n] += w
                    off[b, h, :n] += w * (np.expm1(d) + 2.0 ** -22 + (G * Sq + 8) * 2.0 ** -24) + 2.0 ** -126
    return out, off * 1.01 + 2.0 ** -23 * np.abs(out)


def choose(weights, n, budget, first, recent):
    """The places kept of one row's weights [>= n], ascending."""
    if n <= budget:
        return np.arange(n)
    middle = np.arange(first, n - recent)
    w = weights[middle].astype(np.float64)
    w = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(weights[middle])
    order = np.lexsort((middle, nan, -w))  # by weight, then numbers before NaN, then place
    picked = middle[order[:budget - first - recent]]
    return np.sort(np.concatenate((np.arange(first), picked, np.arange(n - recent, n))))


def evict(pool, table, weights, kv_lens, budget, first, recent, D, to_table=None):
    """(pool, kept, lens, weights) after an eviction, on copies."""
    old, pool, weights = pool, pool.copy(), np.array(weights, np.float32)
    B, kv = weights.shape[:2]
    lens = np.minimum(kv_lens, budget).astype(np.int32)
    kept = np.full((B, kv, budget), -1, np.int32)
    to = table if to_table is None else to_table
    moved = weights.copy() if to_table is None else np.zeros((B, kv, 64 * to.shape[1]), np.float32)
    for b in range(B):
        n = int(kv_lens[b])
        for h in range(kv):
            at = choose(weights[b, h], n, budget, first, recent)
            kept[b, h, :len(at)] = at
            moved[b, h, :len(at)] = weights[b, h, at]
            if to_table is None and n > budget:
                moved[b, h, len(at):n] = 0
            if to_table is None and n <= budget:
                continue
            move(old, pool, table[b], to[b], at, np.arange(len(at)), h, D)
    return pool, kept, lens, moved


def move(old, pool, from_row, to_row, source, place, h, D):
    """Copies tokens `source` of old's head h (pages from_row) to places `place` of to_row in pool."""
    for side in (0, 1):
        for s, t in zip(source, place):
            a, b = old[from_row[s // 64], h], pool[to_row[t // 64], h]
            for width, at in ((D // 2, side * 32 * D), (D // 16, 64 * D + side * 4 * D)):
                x, y = at + (s % 64) * width, at + (t % 64) * width
                b[y:y + width] = a[x:x + width]
