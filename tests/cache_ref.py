"""Plain statement of the 4-bit paged cache for the tests (imported, not collected).

`append` follows the storing rule step by step in fp32 (numpy rounds every
product and sum), so it gives the bytes the library has to give; `attention`
and `stored64` are the definitions in 64 bits.  Nothing here is shared with
the package."""
import numpy as np

PAGE = 64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])  # 0 .. 448


def nearest_code(x, values):
    """Index of the nearest of the ascending `values` (x >= 0, saturating), ties to the even index."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    dlo, dhi = x - values[lo], values[hi] - x
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x, head_scale):
    """fp32 x [..., kv, D] -> (codes uint8 [..., kv, D], scale bytes uint8 [..., kv, D / 16])."""
    f = np.float32
    inv = f(1) / np.asarray(head_scale, f)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.asarray(x, f) * inv[:, None]
    y = np.where(np.isnan(y), f(0), y)
    y = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    with np.errstate(over="ignore"):
        want = np.abs(y).max(-1) * f(1 / 6)
    s = nearest_code(np.minimum(want, f(448)), E4M3)
    sf = E4M3[s].astype(f)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        r = np.where(sf > 0, f(1) / sf, f(0))
        z = y * r[..., None]
    code = nearest_code(np.minimum(np.abs(z), f(6)), E2M1) + 8 * np.signbit(z)
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def value(code, scale, head_scale):
    """The float64 numbers that codes [..., kv, D] and scale bytes [..., kv, D / 16] stand for."""
    code = np.asarray(code)
    v = E2M1[code & 7] * np.where(code > 7, -1.0, 1.0)
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16) * E4M3[np.minimum(scale, 126)][..., None]
    return v.reshape(code.shape) * np.asarray(head_scale, np.float64)[:, None]


def rotate32(x, rope_rows, R, interleaved):
    """fp32 x [..., h, D] by rows [..., R] of the table, every product and sum rounded."""
    if not R:
        return np.asarray(x, np.float32)
    y = np.array(x, np.float32)
    c, s = (rope_rows[..., None, i * (R // 2):(i + 1) * (R // 2)].astype(np.float32) for i in (0, 1))
    left = slice(0, R, 2) if interleaved else slice(0, R // 2)
    right = slice(1, R, 2) if interleaved else slice(R // 2, R)
    a, b = y[..., left].copy(), y[..., right].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., left] = a * c - b * s
        y[..., right] = b * c + a * s
    return y


def put(pool, page, slot, h, D, side, codes, scales):
    """Writes one token's codes [D] and scale bytes [D / 16] of kv head h (side 0: K, 1: V)."""
    at = pool[page, h]
    c0, s0 = side * 32 * D + slot * (D // 2), 64 * D + side * 4 * D + slot * (D // 16)
    at[c0:c0 + D // 2] = codes[0::2] | (codes[1::2] << 4)
    at[s0:s0 + D // 16] = scales


def get(pool, table, n, h, D, side):
    """Codes [n, D] and scale bytes [n, D / 16] of a sequence's tokens 0 .. n - 1 (table: its row)."""
    t = np.arange(n)
    rows = pool[table[t // PAGE], h]
    c = side * 32 * D + (t % PAGE)[:, None] * (D // 2) + np.arange(D // 2)
    byte = np.take_along_axis(rows, c, 1)
    codes = np.stack((byte & 15, byte >> 4), -1).reshape(n, D)
    s = 64 * D + side * 4 * D + (t % PAGE)[:, None] * (D // 16) + np.arange(D // 16)
    return codes, np.take_along_axis(rows, s, 1)


def sequence(pool, table, n, D, kv_scale):
    """float64 K, V [n, kv, D] of a sequence."""
    kv = pool.shape[1]
    out = []
    for side in (0, 1):
        parts = [get(pool, table, n, h, D, side) for h in range(kv)]
        code = np.stack([p[0] for p in parts], 1) if n else np.zeros((0, kv, D), np.uint8)
        scale = np.stack([p[1] for p in parts], 1) if n else np.zeros((0, kv, D // 16), np.uint8)
        out.append(value(code, scale, kv_scale[side]))
    return out


def append(pool, table, k, v, kv_lens, new_lens, kv_scale, rope=None, positions=None, interleaved=False):
    """The storing rule on a copy of `pool`; k, v float32 [B, S, kv, D]."""
    pool = pool.copy()
    B, S, kv, D = k.shape
    R = 0 if rope is None else rope.shape[1]
    for b in range(B):
        n, m = int(kv_lens[b]), int(new_lens[b])
        for i in range(m):
            at = n - m + i
            pos = at if positions is None else int(positions[b, i])
            x = rotate32(k[b, i], rope[pos] if R else None, R, interleaved)
            for side, row in ((0, x), (1, v[b, i])):
                codes, scales = quantise(row, kv_scale[side])
                for h in range(kv):
                    put(pool, table[b, at // PAGE], at % PAGE, h, D, side, codes[h], scales[h])
    return pool


def attention(q, pool, table, kv_lens, q_lens, causal, sm_scale, kv_scale, page_sel=None):
    """float64 (out [B, Sq, heads, D], lse [B, heads, Sq], and what bounds the error of each row:
    sum of w |v| per channel, largest sum of |q k| in logits, 1 / sum of exp(s - max), keys seen)."""
    B, Sq, heads, D = q.shape
    kv = pool.shape[1]
    G = heads // kv
    out, wabs = np.zeros((2, B, Sq, heads, D))
    lse = np.full((B, heads, Sq), -np.inf)
    mag, inv, seen = np.zeros((3, B, heads, Sq))
    for b in range(B):
        n, m = int(kv_lens[b]), int(q_lens[b])
        k, v = sequence(pool, table[b], n, D, kv_scale)
        for h in range(kv):
            t = np.arange(n)
            if page_sel is not None:
                t = t[np.isin(t // PAGE, page_sel[b, h][page_sel[b, h] >= 0])]
            for j in range(h * G, (h + 1) * G):
                for i in range(m):
                    x = t[t <= n - m + i] if causal else t
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
                    seen[b, j, i] = len(x)
    return out, lse, dict(wabs=wabs, mag=mag, inv=inv, seen=seen)


def attention_bounds(out, lse, info, D):
    """How far a kernel's out (bf16) and lse (fp32) may be from the definition.

    A logit is a fp32 sum of D products (D + 4 roundings of at most 2^-24 of sum |q k|), so a weight is
    off by a factor within exp(+-2 d), d = (D + 4) 2^-24 mag, plus 2^-21 for exp2 and the sums; P is
    rounded to fp16: 2^-11 of each weight, or 2^-25 of the largest where that is subnormal; the result
    to bf16: 2^-8 of it."""
    d = (D + 4) * 2.0 ** -24 * info["mag"]
    w = 2.0 ** -11 + 2 * d + 2.0 ** -21
    w = np.moveaxis(w, 1, 2)[..., None]
    sub = np.moveaxis(info["inv"] * info["seen"], 1, 2)[..., None] * 2.0 ** -25
    soft = (w * info["wabs"] + sub) * 1.01
    lim_out = soft + 2.0 ** -8 * (np.abs(out) + soft) + 1e-30
    with np.errstate(invalid="ignore"):
        lim_lse = np.where(np.isfinite(lse), d + 2.0 ** -21 * (2 + np.abs(lse)), 0.0)
    return lim_out, lim_lse
