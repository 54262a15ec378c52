"""Plain 64-bit implementations of the operators between the GEMVs (numpy, no code of the library), for the
tests: head norms and rotation, the 4-bit cache (bytes both ways), attention with a bound on its rounding,
and sampling."""
import numpy as np


def norm(x, w, eps):
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def rope(x, pos, freq, pairing):
    """x [T, H, D]; pairing 0: (i, i + R/2), 1: (2i, 2i + 1)."""
    if freq is None or len(freq) == 0:
        return x.copy()
    R = 2 * len(freq)
    y = x.copy()
    a = pos.astype(np.float64)[:, None, None] * freq
    c, s = np.cos(a), np.sin(a)
    i = np.arange(R // 2)
    u, v = (i, i + R // 2) if pairing == 0 else (2 * i, 2 * i + 1)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., v] * c + x[..., u] * s
    return y


def quantize(x):
    """x [..., D] -> codes, d, m per 64 dimensions (d, m as fp16)."""
    g = x.reshape(*x.shape[:-1], -1, 64)
    lo, hi = g.min(-1), g.max(-1)
    d = np.minimum(((hi - lo) / 15).astype(np.float32), np.float32(65504)).astype(np.float16)
    m = np.clip(lo.astype(np.float32), -65504, 65504).astype(np.float16)
    dd, mm = d.astype(np.float64)[..., None], m.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(dd > 0, (g - mm) / dd, 0.0)
    return np.clip(np.rint(y), 0, 15).astype(np.uint8).reshape(x.shape), d, m


def values(code, d, m):
    """The fp32 values d * code + m (exact before their one rounding)."""
    g = code.reshape(*code.shape[:-1], -1, 64).astype(np.float64)
    v = g * d.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]
    return v.astype(np.float32).reshape(code.shape)


def places(D):
    t = np.arange(16)
    s = (t & 2) | (((t ^ (t >> 2)) & 1) << 2)
    return np.arange(D // 32)[None, :] ^ (s & (D // 32 - 1))[:, None]


def store(cache, page, slot, part, code, d, m):
    """Writes token rows [T, H, D] into cache uint8 [pages, H, page/16, 18 D] at the slots, in place."""
    T, H, D = code.shape
    pl = places(D)
    for i in range(T):
        p = int(slot[i])
        if p < 0 or p >= cache.shape[0] * page:
            continue
        pg, blk, t = p // page, p % page // 16, p % 16
        for h in range(H):
            at = cache[pg, h, blk, part * 9 * D:(part + 1) * 9 * D]
            b = (code[i, h, 0::2] | code[i, h, 1::2] << 4).reshape(D // 32, 16)
            row = np.empty_like(b)
            row[pl[t]] = b
            at[t * D // 2:(t + 1) * D // 2] = row.reshape(-1)
            sc = np.stack([d[i, h], m[i, h]], -1).view(np.uint8).reshape(-1)
            at[8 * D + t * D // 16:8 * D + (t + 1) * D // 16] = sc


def load(cache, page, pg, part):
    """All values of page pg: [H, page, D] in fp64 (d * code + m unrounded)."""
    _, H, nb, w = cache.shape
    D = w // 18
    at = cache[pg, :, :, part * 9 * D:(part + 1) * 9 * D]
    codes = at[..., :8 * D].reshape(H, nb, 16, D // 32, 16)
    codes = np.take_along_axis(codes, places(D)[None, None, :, :, None].repeat(H, 0).repeat(nb, 1), axis=3)
    b = codes.reshape(H, nb, 16, D // 2)
    c = np.stack([b & 15, b >> 4], -1).reshape(H, nb, 16, D // 64, 64).astype(np.float64)
    dm = at[..., 8 * D:].copy().view(np.float16).reshape(H, nb, 16, D // 64, 2).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return (c * dm[..., :1] + dm[..., 1:]).reshape(H, nb * 16, D)


def attention(q, start, cache, page, table, lens, scale, out):
    """q [T, Hq, D] fp16.  Returns the result written over a copy of `out` (fp64) and a bound on how far the
    kernel may be from it.

    The bound.  A cache value enters a product as fp16, off by 2^-11 of itself at most, so a score is off by
    e = scale * sum |q k| * (2^-11 + 2^-13) (the second term for the fp32 sums: at most 256 additions of
    products, 2^-24 each, and their truncation in the matrix unit, taken fourfold).  A normalized weight is
    then off by a factor within exp(+-2 e), e the row's largest; it is rounded to fp16 (2^-11; weights below
    2^-21 of the reference lose 2^-32 of it absolutely, at most 2^-24 of all weight per place) and so are the
    values (2^-11).  The fp32 sums add less than 2^-13.  The output is rounded to fp16 (2^-11 of itself, at
    least 2^-25)."""
    want = out.astype(np.float64).copy()
    bound = np.zeros_like(want)
    T, Hq, D = q.shape
    pages, Hk = cache.shape[:2]
    G = Hq // Hk
    for s in range(len(lens)):
        a, b = int(start[s]), int(start[s + 1])
        L = max(0, min(int(lens[s]), table.shape[1] * page))
        np_ = (L + page - 1) // page
        k = np.zeros((Hk, np_ * page, D))
        v = np.zeros((Hk, np_ * page, D))
        there = np.zeros(np_ * page, bool)
        for i in range(np_):
            pg = int(table[s, i])
            if 0 <= pg < pages:
                k[:, i * page:(i + 1) * page] = load(cache, page, pg, 0)
                v[:, i * page:(i + 1) * page] = load(cache, page, pg, 1)
                there[i * page:(i + 1) * page] = True
        for t in range(a, b):
            last = L - (b - a) + (t - a)
            see = np.flatnonzero(there & (np.arange(np_ * page) <= last))
            for h in range(Hq):
                if len(see) == 0:
                    want[t, h] = 0.0
                    continue
                qq = q[t, h].astype(np.float64)
                kk, vv = k[h // G][see], v[h // G][see]
                x = scale * (kk @ qq)
                e = (scale * (np.abs(kk) @ np.abs(qq))).max() * (2.0 ** -11 + 2.0 ** -13)
                p = np.exp(x - x.max())
                p /= p.sum()
                o = p @ vv
                want[t, h] = o
                mag = p @ np.abs(vv)
                rel = np.expm1(2 * e) + 2 * 2.0 ** -11 + 2.0 ** -13
                bound[t, h] = mag * rel * 1.01 + np.abs(vv).max() * len(see) * 2.0 ** -31 + np.abs(o) * 2.0 ** -11 + 2.0 ** -25
    return want, bound


def sample(x, t, k, p, mp, u):
    """The token of one row by sorting, in 64 bits (filters of None are off)."""
    x = x.astype(np.float32)
    ok = ~np.isnan(x) & (x > -np.inf)
    if not ok.any():
        return -1
    x = np.where(ok, x, -np.inf) + np.float32(0)
    order = np.lexsort((np.arange(len(x)), -x))
    if t is not None and not t > 0:
        return int(order[0])
    z = x[order].astype(np.float64) / (1.0 if t is None else float(t))
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == x[order[0]], 1.0, np.exp(z - z[0]))
    keep = ok[order]
    if k is not None and 0 < k < len(x):
        keep &= np.arange(len(x)) < k
    w = np.where(keep, w, 0.0)
    if p is not None and float(p) < 1:
        keep &= (np.cumsum(w) - w) < max(0.0, float(p)) * w.sum()
    if mp is not None:
        keep &= w >= float(mp)
    keep[0] = True
    full = np.zeros(len(x))
    full[order] = np.where(keep, w, 0.0)
    c = np.cumsum(full)
    hit = np.flatnonzero(c > float(u) * c[-1])
    return int(hit[0]) if len(hit) else int(np.flatnonzero(full)[-1])
