"""float64 CPU oracle of the decoder-layer operators: RMS norm, rotary
positions, the 8-bit key/value cache and attention over it.  Test
infrastructure: plain loops over the definitions, no code of the package."""
from __future__ import annotations

import numpy as np

E4M3, INT8 = 0, 1
TOP = {E4M3: 448.0, INT8: 127.0}


def _e4m3_table():
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if s else x)
    return v


E4M3_VALUES = _e4m3_table()


def e4m3_codes(x):
    """Nearest e4m3 code of x, ties to the even mantissa, saturating."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    grid = E4M3_VALUES[:127]                       # 0 .. 448, ascending; code = index
    hi = np.clip(np.searchsorted(grid, mag, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = mag - grid[lo], grid[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def codes(x, fmt):
    if fmt == E4M3:
        return e4m3_codes(x)
    return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)


def values(c, fmt):
    c = np.asarray(c, np.uint8)
    return E4M3_VALUES[c] if fmt == E4M3 else c.view(np.int8).astype(np.float64)


def least_scale(top, fmt):
    """The least power of two >= 2^-126 with top / scale within the range."""
    if top == 0:
        return 2.0 ** -126
    m, e = np.frexp(top / TOP[fmt])                # m in [0.5, 1)
    return 2.0 ** max(-126, int(e) - (1 if m == 0.5 else 0))


def rmsnorm(x, r, w, eps):
    s = x + r if r is not None else x
    n = s / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps)
    return s, n * w if w is not None else n


def rope(x, positions, inv_freq, axis, halves):
    """x [T, H, D], positions [A, T], axis [rot / 2]."""
    y = x.copy()
    n = len(inv_freq)
    for i in range(n):
        a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
        ang = positions[axis[i]].astype(np.float64) * inv_freq[i]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def append(x, cache, scale, table, kv_lens, cu_q, fmt):
    """Writes x [T, heads, D] into cache (codes [blocks, heads, block, D],
    scale [blocks, heads]) in place, by the rule of the scale."""
    block = cache.shape[2]
    for b, kv in enumerate(kv_lens):
        n = cu_q[b + 1] - cu_q[b]
        p0 = max(0, kv - n)
        for j in range(p0 // block, -(-kv // block)):
            lo, hi = max(p0, j * block), min(kv, (j + 1) * block)
            if lo >= hi:
                continue
            c = table[b][j]
            for h in range(cache.shape[1]):
                new = x[cu_q[b] + lo - (kv - n):cu_q[b] + hi - (kv - n), h]
                finite = np.where(np.isnan(new), 0.0, np.clip(new, -3.3895313892515355e38, 3.3895313892515355e38))
                s = least_scale(np.abs(finite).max(), fmt)
                kept = lo - j * block
                if kept:
                    old = float(scale[c, h])
                    if old >= s:
                        s = old
                    else:
                        cache[c, h, :kept] = codes(values(cache[c, h, :kept], fmt) * (old / s), fmt)
                cache[c, h, kept:hi - j * block] = codes(finite / s, fmt)
                scale[c, h] = s


def gather(cache, scale, row, kv, fmt):
    """Tokens 0 .. kv-1 of one sequence as values [heads, kv, D]."""
    block = cache.shape[2]
    v = [values(cache[row[j]], fmt) * scale[row[j]].astype(np.float64)[:, None, None] for j in range(-(-kv // block))]
    if not v:
        return np.zeros((cache.shape[1], 0, cache.shape[3]))
    return np.concatenate(v, 1)[:, :kv]


def attention(q, kc, vc, ks, vs, table, kv_lens, cu_q, fmt, scale, window=0):
    """out [T, Hq, D], lse [T, Hq] and an elementwise tolerance for each: the
    bf16 rounding of out (2^-8 of it), the weights' rounding to f16 (2^-11 of
    sum p |v|), and the fp32 error of the scores (2^-23 a term of q.k, and
    2^-25 of the row's largest q where f16 holds q), which moves every weight
    and their sum."""
    T, Hq, D = q.shape
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, ltol = np.full((T, Hq, D), 1e-30), np.zeros((T, Hq))
    for b, kv in enumerate(kv_lens):
        n = cu_q[b + 1] - cu_q[b]
        if n == 0:
            continue
        k, v = gather(kc, ks, table[b], kv, fmt), gather(vc, vs, table[b], kv, fmt)
        group = Hq // k.shape[0]
        for i in range(n):
            pos = kv - n + i
            lo = max(0, pos + 1 - window) if window else 0
            if pos < lo:
                continue
            for h in range(Hq):
                kk, vv = k[h // group, lo:pos + 1], v[h // group, lo:pos + 1]
                t = cu_q[b] + i
                s = scale * (kk @ q[t, h])
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[t, h] = p @ vv / l
                lse[t, h] = m + np.log(l)
                mag = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
                sub = abs(scale) * 2.0 ** -25 * np.abs(q[t, h]).max() * np.abs(kk).sum(-1).max()
                ds = D * 2.0 ** -23 * mag + sub + 2.0 ** -22 * (np.abs(s).max() + 1)
                av = p @ np.abs(vv) / l
                tol[t, h] = (2.0 ** -8 * np.abs(out[t, h]) + (2.0 ** -11 + 2 * ds + 2.0 ** -18) * av
                             + 2.0 ** -28 * np.abs(vv).max(0) + 1e-30)
                ltol[t, h] = ds + 2.0 ** -21 * abs(lse[t, h]) + 2.0 ** -20
    return out, lse, tol, ltol
