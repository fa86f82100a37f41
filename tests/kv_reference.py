"""Plain 64-bit form of the 8-bit key / value cache and of attention over it, in numpy: one block, one
sequence and one head at a time. It shares nothing with the library but the layouts of include/fp4.h."""
import math

import numpy as np


def e4m3_table():
    """The value of each E4M3 code (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c & 0x80, -v, v)


E4M3 = e4m3_table()


def e4m3_encode(x):
    """Codes of float64 values, nearest with ties to even, saturating; the sign of zero is kept."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:0x7F]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def exponent(amax, ceil):
    if amax == 0:
        return -127
    m, ex = math.frexp(float(amax))  # amax = m 2^ex, m in [1/2, 1)
    e = ex - 1 - 8
    if ceil and 2 * m > 1.75:
        e += 1
    return min(127, max(-127, e))


class Cache:
    """Host copy of a cache's four arrays."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.k, self.v, self.ks, self.vs = (np.array(a) for a in (k_codes, v_codes, k_scales, v_scales))
        self.pages, self.heads, self.page, self.dim = self.k.shape


def _place(cache, table, s, pos):
    j = pos // cache.page
    if pos < 0 or j >= table.shape[1] or not 0 <= table[s, j] < cache.pages:
        return None
    return int(table[s, j]), pos % cache.page


def append(cache, k, v, cu, context, table, ceil):
    """In place. k, v float64 [tokens, heads, dim]."""
    for s in range(len(context)):
        n, ctx = cu[s + 1] - cu[s], int(context[s])
        blocks = {}
        for i in range(n):
            at = _place(cache, table, s, ctx - n + i)
            if at is not None:
                blocks.setdefault(at[0], []).append((at[1], cu[s] + i))
        for page, rows in blocks.items():
            t0 = min(t for t, _ in rows)
            for x, codes, scales, tr in ((k, cache.k, cache.ks, False), (v, cache.v, cache.vs, True)):
                for h in range(cache.heads):
                    blk = codes[page, h].T if tr else codes[page, h]  # [token, dim], a view
                    e = exponent(max(np.abs(x[r, h]).max() for _, r in rows), ceil)
                    if t0 > 0:
                        old = int(scales[page, h]) - 127
                        if e > old:
                            blk[:t0] = e4m3_encode(E4M3[blk[:t0]] * 2.0 ** (old - e))
                        e = max(e, old)
                    for t, r in rows:
                        blk[t] = e4m3_encode(x[r, h] * 2.0 ** -e)
                    scales[page, h] = e + 127


def read(cache, cu, context, table):
    """k, v float64 [tokens, heads, dim] (NaN: a row with no token)."""
    k = np.full((cu[-1], cache.heads, cache.dim), np.nan)
    v = k.copy()
    for s in range(len(context)):
        n, ctx = cu[s + 1] - cu[s], int(context[s])
        for i in range(n):
            at = _place(cache, table, s, ctx - n + i)
            if at is not None:
                p, t = at
                k[cu[s] + i] = E4M3[cache.k[p, :, t]] * 2.0 ** (cache.ks[p].astype(np.float64) - 127)[:, None]
                v[cu[s] + i] = E4M3[cache.v[p, :, :, t]] * 2.0 ** (cache.vs[p].astype(np.float64) - 127)[:, None]
    return k, v


def attention(q, cache, cu, context, table, scale, causal, window):
    """out, lse and, for error bounds, per row: sum_j w_j |v_j| / sum_j w_j, max_j scale sum_d |q k_j|,
    the number of keys. q float64 [tokens, q_heads, dim]."""
    T, Hq, D = q.shape
    G = Hq // cache.heads
    out, absv = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, mag, cnt = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    for s in range(len(context)):
        n, ctx = int(cu[s + 1] - cu[s]), max(int(context[s]), 0)
        if n <= 0:
            continue
        limit = min(ctx, table.shape[1] * cache.page)
        keys = np.arange(limit)
        idx = table[s, keys // cache.page]
        there = (idx >= 0) & (idx < cache.pages)
        pg, tk = np.where(there, idx, 0), keys % cache.page
        pos = ctx - n + np.arange(n)
        allowed = np.broadcast_to(there, (n, limit)).copy()
        if causal:
            allowed &= keys <= pos[:, None]
        if window:
            allowed &= keys > pos[:, None] - window
        some = allowed.any(0)  # the rest is not looked at
        keys, pg, tk, allowed = keys[some], pg[some], tk[some], allowed[:, some]
        if not len(keys):
            continue
        for h in range(cache.heads):
            k = E4M3[cache.k[pg, h, tk]] * 2.0 ** (cache.ks[pg, h].astype(np.float64) - 127)[:, None]
            v = E4M3[cache.v[pg, h, :, tk]] * 2.0 ** (cache.vs[pg, h].astype(np.float64) - 127)[:, None]
            for hq in range(h * G, (h + 1) * G):
                x = q[cu[s]:cu[s] + n, hq]
                sc = np.where(allowed, (x @ k.T) * scale, -np.inf)
                top = sc.max(1)
                ok = np.isfinite(top)
                w = np.exp(sc - np.where(ok, top, 0.0)[:, None])
                l = w.sum(1)
                r = slice(cu[s], cu[s] + n)
                safe = np.where(ok, l, 1.0)[:, None]
                out[r, hq] = (w @ v) / safe
                absv[r, hq] = (w @ np.abs(v)) / safe
                lse[r, hq] = np.where(ok, np.log(np.where(ok, l, 1.0)) + top, -np.inf)
                mag[r, hq] = np.where(allowed, (np.abs(x) @ np.abs(k).T) * abs(scale), 0).max(1)
                cnt[r, hq] = allowed.sum(1)
    return out, lse, absv, mag, cnt
