"""Plain 64-bit restatement of the operators of paged decoding, for their tests (numpy, no code shared with
the library)."""
import math

import numpy as np


def gather(pool, table, n, page_size):
    """Rows 0..n-1 of a sequence: ([H_kv][n][hd], there [n]) of a pool [pages][H_kv][page_size][hd]; rows that lie on
    no page are zeros and not there."""
    t = np.arange(n)
    page = table[t // page_size]
    there = (page >= 0) & (page < pool.shape[0])
    rows = pool[np.where(there, page, 0), :, t % page_size].transpose(1, 0, 2).copy()
    rows[:, ~there] = 0
    return rows, there


def attention(q, k, v, there, scale):
    """q [R][H][hd], k and v [H_kv][n][hd] -> out [R][H][hd], mass [H_kv][n], and for tolerances the sum of p|v|, the
    sum of |v| and the largest sum of scale |q||k| of every row and head."""
    R, H, hd = q.shape
    g, n = H // k.shape[0], k.shape[1]
    out, pv, sv = (np.zeros((R, H, hd)) for _ in range(3))
    sk = np.zeros((R, H, 1))
    mass = np.zeros((k.shape[0], n))
    if not there.any():
        return out, mass, pv, sv, sk
    for i in range(R):
        for h in range(H):
            kk, vv = k[h // g][there], v[h // g][there]
            z = scale * (kk @ q[i, h])
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h], pv[i, h], sv[i, h] = p @ vv, p @ np.abs(vv), np.abs(vv).sum(0)
            sk[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            mass[h // g][there] += p
    return out, mass, pv, sv, sk


def norm_rope(x, w, eps, pos, rot, layout, rates, amp=1.0):
    """x [rows][heads][hd]; w None: ones; eps < 0: no norm; rates None: nothing turns."""
    y = x.astype(np.float64)
    if eps >= 0:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if w is not None:
            y = y * w
    if rates is None:
        return y
    out = y.copy()
    i0 = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
    i1 = i0 + (rot // 2 if layout == "half" else 1)
    a = pos.astype(np.float64)[:, None] * rates
    c, s = (amp * np.cos(a))[:, None], (amp * np.sin(a))[:, None]
    out[..., i0] = y[..., i0] * c - y[..., i1] * s
    out[..., i1] = y[..., i1] * c + y[..., i0] * s
    return out


def kept(mass, n, keep, sinks, recent):
    """Positions of mass[0..n) that stay, ascending."""
    if n <= keep:
        return np.arange(n)
    lo, hi = sinks, n - recent
    w = [(-math.inf, 1) if math.isnan(x) else (float(x), 0) for x in mass[lo:hi]]
    order = sorted(range(lo, hi), key=lambda t: (w[t - lo][1], -w[t - lo][0], t))
    return np.array(sorted(list(range(lo)) + order[:keep - sinks - recent] + list(range(hi, n))), dtype=np.int64)


def logprobs(z, scale, target, top):
    """One row: (log p of target, entropy, ids, their log p, and for tolerances sum e^d, sum |d| e^d, sum d^2 e^d over
    all but the largest)."""
    z = z.astype(np.float64)
    nan = math.nan
    order = [int(i) for i in np.argsort(-z, kind="stable")[:top] if not math.isnan(z[i])]   # (NaN sorts last)
    ids = (order + [-1] * top)[:top]
    m = np.nanmax(z) if not np.isnan(z).all() else nan
    if np.isnan(z).any() or not math.isfinite(m):
        return nan, nan, ids, [nan] * top, 0.0, 0.0, 0.0
    a = int(np.argmax(z))
    d = scale * (z - m)
    e = np.exp(d)
    e[a] = 0.0
    d0 = np.where(e > 0, d, 0.0)
    S, W, D = math.fsum(e), math.fsum(d0 * e), math.fsum(d0 * d0 * e)
    lse = math.log1p(S)
    lp = [d[i] - lse if i >= 0 else nan for i in ids]
    return (d[target] - lse if 0 <= target < len(z) else nan), lse - W / (1 + S), ids, lp, S, -W, D
