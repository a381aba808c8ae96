"""Plain fp64 forms of the rotary positions and of attention over the paged
16-bit cache (test infrastructure; numpy, no code shared with the kernels)."""
import math

import numpy as np

TWO_PI = 8 * np.arctan(np.longdouble(1))


def rotate(x, positions, inv_freq, axes=None, interleaved=False, inverse=False):
    """x [..., d] with positions [n_axes, ...] of the same leading sizes; the
    first 2 * len(inv_freq) elements are rotated, pair i by
    positions[axes[i]] * inv_freq[i] (reduced to a turn in extended precision)."""
    x = np.asarray(x, np.float64)
    f = np.asarray(inv_freq, np.float32).astype(np.longdouble)
    P = len(f)
    which = np.zeros(P, int) if axes is None else np.asarray(axes)
    angle = np.moveaxis(np.asarray(positions, np.int64)[which], 0, -1).astype(np.longdouble) * f
    angle = (angle - np.floor(angle / TWO_PI) * TWO_PI).astype(np.float64)
    c, s = np.cos(angle), np.sin(angle) * (-1 if inverse else 1)
    i = np.arange(P)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def tokens(cache, table_row, n, part):
    """fp64 [H_kv, n, d]: the first n cached keys (part 0) or values (1)."""
    P, H, _, page, d = cache.shape
    out = np.zeros((H, n, d))
    for j in range(-(-n // page)):
        m = min(page, n - j * page)
        out[:, j * page: j * page + m] = cache[int(table_row[j]), :, part, :m]
    return out


def attention(q, keys, values, scale, causal):
    """One request: q fp64 [n, Hq, d], keys and values fp64 [Hkv, L, d].
    Returns o [n, Hq, d], lse [n, Hq], and per row sum_j p_j |v_j| and the
    largest sum_d |q_d k_d| * scale (what error bounds are made of)."""
    n, Hq, d = q.shape
    H, L, _ = keys.shape
    G = Hq // H
    o, av = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, big = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    seen = np.minimum(L, L - n + 1 + np.arange(n)) if causal else np.full(n, L)
    for h in range(Hq):
        if L == 0:
            break
        k, v = keys[h // G], values[h // G]
        s = scale * (q[:, h] @ k.T)
        mag = scale * (np.abs(q[:, h]) @ np.abs(k).T)
        off = np.arange(L)[None] >= seen[:, None]
        s = np.where(off, -np.inf, s)
        rows = seen > 0
        top = s[rows].max(1, keepdims=True)
        p = np.exp(s[rows] - top)
        z = p.sum(1, keepdims=True)
        vv = np.where(np.isfinite(v), v, 0.0)
        o[rows, h] = p @ vv / z
        av[rows, h] = p @ np.abs(vv) / z
        lse[rows, h] = (top + np.log(z))[:, 0]
        big[rows, h] = np.where(off, 0.0, mag)[rows].max(1)
    return o, lse, av, big
