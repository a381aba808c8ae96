"""Plain fp64 reference of the paged 4-bit KV cache: formats, plan, attention.

Written from the definitions in include/fa2.h, one token at a time where that
is the plain way; shares no code with the CUDA library. Tensors are torch CPU
tensors; caches are uint8 [num_pages, H_kv, 2, page*(d/2 + d/16)].
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if (c & 0x7F) == 0x7F:
            v = math.nan
        t[c] = -v if c & 0x80 else v
    return t


E4M3 = _e4m3_table()


def split(cache, d):
    """(codes [P, H, 2, page, d], scale bytes [P, H, 2, page, d/16]) of a cache."""
    c = np.asarray(cache)
    page = c.shape[3] // (d // 2 + d // 16)
    packed = c[..., : page * d // 2].reshape(*c.shape[:3], page, d // 2)
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(*c.shape[:3], page, d)
    return codes, c[..., page * d // 2:].reshape(*c.shape[:3], page, d // 16)


def scale32(scale_bytes, descale):
    """scale * descale in fp32: [..., d/16] bytes, descale broadcast against them."""
    return (E4M3[scale_bytes].astype(np.float32) * np.asarray(descale, np.float32)).astype(np.float32)


def nearest(table, y):
    """Index of the entry of an ascending table nearest to y >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(table, y), 1, len(table) - 1)
    a, b = y - table[hi - 1], table[hi] - y
    return np.where((a < b) | ((a == b) & (hi % 2 == 1)), hi - 1, hi)


def rounded(x, descale):
    """fp64 [..., d] finite values as append keeps them (t = scale * descale in fp32)."""
    blk = x.reshape(*x.shape[:-1], -1, 16)
    s = E4M3[:127][nearest(E4M3[:127], np.abs(blk).max(-1) / (6 * float(descale)))]
    t = (s.astype(np.float32) * np.float32(descale)).astype(np.float64)[..., None]
    y = np.divide(np.abs(blk), t, out=np.zeros_like(blk), where=t > 0)
    return (np.sign(blk) * E2M1[:8][nearest(E2M1[:8], y)] * t).reshape(x.shape)


def tokens(cache, d, table_row, n, h, part, descale):
    """fp64 [n, d]: the first n cached keys (part 0) or values (1) of head h."""
    codes, scales = split(cache, d)
    page = codes.shape[3]
    out = np.zeros((n, d))
    for i in range(n):
        pg = int(table_row[i // page])
        x, s = codes[pg, h, part, i % page], scales[pg, h, part, i % page]
        out[i] = E2M1[x] * np.repeat(E4M3[s], 16) * float(descale)
    return out


def attention(q, keys, values, scale, causal, lens):
    """q fp64 [B, Hq, Nq, d]; keys/values: lists over b of fp64 [Hkv, n_b, d].
    Returns o, lse and, per row, sum_j p_j |v_j| and the largest
    sum_d |q_d k_d| * scale (what error bounds are made of)."""
    B, Hq, Nq, d = q.shape
    o = np.zeros((B, Hq, Nq, d))
    lse = np.full((B, Hq, Nq), -np.inf)
    av = np.zeros((B, Hq, Nq, d))
    big = np.zeros((B, Hq, Nq))
    for b in range(B):
        n = lens[b]
        if n <= 0:
            continue
        G = Hq // keys[b].shape[0]
        for hq in range(Hq):
            k, v = keys[b][hq // G], values[b][hq // G]
            for i in range(Nq):
                m = min(n, i + 1 + n - Nq) if causal else n
                if m <= 0:
                    continue
                s = scale * (k[:m] @ q[b, hq, i])
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                o[b, hq, i] = p @ v[:m] / z
                lse[b, hq, i] = top + math.log(z)
                av[b, hq, i] = p @ np.abs(v[:m]) / z
                big[b, hq, i] = scale * (np.abs(k[:m]) @ np.abs(q[b, hq, i])).max()
    return o, lse, av, big


def plan(seq_lens, new_lens, table, ring, state, page, N):
    """One scheduling step, one request and page at a time. Changes copies of
    table and ring; returns (seq_lens, accepted, slots, state, table, ring)."""
    seq_lens, table, ring = list(map(int, seq_lens)), np.array(table), np.array(ring)
    B, W = table.shape
    P = len(ring)
    first, count = int(state[0]), int(state[1])
    accepted, slots = [0] * B, np.full((B, N), -1, np.int64)
    wanted, taken, back = 0, 0, 0
    for b in range(B):
        n, add = seq_lens[b], int(new_lens[b])
        have = -(-n // page)
        if add < 0:
            for j in range(have):
                if 0 <= table[b, j] < P:   # an id outside the cache does not join the ring
                    ring[(first + count + back) % P] = table[b, j]
                    back += 1
            seq_lens[b] = 0
            continue
        if add > N or n + add > W * page:
            continue
        need = -(-(n + add) // page) - have
        wanted += need
        if need and wanted > count:
            continue
        for j in range(need):
            table[b, have + j] = ring[(first + taken) % P]
            taken += 1
        for i in range(add):
            slots[b, i] = int(table[b, (n + i) // page]) * page + (n + i) % page
        seq_lens[b], accepted[b] = n + add, add
    return seq_lens, accepted, slots, [(first + taken) % P, count - taken + back], table, ring
