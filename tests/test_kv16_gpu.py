"""Attention over the paged 16-bit KV cache on the GPU against the fp64 oracle
(oracle/kv16.py).

Bounds, with A = sum_j p_j |v_j| (softmax p), u half a step of the type (bf16
2^-8, fp16 2^-11) and n keys:
    |O - ref| <= (u + 2 e + r) A + w n max|v| + u |ref| + s,
    |LSE - ref| <= e + r + 2^-22 |ref|
The first u is the rounding of the softmax's weights, the second that of O. e
bounds the error of a score: products of d fp32 terms at 2^-23 each relative to
sum_d |q_d k_d| scale, and the roundings of the exponent's terms; r the fp32
sums over the keys and partial results, (n / 8 + 64) 2^-23. fp16 weights below
2^-14 are multiples of 2^-24: w = 2^-25 (0 for bf16); so are fp16 outputs: s.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv16

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}
KEEP = 123.0   # what rows that belong to no request hold before the call


def ok(fa2):
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_OK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Step:
    """Requests (new, cached) with their cache, tables and queries. Whatever
    no request owns is NaN: places behind a last token, pages of nobody, rows of
    q between and behind the requests' rows."""

    def __init__(self, seed, reqs, Hq, Hkv, d, page, dtype, amp=1.0, gap=0, behind=3, strided=False):
        rng = np.random.default_rng(seed)
        self.reqs, self.Hq, self.Hkv, self.d, self.page, self.dtype = reqs, Hq, Hkv, d, page, dtype
        need = [-(-L // page) for _, L in reqs]
        W, P = max(need) + 2, sum(need) + 2
        ids = rng.permutation(P)
        self.table = np.full((len(reqs), W), -1, np.int64)
        cache = torch.full((P, Hkv, 2, page, d), math.nan, dtype=DT[dtype])
        at = 0
        for b, (_, L) in enumerate(reqs):
            self.table[b, : need[b]] = ids[at: at + need[b]]
            at += need[b]
            for j in range(need[b]):
                m = min(page, L - j * page)
                cache[int(self.table[b, j]), :, :, :m] = torch.tensor(rng.standard_normal((Hkv, 2, m, d))).to(DT[dtype])
        self.cache = cache
        starts, t = [], 0
        for n, _ in reqs:
            starts.append(t)
            t += n + gap
        self.T = max(t + behind, 1)
        self.starts = starts
        wide = Hq + 2 if strided else Hq
        q = torch.full((self.T, wide, d), math.nan, dtype=DT[dtype])
        for (n, _), s in zip(reqs, starts):
            q[s: s + n, :Hq] = torch.tensor(rng.standard_normal((n, Hq, d)) * amp).to(DT[dtype])
        self.q = q[:, :Hq]
        self.scale = d ** -0.5

    def args(self):
        dev = self.q.cuda() if self.q.is_contiguous() else torch.as_strided(self.q, (self.T, self.Hq + 2, self.d), self.q.stride()).cuda()[:, : self.Hq]
        return [dev, self.cache.cuda(), i32(self.table), i32([L for _, L in self.reqs]), i32(self.starts),
                i32([n for n, _ in self.reqs])]

    def run(self, fa2, causal=True):
        o = torch.full((self.T, self.Hq, self.d), KEEP, dtype=DT[self.dtype], device="cuda")
        lse = torch.full((self.T, self.Hq), KEEP, device="cuda")
        out = fa2.fa2_fwd_kv16(*self.args(), o=o, lse=lse, scale=self.scale, causal=causal)
        assert out[0] is o and out[1] is lse
        ok(fa2)
        return o, lse

    def check(self, o, lse, causal=True):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        cache, q = self.cache.double().numpy(), self.q.double().numpy()
        free = np.ones(self.T, bool)
        for b, (n, L) in enumerate(self.reqs):
            rows = slice(self.starts[b], self.starts[b] + n)
            free[rows] = False
            if n == 0:
                continue
            k, v = (kv16.tokens(cache, self.table[b], L, part) for part in (0, 1))
            ref, lref, A, big = kv16.attention(q[rows], k, v, self.scale, causal)
            compare(o[rows], lse[rows], ref, lref, A, big, L, v, self.d, self.dtype)
        assert np.all(o[free] == KEEP) and np.all(lse[free] == KEEP)


def compare(o, lse, ref, lref, A, big, L, v, d, dtype):
    empty = np.isneginf(lref)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(o[empty] == 0)
    full = ~empty
    if not full.any():
        return
    u = U[dtype]
    lr = np.where(full, lref, 0)
    e = (d + 8) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * np.abs(lr) + 2.0 ** -21
    r = (L / 8 + 64) * 2.0 ** -23
    bound = (u + 2 * e + r)[..., None] * A + SUB[dtype] * (L * np.abs(v).max() + 1) + u * np.abs(ref)
    err = np.abs(o - ref)
    assert np.all(err[full] <= bound[full]), f"O off by {np.nanmax(err[full] / np.maximum(bound[full], 1e-300)):.3g} bounds"
    assert np.all(np.abs(lse - lr)[full] <= (e + r + 2.0 ** -22 * np.abs(lr))[full]), "LSE"


CASES = [
    # (new, cached) of each request, Hq, Hkv, d, page, causal, dtype
    ([(1, 1)], 1, 1, 128, 16, True, "bf16"),
    ([(1, 1)], 4, 1, 64, 128, False, "fp16"),
    ([(1, 0)], 8, 2, 128, 64, True, "bf16"),
    ([(0, 0), (0, 5), (1, 0), (1, 5)], 8, 2, 64, 64, False, "bf16"),
    ([(1, n) for n in (15, 16, 17, 127, 128, 129, 255, 256, 257)], 8, 2, 128, 16, True, "bf16"),
    ([(1, n) for n in (63, 64, 65, 128, 384, 385, 1, 640)], 8, 2, 64, 32, True, "fp16"),
    ([(1, 1000), (1, 3), (1, 517)], 16, 16, 128, 64, True, "bf16"),
    ([(1, 700), (0, 0), (1, 130)], 14, 2, 128, 64, True, "fp16"),          # 7 heads a KV head
    ([(5, 300), (3, 40), (1, 1), (2, 130)], 9, 3, 128, 128, True, "bf16"),
    ([(31, 31), (32, 32), (33, 33), (34, 200)], 4, 1, 128, 32, True, "bf16"),      # 32 tokens a tile
    ([(63, 70), (64, 300), (65, 65), (66, 129)], 8, 2, 64, 16, True, "fp16"),      # 64 tokens a block
    ([(127, 127), (128, 128), (129, 129), (257, 400)], 2, 2, 128, 64, True, "bf16"),
    ([(300, 300), (1, 777), (200, 513)], 6, 2, 64, 16, True, "bf16"),      # 42 tokens a tile: rows of a tile unused
    ([(100, 200), (300, 77)], 5, 1, 128, 64, False, "bf16"),
    ([(90, 20), (40, 0), (1, 9)], 2, 2, 64, 128, True, "fp16"),            # more new tokens than cached
    ([(700, 130)], 2, 1, 128, 16, True, "bf16"),                           # whole blocks of rows without a key
    ([(5, 9)], 128, 1, 128, 16, True, "bf16"),                             # a token a tile
    ([(3, 300)], 100, 1, 64, 32, True, "fp16"),
    ([(1, 7)] * 90, 2, 1, 64, 16, True, "bf16"),
    ([(2, 5), (0, 0), (1, 70)] * 70, 4, 4, 64, 16, True, "fp16"),          # more requests than threads of a warp
    ([(600, 1800)], 8, 2, 128, 128, True, "bf16"),
]


@pytest.mark.parametrize("reqs,Hq,Hkv,d,page,causal,dtype", CASES)
def test_every_element(gpu_lib, reqs, Hq, Hkv, d, page, causal, dtype):
    s = Step(3 + len(reqs) + Hq + d, reqs, Hq, Hkv, d, page, dtype)
    s.check(*s.run(gpu_lib, causal), causal)


def poison(s, b, pos, part, head, col, value):
    s.cache[int(s.table[b, pos // s.page]), head, part, pos % s.page, col] = value


@pytest.mark.parametrize("d,page,dtype,G,new,L", [
    (128, 64, "bf16", 4, 70, 300), (128, 16, "fp16", 1, 300, 300), (64, 32, "bf16", 2, 200, 513), (128, 128, "bf16", 8, 5, 129),
    (64, 16, "fp16", 4, 33, 40),
])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_what_is_not_finite_reaches_only_rows_that_see_it(gpu_lib, d, page, dtype, G, new, L, value):
    """Keys and values of some new tokens are not finite: rows that do not see
    them by the mask keep every bit. Of the values, only the column is lost."""
    fa2 = gpu_lib
    reqs = [(1, 200), (new, L), (2, 9)]
    for part in (0, 1):
        s = Step(17 + d + new, reqs, 2 * G, 2, d, page, dtype)
        o, lse = s.run(fa2)
        at = [L - 1, L - new // 2, L - new + 1]   # the last new token's position, ...
        for pos, col in zip(at, (5, d - 1, 5)):
            poison(s, 1, pos, part, 1, col, value)
        o2, lse2 = s.run(fa2)
        rows = np.arange(s.starts[1], s.starts[1] + new)
        seen = L - new + np.arange(new)           # the last position that a row sees
        same = torch.ones(s.T, 2 * G, d, dtype=torch.bool)
        if part:
            for pos, col in zip(at, (5, d - 1, 5)):
                same[rows[seen >= pos], G:, col] = False
            assert torch.equal(lse2, lse)
            assert not torch.isfinite(o2.cpu()[~same]).any()
        else:
            hit = seen >= min(at)
            same[rows[hit], G:] = False
            keep = torch.ones(s.T, 2 * G, dtype=torch.bool)
            keep[rows[hit], G:] = False
            assert torch.equal(lse2.cpu()[keep], lse.cpu()[keep])
            # an infinite product with the row is no NaN where it is -inf: that key has no weight
            if math.isnan(value):
                assert lse2.cpu()[~keep].isnan().all() and o2.cpu()[~same].isnan().all()
        assert torch.equal(o2.cpu()[same], o.cpu()[same])


def test_rows_of_q_that_are_not_finite_stay_alone(gpu_lib):
    fa2 = gpu_lib
    s = Step(23, [(1, 300), (40, 200), (150, 150)], 8, 2, 128, 64, "bf16")
    o, lse = s.run(fa2)
    bad = [(0, 3), (20, 0), (100, 7), (s.starts[2] + 149, 4)]
    for t, h in bad:
        s.q[t, h, 17] = math.nan
    o2, lse2 = s.run(fa2)
    keep = torch.ones(s.T, 8, dtype=torch.bool)
    for t, h in bad:
        keep[t, h] = False
    assert o2.cpu()[~keep].isnan().all() and lse2.cpu()[~keep].isnan().all()
    assert torch.equal(o2.cpu()[keep], o.cpu()[keep]) and torch.equal(lse2.cpu()[keep], lse.cpu()[keep])
