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


@pytest.mark.parametrize("d,page,dtype", [(128, 16, "fp16"), (128, 64, "bf16"), (64, 128, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_views_gaps_and_rows_of_nobody(gpu_lib, d, page, dtype, causal):
    """q as a view of a wider tensor; rows between and behind the requests'."""
    s = Step(31 + d, [(3, 400), (130, 333), (0, 70), (1, 129), (64, 64)], 12, 4, d, page, dtype, gap=5, behind=40, strided=True)
    assert not s.q.is_contiguous()
    s.check(*s.run(gpu_lib, causal), causal)


@pytest.mark.parametrize("d,page,dtype,reqs,Hq,Hkv", [
    (128, 64, "bf16", [(1, 20011)], 4, 1), (64, 16, "fp16", [(1, 30001), (1, 5)], 8, 2), (128, 16, "bf16", [(7, 9001), (1, 12000)], 16, 2),
    (128, 128, "fp16", [(150, 7000)], 8, 2), (64, 32, "bf16", [(1000, 5000), (1, 3000), (40, 2000)], 4, 2),
])
def test_long_contexts_are_split_and_joined(gpu_lib, d, page, dtype, reqs, Hq, Hkv):
    s = Step(41 + d + page, reqs, Hq, Hkv, d, page, dtype)
    s.check(*s.run(gpu_lib))


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_page_size_makes_no_difference(gpu_lib, d, dtype):
    """The same tokens in pages of every size, tables of the same number of
    tokens: every bit is the same."""
    fa2 = gpu_lib
    s = Step(57 + d, [(1, 700), (150, 600), (33, 257), (1, 16)], 8, 2, d, 128, dtype)
    first = None
    for page in (128, 64, 32, 16):
        each = 128 // page
        args = s.args()
        P, Hkv = s.cache.shape[:2]
        args[1] = args[1].view(P, Hkv, 2, each, page, d).permute(0, 3, 1, 2, 4, 5).reshape(P * each, Hkv, 2, page, d).contiguous()
        args[2] = i32(np.where(s.table[:, :, None] < 0, -1, s.table[:, :, None] * each + np.arange(each)).reshape(len(s.reqs), -1))
        used = s.T - 3   # rows that belong to a request
        o, lse = fa2.fa2_fwd_kv16(*args, scale=s.scale, causal=True)
        ok(fa2)
        got = o[:used].cpu(), lse[:used].cpu()
        if first is None:
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_sharp_scores(gpu_lib):
    s = Step(5, [(1, 900), (70, 411)], 8, 2, 128, 64, "bf16", amp=8.0)
    s.check(*s.run(gpu_lib))


@pytest.mark.parametrize("step", [0.5, 6.0, 40.0])
def test_running_maximum_grows(gpu_lib, step):
    """Scores that grow from tile to tile: O is rescaled at every one."""
    s = Step(6, [(1, 1500), (80, 1200)], 4, 1, 128, 32, "bf16")
    for b, (_, L) in enumerate(s.reqs):
        for j in range(L):
            s.cache[int(s.table[b, j // s.page]), :, 0, j % s.page] = step * (1 + j // 128) / 8
    s.q[...] = torch.where(torch.isnan(s.q), s.q, torch.ones((), dtype=s.q.dtype))
    s.scale = 1.0 / 16
    s.check(*s.run(gpu_lib))


def test_output_aligned_to_16_bytes_only(gpu_lib):
    fa2 = gpu_lib
    s = Step(8, [(1, 300), (40, 200)], 4, 2, 64, 16, "bf16")
    room = torch.full((s.T * 4 * 64 + 8,), KEEP, dtype=torch.bfloat16, device="cuda")
    o = room[8:].view(s.T, 4, 64)
    assert o.data_ptr() % 32 == 16
    lse = torch.full((s.T, 4), KEEP, device="cuda")
    fa2.fa2_fwd_kv16(*s.args(), o=o, lse=lse, scale=s.scale, causal=True)
    ok(fa2)
    s.check(o, lse)
    assert (room[:8] == KEEP).all()


def test_workspace_holds_anything_and_is_enough(gpu_lib):
    """Exactly the bytes asked for, full of NaN, at an odd multiple of 16 bytes,
    beside bytes that stay as they were."""
    fa2 = gpu_lib
    s = Step(9, [(1, 3000), (200, 900), (1, 10)], 8, 2, 128, 64, "bf16")
    n = fa2.fa2_fwd_kv16_workspace(s.T, 3, 8, 2, 128, s.table.shape[1], 64)
    for off in (16, 32):
        room = torch.full((n + 96,), 0xFF, dtype=torch.uint8, device="cuda")
        o = torch.full((s.T, 8, 128), KEEP, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((s.T, 8), KEEP, device="cuda")
        fa2.fa2_fwd_kv16(*s.args(), o=o, lse=lse, workspace=room[off: off + n], scale=s.scale, causal=True)
        ok(fa2)
        s.check(o, lse)
        assert (room[:off] == 0xFF).all() and (room[off + n:] == 0xFF).all()
        with pytest.raises(fa2.FA2Error):
            fa2.fa2_fwd_kv16(*s.args(), o=o, lse=lse, workspace=room[off: off + n - 1], scale=s.scale, causal=True)


def test_results_repeat_bit_for_bit(gpu_lib):
    fa2 = gpu_lib
    s = Step(61, [(1, 9000), (0, 0), (333, 700), (1, 4097), (64, 2000)], 16, 2, 64, 32, "bf16")
    a = [s.run(fa2) for _ in range(5)]
    assert all(torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1]) for x in a)


def test_two_calls_on_two_streams(gpu_lib):
    fa2 = gpu_lib
    s = [Step(70 + i, [(1, 5000), (100, 1200)], 8, 2, 128, 64, "bf16", behind=0) for i in range(2)]
    args = [x.args() for x in s]
    want = [fa2.fa2_fwd_kv16(*a, causal=True) for a in args]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [fa2.fa2_fwd_kv16(*args[i % 2], causal=True, stream=st[i % 2]) for i in range(20)]
    for x in st:
        assert fa2.fa2_check_status(x.cuda_stream) == fa2.FA2_OK
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_what_points_outside_is_reported(gpu_lib):
    """Ids of pages, lengths and rows outside the cache, the table and q
    (checked on the device)."""
    fa2 = gpu_lib
    stream = torch.cuda.current_stream().cuda_stream
    s = Step(12, [(1, 64), (2, 40)], 4, 1, 64, 16, "bf16")
    s.cache = torch.where(torch.isnan(s.cache), torch.zeros((), dtype=s.cache.dtype), s.cache)
    o, lse = s.run(fa2)
    good = s.args()

    def call(**kw):
        a = list(good)
        for i, x in kw.values():
            a[i] = x
        o2, l2 = torch.full_like(o, KEEP), torch.full_like(lse, KEEP)
        fa2.fa2_fwd_kv16(*a, o=o2, lse=l2, scale=s.scale, causal=True)
        assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
        return o2, l2

    # a page that is none reads as zeros
    bad = s.table.copy()
    bad[0, 1], bad[0, 2] = s.cache.shape[0], -5
    o2, l2 = call(x=(2, i32(bad)))
    assert torch.equal(o2[1:], o[1:]) and torch.equal(l2[1:], lse[1:])
    keep = s.cache.clone()
    s.cache[torch.tensor(s.table[0, 1:3])] = 0
    want = s.run(fa2)
    assert torch.equal(o2, want[0]) and torch.equal(l2, want[1])
    s.cache = keep
    # a length behind the table's end is cut to it, one below 0 is none
    o2, l2 = call(x=(2, i32(s.table[:, :4])), y=(3, i32([65, 40])))
    assert torch.equal(o2, o) and torch.equal(l2, lse)
    o2, l2 = call(x=(3, i32([-1, 40])))
    assert torch.equal(o2[1:], o[1:]) and not o2[0].any() and torch.isneginf(l2[0]).all()
    # rows outside q: the request is left out
    for start, n in ((s.T, 1), (-1, 1), (s.T - 1, 2), (0, -3), (2 ** 31 - 1, 5), (-2 ** 31, 2)):
        o2, l2 = call(x=(4, i32([start, 1])), y=(5, i32([n, 2])))
        assert torch.equal(o2[1:], o[1:]) and torch.equal(l2[1:], lse[1:]) and (o2[0] == KEEP).all()
    # more rows than there are
    a = list(good)
    a[4], a[5] = i32([0, 0]), i32([s.T, s.T])
    fa2.fa2_fwd_kv16(*a, causal=True)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    s.check(*s.run(fa2))


def test_a_wait_that_runs_out(gpu_lib):
    """Query tiles that are not loaded: the kernel gives up and says so, and the
    next call is right."""
    fa2 = gpu_lib
    s = Step(13, [(1, 500), (70, 300)], 8, 2, 128, 64, "bf16")
    args = s.args()
    old, limit = fa2.fa2_set_debug_flags(1), fa2.fa2_set_wait_limit_ns(50_000_000)
    try:
        fa2.fa2_fwd_kv16(*args, causal=True)
        assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_ERR_TIMEOUT
    finally:
        fa2.fa2_set_debug_flags(old)
        fa2.fa2_set_wait_limit_ns(limit)
    s.check(*s.run(fa2))


def test_cache_behind_four_gigabytes(gpu_lib):
    """Pages whose byte offsets pass 32 bits."""
    fa2 = gpu_lib
    rng = np.random.default_rng(51)
    Hkv, d, page = 8, 128, 16
    P = (1 << 32) // (Hkv * 2 * page * d * 2) + 300
    cache = torch.empty(fa2.fa2_kv16_cache_shape(P, Hkv, page, d), dtype=torch.float16, device="cuda")
    n = 40
    table = np.array([[P - 1, P - 7, 2, -1]])
    slots = [int(table[0, i // page]) * page + i % page for i in range(n)]
    k, v = (torch.tensor(rng.standard_normal((n, Hkv, d))).half() for _ in range(2))
    fa2.fa2_kv16_append(k.cuda(), v.cuda(), i32(slots), cache)
    q = torch.tensor(rng.standard_normal((n, Hkv, d))).half()
    o, lse = fa2.fa2_fwd_kv16(q.cuda(), cache, i32(table), i32([n]), i32([0]), i32([n]), causal=True)
    ok(fa2)
    kk, vv = k.double().numpy().transpose(1, 0, 2), v.double().numpy().transpose(1, 0, 2)
    ref = kv16.attention(q.double().numpy(), kk, vv, d ** -0.5, True)
    compare(o.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, n, vv, d, "fp16")


def test_refusals(gpu_lib):
    fa2 = gpu_lib
    dev = "cuda"
    cache = torch.zeros(fa2.fa2_kv16_cache_shape(4, 2, 16, 64), dtype=torch.bfloat16, device=dev)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=dev)
    good = (q, cache, i32(np.zeros((1, 4))), i32([5]), i32([0]), i32([3]))
    fa2.fa2_fwd_kv16(*good)
    wide = torch.zeros(3, 4, 72, dtype=torch.bfloat16, device=dev)
    for i, bad in ((0, q.float()), (0, q.half()), (0, q[:, :3]), (0, q[..., :32]), (0, q[0]), (0, wide[..., 4:68]), (0, q.transpose(1, 2)),
                   (0, torch.zeros(3, 4, 68, dtype=torch.bfloat16, device=dev)[..., :64]), (0, q[:1].expand(3, 4, 64)),
                   (1, cache[:, :1]), (1, cache.half()), (1, cache[..., :32]), (1, cache[:, :, :1]), (1, cache.cpu()),
                   (2, good[2].long()), (2, good[2][:, ::2]), (3, i32([5, 5])), (3, good[3].cpu()), (4, i32([0, 1])), (5, good[5].long())):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
            fa2.fa2_fwd_kv16(*args)
    for kw in (dict(o=torch.empty(3, 4, 64, device=dev)), dict(o=torch.empty(4, 4, 64, dtype=torch.bfloat16, device=dev)),
               dict(lse=torch.empty(4, 3, device=dev)), dict(scale=0.0), dict(scale=math.nan),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device=dev)), dict(workspace=torch.empty(1 << 24, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
            fa2.fa2_fwd_kv16(*good, **kw)
    ok(fa2)


# ------------------------------------------------------------------ as a program uses them

def freqs(rot):
    return (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


@pytest.mark.parametrize("d,page,dtype", [(128, 16, "bf16"), (64, 32, "fp16")])
def test_plan_append_attend_together(gpu_lib, d, page, dtype):
    """A serving loop: pages and slots from the plan, new tokens rotated and
    written, attention over them. Each step against the oracle, which keeps the
    tokens themselves, rotates them in 64 bits and rounds them once."""
    fa2 = gpu_lib
    rng = np.random.default_rng(77)
    B, Hq, Hkv, W, P = 5, 4, 2, 12, 40
    dev = "cuda"
    cache = torch.full(fa2.fa2_kv16_cache_shape(P, Hkv, page, d), math.nan, dtype=DT[dtype], device=dev)
    lens, state = i32(np.zeros(B)), i32([0, P])
    table, ring = i32(np.full((B, W), -1)), i32(rng.permutation(P))
    f = freqs(d)
    axes = rng.integers(0, 3, d // 2).astype(np.int32)
    kept = [[] for _ in range(B)]   # rotated keys and values of each request
    for step in range(7):
        N = 70 if step % 3 == 0 else 3
        new = rng.integers(0, N + 1, B)
        if step:
            new[rng.random(B) < 0.2] = -1
        _, acc, slots, _ = fa2.fa2_kv4_plan(lens, i32(new), table, ring, state, page, N, seq_lens_out=lens, free_state_out=state)
        x = torch.tensor(rng.standard_normal((B * N, Hq + 2 * Hkv, d))).to(DT[dtype])
        pos = rng.integers(0, 100000, (3, B * N))
        y = x.to(dev)
        _, q = fa2.fa2_kv16_append(y[:, Hq: Hq + Hkv], y[:, Hq + Hkv:], slots.view(-1), cache, q=y[:, :Hq], positions=i32(pos),
                                   inv_freq=torch.tensor(f).to(dev), axes=i32(axes))
        o = torch.full((B * N, Hq, d), KEEP, dtype=DT[dtype], device=dev)
        lse = torch.full((B * N, Hq), KEEP, device=dev)
        fa2.fa2_fwd_kv16(q, cache, table, lens, i32(np.arange(B) * N), acc, o=o, lse=lse, causal=True)
        ok(fa2)
        spread = lambda h: np.broadcast_to(pos[:, :, None], (3, B * N, h))
        rk = torch.tensor(kv16.rotate(x[:, Hq: Hq + Hkv].double().numpy(), spread(Hkv), f, axes)).to(DT[dtype]).double().numpy()
        rv = x[:, Hq + Hkv:].double().numpy()
        qq = q.double().cpu().numpy()
        rq = kv16.rotate(x[:, :Hq].double().numpy(), spread(Hq), f, axes)
        assert np.abs(qq - rq).max() <= U[dtype] * np.abs(rq).max() + 2.0 ** -19 * np.abs(rq).max()
        for b, (a, n) in enumerate(zip(acc.tolist(), new.tolist())):
            rows = slice(b * N, b * N + a)
            kept[b] = [] if n < 0 else kept[b] + [(rk[i], rv[i]) for i in range(b * N, b * N + a)]
            assert len(kept[b]) == int(lens[b])
            assert (o[b * N + a: (b + 1) * N] == KEEP).all() and (lse[b * N + a: (b + 1) * N] == KEEP).all()
            if a == 0:
                continue
            k, v = (np.stack([t[i] for t in kept[b]]).transpose(1, 0, 2) for i in (0, 1))
            ref, lref, A, big = kv16.attention(qq[rows], k, v, d ** -0.5, True)
            # the kernel's rotated keys may be the neighbours of the oracle's: a step of each, 2 u, in every score
            L = len(kept[b])
            slack = 2 * U[dtype] * big
            err = np.abs(o[rows].double().cpu().numpy() - ref)
            e = (d + 8) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * np.abs(lref) + 2.0 ** -21 + slack
            r = (L / 8 + 64) * 2.0 ** -23
            assert np.all(err <= (U[dtype] + 2 * e + r)[..., None] * A + SUB[dtype] * (L * np.abs(v).max() + 1) + U[dtype] * np.abs(ref))
            assert np.all(np.abs(lse[rows].double().cpu().numpy() - lref) <= e + r + 2.0 ** -22 * np.abs(lref))


def test_captured_step_replays_with_new_lengths(gpu_lib):
    """plan, append and attention in one CUDA graph: every replay goes on from
    the lengths that the last one left, as calls one by one do."""
    fa2 = gpu_lib
    rng = np.random.default_rng(31)
    B, Hq, Hkv, d, page, W, P = 3, 8, 2, 128, 16, 8, 40
    dev = "cuda"
    toks = torch.tensor(rng.standard_normal((6, B, Hq + 2 * Hkv, d))).to(torch.bfloat16).to(dev)
    x, pos, f = torch.empty_like(toks[0]), i32([0, 0, 0]), torch.tensor(freqs(d)).to(dev)
    new, starts = i32([1, 1, 1]), i32([0, 1, 2])
    acc, slots = torch.empty_like(new), torch.empty((B, 1), dtype=torch.int32, device=dev)
    ws = torch.empty(fa2.fa2_fwd_kv16_workspace(B, B, Hq, Hkv, d, W, page), dtype=torch.uint8, device=dev)
    q, o, lse = torch.empty(B, Hq, d, dtype=torch.bfloat16, device=dev), torch.empty(B, Hq, d, dtype=torch.bfloat16, device=dev), torch.empty((B, Hq), device=dev)

    def fresh():
        return (torch.full(fa2.fa2_kv16_cache_shape(P, Hkv, page, d), math.nan, dtype=torch.bfloat16, device=dev), i32([0, 0, 0]),
                i32(np.full((B, W), -1)), i32(np.arange(P)), i32([0, P]))

    def step(s):
        cache, lens, table, ring, state = s
        fa2.fa2_kv4_plan(lens, new, table, ring, state, page, 1, lens, acc, slots, state)
        fa2.fa2_kv16_append(x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:], slots.view(-1), cache, q=x[:, :Hq], positions=pos, inv_freq=f, q_out=q)
        fa2.fa2_fwd_kv16(q, cache, table, lens, starts, acc, o, lse, ws, causal=True)

    s = fresh()
    want = []
    for i in range(6):
        x.copy_(toks[i]), pos.fill_(i)
        step(s)
        want.append((o.clone(), lse.clone(), s[1].clone()))
    s = fresh()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(s)
    for i in range(6):
        x.copy_(toks[i]), pos.fill_(i)
        g.replay()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) and torch.equal(s[1], want[i][2])
    ok(fa2)


def test_chunks_give_what_the_whole_prompt_gives(gpu_lib):
    """A prompt in chunks over the cache, and dense by fa2_fwd_ex: within both bounds."""
    fa2 = gpu_lib
    rng = np.random.default_rng(88)
    n, Hq, Hkv, d, page = 700, 8, 2, 128, 64
    x = torch.tensor(rng.standard_normal((n, Hq + 2 * Hkv, d))).to(torch.bfloat16).cuda()
    W = -(-n // page)
    cache = torch.zeros(fa2.fa2_kv16_cache_shape(W, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    table = i32(rng.permutation(W)[None])
    pos, f = torch.arange(n, dtype=torch.int32, device="cuda"), torch.tensor(freqs(d)).cuda()
    qs, out, at = [], [], 0
    for m in (1, 300, 5, 250, 144):
        i = torch.arange(at, at + m, device="cuda")
        slots = (table[0, i // page] * page + i % page).int()
        part = x[at: at + m]
        _, q = fa2.fa2_kv16_append(part[:, Hq: Hq + Hkv], part[:, Hq + Hkv:], slots, cache, q=part[:, :Hq], positions=pos[at: at + m], inv_freq=f)
        qs.append(q)
        out.append(fa2.fa2_fwd_kv16(q, cache, table, i32([at + m]), i32([0]), i32([m]), causal=True))
        at += m
    q, k = fa2.fa2_rope(x[None, :, :Hq].transpose(1, 2), x[None, :, Hq: Hq + Hkv].transpose(1, 2), pos[None], f)
    assert torch.equal(torch.cat(qs), q[0].transpose(0, 1))
    o, lse = fa2.fa2_fwd_ex(q, k, x[None, :, Hq + Hkv:].transpose(1, 2).contiguous(), causal=True)
    ok(fa2)
    a, b = torch.cat([y[0] for y in out]).float(), o[0].transpose(0, 1).float()
    # weights and outputs round once on each side
    assert torch.allclose(torch.cat([y[1] for y in out]), lse[0].T, atol=1e-5, rtol=0)
    assert (a - b).abs().max() <= 2 * (2 * U["bf16"]) * float(x[:, Hq + Hkv:].abs().max())
