"""The paged 4-bit KV cache on the GPU against the fp64 oracle (oracle/kv4.py).

Bounds. append: every scale is a nearest e4m3 to max|x| / (6 descale) and
every code a nearest e2m1 to x / t, ties to even, up to 2^-20 of the value
for the fp32 quotients. gather: the definition's own fp32 products and one
rounding, so bit for bit. Attention, with A = sum_j p_j |v_j| (softmax p) and
u half a step of the output type (bf16 2^-8, fp16 2^-11):
    |O - ref| <= (2^-11 + 2 e + r) A + u |ref|,    |LSE - ref| <= e + r + 2^-22 |ref|
2^-11 is the fp16 rounding of the weights; e bounds the error of a score:
products of d fp32 terms at 2^-23 each relative to sum_d |q_d k_d| scale, and
four roundings of the exponent's terms; r the fp32 sums over the tokens and
partial results, (n / 8 + 64) 2^-23. Weights below 2^-22 of the largest may
round as fp16 subnormals, which adds 2^-32 n max|v| (2^-25 over the lift of 2^7).
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
# fp16 results below 2^-14 are multiples of 2^-24, half a step of which is
# 2^-25: more than U of them. Two keys one of which has almost all the weight
# give such elements where that one's value is 0.
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}


def ok(fa2):
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_OK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make_cache(rng, num_pages, Hkv, page, d, garbage=False):
    """Random codes and scales; `garbage`: any byte, NaN scales among them."""
    c = rng.integers(0, 256, (num_pages, Hkv, 2, page * (d // 2 + d // 16)), dtype=np.uint8)
    if not garbage:
        s = c[..., page * d // 2:]
        s[...] = rng.integers(0x28, 0x48, s.shape, dtype=np.uint8)   # 0.25 .. 3.75
    return c


def make_tables(rng, lens, page, spare=2, unused=-1):
    need = [-(-max(n, 0) // page) for n in lens]
    W = max(need) + spare
    ids = rng.permutation(sum(need) + 1)
    table, at = np.full((len(lens), W), unused, np.int64), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at: at + n]
        at += n
    return table, sum(need) + 1


def context(cache, table, lens, d, kd, vd):
    Hkv = cache.shape[1]
    out = []
    for part, ds in ((0, kd), (1, vd)):
        out.append([np.stack([kv4.tokens(cache, d, table[b], n, h, part, ds[h]) for h in range(Hkv)])
                    if n > 0 else np.zeros((Hkv, 0, d)) for b, n in enumerate(lens)])
    return out


def check_attention(o, lse, q, keys, values, scale, causal, lens, dtype):
    o, lse, q = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    ref, lref, A, big = kv4.attention(q, keys, values, scale, causal, lens)
    empty = np.isneginf(lref)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(o[empty] == 0)
    d = q.shape[-1]
    n = np.array([max(x, 0) for x in lens], float).reshape(-1, 1, 1)
    vmax = np.array([np.abs(v).max() if v.size else 0.0 for v in values]).reshape(-1, 1, 1, 1)
    full = ~empty
    e = (d + 8) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * np.abs(np.where(full, lref, 0)) + 2.0 ** -21
    r = np.broadcast_to((n / 8 + 64) * 2.0 ** -23, big.shape)
    bound = (2.0 ** -11 + 2 * e + r)[..., None] * A + 2.0 ** -32 * n[..., None] * vmax + U[dtype] * np.abs(ref) + SUB[dtype]
    err = np.abs(o - ref)
    assert np.all(err[full] <= bound[full]), f"O off by {(err[full] / np.maximum(bound[full], 1e-300)).max():.3g} bounds"
    lb = e + r + 2.0 ** -22 * np.abs(np.where(full, lref, 0))
    assert np.all(np.abs(lse[full] - lref[full]) <= lb[full]), "LSE"


def run_case(fa2, seed, lens, Hq, Hkv, Nq, d, page, causal, dtype, amp=1.0, garbage_behind=True):
    rng = np.random.default_rng(seed)
    table, P = make_tables(rng, lens, page)
    cache = make_cache(rng, P, Hkv, page, d)
    if garbage_behind:   # whatever lies behind a sequence, NaN scales too
        g = make_cache(rng, P, Hkv, page, d, garbage=True)
        cd, sc = cache[..., : page * d // 2], cache[..., page * d // 2:]
        gd, gs = g[..., : page * d // 2], g[..., page * d // 2:]
        used = np.zeros((P, page), bool)
        for b, n in enumerate(lens):
            for i in range(max(n, 0)):
                used[table[b, i // page], i % page] = True
        keep = used[:, None, None, :, None]
        shp = (P, Hkv, 2, page)
        cd[...] = np.where(keep, cd.reshape(*shp, -1), gd.reshape(*shp, -1)).reshape(cd.shape)
        sc[...] = np.where(keep, sc.reshape(*shp, -1), gs.reshape(*shp, -1)).reshape(sc.shape)
    kd, vd = (rng.uniform(0.3, 0.7, Hkv).astype(np.float32) for _ in range(2))
    q = torch.tensor(rng.standard_normal((len(lens), Hq, Nq, d)) * amp).to(DT[dtype])
    scale = d ** -0.5
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), torch.tensor(cache).cuda(), i32(table), i32(lens), torch.tensor(kd).cuda(),
                             torch.tensor(vd).cuda(), scale=scale, causal=causal)
    ok(fa2)
    keys, values = context(cache, table, lens, d, kd, vd)
    check_attention(o, lse, q, keys, values, scale, causal, lens, dtype)


CASES = [
    # lens, Hq, Hkv, Nq, d, page, causal, dtype
    ([1], 1, 1, 1, 128, 16, False, "bf16"),
    ([1], 4, 1, 1, 64, 128, False, "fp16"),
    ([0], 8, 2, 1, 128, 64, False, "bf16"),
    ([0, 0, 5, 0], 8, 2, 1, 64, 64, False, "bf16"),
    ([15, 16, 17, 31, 32, 33, 47, 48, 49], 8, 2, 1, 128, 16, False, "bf16"),
    ([63, 64, 65, 127, 128, 129, 1, 0, 200], 8, 2, 1, 64, 32, False, "fp16"),
    ([1000, 3, 517], 16, 2, 1, 128, 64, False, "bf16"),
    ([1000, 3, 517], 16, 16, 1, 64, 128, False, "bf16"),
    ([700, 0, 130], 14, 2, 1, 128, 64, False, "fp16"),     # 7 rows a head
    ([300, 40], 9, 1, 1, 128, 64, False, "bf16"),          # 9 rows: two blocks of eight
    ([300, 40], 32, 2, 1, 64, 16, False, "bf16"),          # 16 rows
    ([300, 40], 17, 1, 1, 128, 32, False, "fp16"),         # 17 rows
    ([3, 33, 300], 8, 2, 5, 128, 16, True, "bf16"),        # 20 rows, rows without a key
    ([3, 33, 300], 8, 2, 5, 128, 16, False, "bf16"),
    ([64, 97], 8, 1, 5, 64, 64, True, "fp16"),             # 40 rows: two row blocks
    ([150, 20], 4, 2, 37, 128, 32, True, "bf16"),          # 74 rows: three row blocks
    ([90], 2, 2, 100, 64, 128, True, "bf16"),              # more queries than keys
    ([7] * 90, 2, 1, 1, 64, 16, False, "bf16"),            # many short requests
    ([5, 0, 70] * 70, 4, 4, 2, 64, 16, True, "fp16"),      # more requests than threads
]


@pytest.mark.parametrize("lens,Hq,Hkv,Nq,d,page,causal,dtype", CASES)
def test_attention_every_element(gpu_lib, lens, Hq, Hkv, Nq, d, page, causal, dtype):
    run_case(gpu_lib, 11 + len(lens) + 7 * Hq + Nq + d + page, lens, Hq, Hkv, Nq, d, page, causal, dtype)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_context_is_split_and_joined(gpu_lib, d, page):
    run_case(gpu_lib, d + page, [20011], 4, 1, 1, d, page, False, "bf16", garbage_behind=False)


def test_attention_sharp_scores(gpu_lib):
    run_case(gpu_lib, 5, [900, 411], 8, 2, 1, 128, 64, False, "bf16", amp=8.0)


@pytest.mark.parametrize("step", [1.0, 6.0, 40.0])
def test_running_maximum_grows(gpu_lib, step):
    """Scores that grow from tile to tile by less, about and more than the slack."""
    fa2 = gpu_lib
    d, page, n = 128, 32, 640
    table, P = make_tables(np.random.default_rng(3), [n], page)
    rng = np.random.default_rng(int(step))
    cache = make_cache(rng, P, 1, page, d)
    codes, scales = cache[..., : page * d // 2], cache[..., page * d // 2:]
    scales = scales.reshape(P, 1, 2, page, d // 16)
    codes = codes.reshape(P, 1, 2, page, d // 2)
    for j in range(n):   # key j = level * (1, ..., 1), level growing with the tile
        codes[table[0, j // page], 0, 0, j % page] = 0x22      # 1.0
        level = int(np.searchsorted(kv4.E4M3[:127], (1 + j // 32) * step / 64.0))
        scales[table[0, j // page], 0, 0, j % page] = min(level, 126)
    ck = np.concatenate([codes.reshape(P, 1, 2, -1), scales.reshape(P, 1, 2, -1)], -1)
    q = torch.full((1, 4, 1, d), 64.0 * math.log(2) / d).to(torch.bfloat16)
    one = np.ones(1, np.float32)
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), torch.tensor(ck).cuda(), i32(table), i32([n]), torch.tensor(one).cuda(),
                             torch.tensor(one).cuda(), scale=1.0)
    ok(fa2)
    keys, values = context(ck, table, [n], d, one, one)
    check_attention(o, lse, q, keys, values, 1.0, False, [n], "bf16")


@pytest.mark.parametrize("mag", [1e-38, 1e-20, 1e30])
def test_bf16_query_rows_of_any_magnitude(gpu_lib, mag):
    fa2 = gpu_lib
    rng = np.random.default_rng(8)
    lens, d, page = [77], 64, 16
    table, P = make_tables(rng, lens, page)
    cache = make_cache(rng, P, 1, page, d)
    q = torch.tensor(rng.standard_normal((1, 3, 1, d))).to(torch.bfloat16)
    q[0, 1] = (q[0, 1].float() * mag).to(torch.bfloat16)
    one = np.ones(1, np.float32)
    scale = 0.1 if mag < 1 else 1e-30
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), torch.tensor(cache).cuda(), i32(table), i32(lens), torch.tensor(one).cuda(),
                             torch.tensor(one).cuda(), scale=scale)
    ok(fa2)
    keys, values = context(cache, table, lens, d, one, one)
    check_attention(o, lse, q, keys, values, scale, False, lens, "bf16")


def test_rows_that_are_not_finite_stay_alone(gpu_lib):
    fa2 = gpu_lib
    rng = np.random.default_rng(9)
    lens, d, page = [200, 60], 128, 64
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, 2, page, d)).cuda()
    one = torch.ones(2, device="cuda")
    q = torch.tensor(rng.standard_normal((2, 8, 1, d))).to(torch.bfloat16).cuda()
    o, lse = fa2.fa2_fwd_kv4(q, cache, i32(table), i32(lens), one, one)
    q2 = q.clone()
    q2[0, 1, 0, 5] = float("nan")
    q2[1, 6, 0, 100] = float("inf")
    o2, lse2 = fa2.fa2_fwd_kv4(q2, cache, i32(table), i32(lens), one, one)
    ok(fa2)
    assert o2[0, 1].isnan().all() and lse2[0, 1].isnan().all() and o2[1, 6].isnan().all()
    keep = torch.ones(2, 8, dtype=torch.bool)
    keep[0, 1] = keep[1, 6] = False
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])


def test_nan_in_the_cache_reaches_only_rows_that_see_it(gpu_lib):
    """A NaN scale in the key and the value of the last of four new tokens:
    under the mask only the last query row sees it."""
    fa2 = gpu_lib
    rng = np.random.default_rng(10)
    n, d, page, Nq = 70, 128, 16, 4
    table, P = make_tables(rng, [n], page)
    for part in (0, 1):
        cache = make_cache(rng, P, 1, page, d)
        one = torch.ones(1, device="cuda")
        q = torch.tensor(rng.standard_normal((1, 2, Nq, d))).to(torch.float16).cuda()
        o, lse = fa2.fa2_fwd_kv4(q, torch.tensor(cache).cuda(), i32(table), i32([n]), one, one, causal=True)
        cache[table[0, (n - 1) // page], 0, part, page * d // 2 + (n - 1) % page * (d // 16) + 3] = 0x7F
        o2, lse2 = fa2.fa2_fwd_kv4(q, torch.tensor(cache).cuda(), i32(table), i32([n]), one, one, causal=True)
        ok(fa2)
        assert torch.equal(o2[:, :, :3], o[:, :, :3]) and torch.equal(lse2[:, :, :3], lse[:, :, :3])
        if part:
            assert o2[:, :, 3, 48:64].isnan().all()
        else:
            assert o2[:, :, 3].isnan().all() and lse2[:, :, 3].isnan().all()


def test_bad_pages_are_skipped_and_reported(gpu_lib):
    """Ids outside the cache among a request's pages (checked on the device):
    their tokens count as absent, the call reports FA2_ERR_BOUNDS."""
    fa2 = gpu_lib
    rng = np.random.default_rng(12)
    n, d, page = 64, 64, 16
    table, P = make_tables(rng, [n], page)
    cache = make_cache(rng, P, 1, page, d)
    one = np.ones(1, np.float32)
    q = torch.tensor(rng.standard_normal((1, 4, 1, d))).to(torch.bfloat16)
    bad = table.copy()
    bad[0, 1], bad[0, 2] = P, -5
    c, ones = torch.tensor(cache).cuda(), torch.ones(1, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), c, i32(bad), i32([n]), ones, ones)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    keys, values = context(cache, table, [n], d, one, one)
    seen = np.r_[0:16, 48:64]
    check_attention(o, lse, q, [keys[0][:, seen]], [values[0][:, seen]], d ** -0.5, False, [32], "bf16")
    k, _ = fa2.fa2_kv4_gather(c, i32(bad), i32([n]), ones, ones, n, d)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    assert not k[0, 0, 16:48].any() and k[0, 0, :16].any()
    # a length behind the table's end is cut to it
    o2, lse2 = fa2.fa2_fwd_kv4(q.cuda(), c, i32(table[:, :4]), i32([n + 1]), ones, ones)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    check_attention(o2, lse2, q, keys, values, d ** -0.5, False, [n], "bf16")
    # slots outside the cache write nothing
    before = c.clone()
    kk = torch.ones(1, 1, 2, d, dtype=torch.bfloat16, device="cuda")
    fa2.fa2_kv4_append(kk, kk, i32([[P * page, -1]]), c, ones, ones)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    assert torch.equal(c, before)
    ok(fa2)


# ------------------------------------------------------------------ append and gather

MID = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def check_append(cache, x, slots, part, descale, d):
    """cache bytes against fp64 x [B, H, N, d] at slots [B, N]."""
    codes, scales = kv4.split(cache, d)
    page = codes.shape[3]
    B, H, N, _ = x.shape
    for b in range(B):
        for i in range(N):
            if slots[b, i] < 0:
                continue
            pg, row = divmod(int(slots[b, i]), page)
            for h in range(H):
                blk = x[b, h, i].reshape(-1, 16)
                sb = scales[pg, h, part, row]
                code = codes[pg, h, part, row].reshape(-1, 16)
                s = kv4.E4M3[sb]
                bad = ~np.isfinite(blk).all(1)
                assert np.isnan(s[bad]).all() and np.isfinite(s[~bad]).all() and (sb[~bad] < 0x80).all()
                blk, s, code, sb = blk[~bad], s[~bad], code[~bad], sb[~bad].astype(int)
                want = np.minimum(np.abs(blk).max(1) / (6 * float(descale[h])), 448.0)
                lo = (kv4.E4M3[np.maximum(sb - 1, 0)] + s) / 2
                hi = np.where(sb < 126, (kv4.E4M3[np.minimum(sb + 1, 126)] + s) / 2, np.inf)
                tol = 2.0 ** -20 * np.maximum(want, 2.0 ** -10)
                odd = (sb & 1) == 1
                assert np.all((want >= lo - tol) | (sb == 0)) and np.all(want <= hi + tol)
                # at a tie (exact when descale is a power of two) the even neighbour
                exact = np.log2(float(descale[h])) % 1 == 0
                if exact:
                    assert not np.any(odd & ((want == lo) | (want == hi)))
                t = (s.astype(np.float32) * np.float32(descale[h])).astype(np.float64)[:, None]
                y = np.divide(np.abs(blk), t, out=np.zeros_like(blk), where=t > 0)
                code = code.astype(int)
                m = code & 7
                v = np.abs(kv4.E2M1[code])
                lo = np.where(m > 0, MID[np.maximum(m - 1, 0)], -1.0)
                hi = np.where(m < 7, MID[np.minimum(m, 6)], np.inf)
                tol = 2.0 ** -20 * np.maximum(y, 2.0 ** -10)
                assert np.all(y >= lo - tol) and np.all(y <= hi + tol), (y, v)
                assert not np.any((m & 1 == 1) & ((y == lo) | (y == hi)))
                neg = (blk < 0) & (v > 0)
                assert np.array_equal(neg, (code > 7) & (v > 0))


@pytest.mark.parametrize("B,H,N,d,page,dtype,descale", [
    (1, 1, 1, 128, 16, "bf16", 1.0),
    (3, 2, 5, 64, 16, "fp16", 0.25),
    (2, 3, 37, 128, 32, "bf16", 0.0017),
    (1, 8, 130, 128, 64, "bf16", 0.37),
    (2, 1, 300, 64, 128, "fp16", 0.0625),
])
def test_append_and_gather(gpu_lib, B, H, N, d, page, dtype, descale):
    fa2 = gpu_lib
    rng = np.random.default_rng(B + N + d)
    counts = [N] + [int(rng.integers(0, N + 1)) for _ in range(B - 1)]
    starts = [int(rng.integers(0, 40)) for _ in range(B)]
    lens = [s + n for s, n in zip(starts, counts)]
    table, P = make_tables(rng, lens, page)
    kd, vd = (np.full(H, descale, np.float32) * np.float32(f) for f in (1.0, 2.0))
    k, v = (torch.tensor(rng.standard_normal((B, H, N, d))).to(DT[dtype]) for _ in range(2))
    k[..., :16] = 0                                  # a block of zeros
    v[..., 16:32] *= 2.0 ** -14 if dtype == "fp16" else 2.0 ** -40   # far below the scales' range
    v[0, 0, 0, 40] = 6e4                             # far above the others
    slots = np.full((B, N), -1)
    for b in range(B):
        for i in range(counts[b]):
            p = starts[b] + i
            slots[b, i] = table[b, p // page] * page + p % page
    old = torch.tensor(make_cache(rng, P, H, page, d))
    cache = old.cuda()
    dk, dv = torch.tensor(kd).cuda(), torch.tensor(vd).cuda()
    # a view of one projection's output [B, N, 2, H, d], no copy
    both = torch.stack([k, v], 1).permute(0, 3, 1, 2, 4).contiguous().cuda()
    fa2.fa2_kv4_append(both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2), i32(slots), cache, dk, dv)
    ok(fa2)
    got = cache.cpu().numpy()
    check_append(got, k.double().numpy(), slots, 0, kd, d)
    check_append(got, v.double().numpy(), slots, 1, vd, d)
    # every other token's bytes stay as they were
    oc, osc = kv4.split(old.numpy(), d)
    nc, nsc = kv4.split(got, d)
    touched = np.zeros((P, page), bool)
    touched.reshape(-1)[slots[slots >= 0]] = True
    same = ~touched
    assert np.array_equal(nc.transpose(0, 3, 1, 2, 4)[same], oc.transpose(0, 3, 1, 2, 4)[same])
    assert np.array_equal(nsc.transpose(0, 3, 1, 2, 4)[same], osc.transpose(0, 3, 1, 2, 4)[same])
    # contiguous inputs write the same bytes
    again = old.cuda()
    fa2.fa2_kv4_append(k.cuda(), v.cuda(), i32(slots), again, dk, dv)
    assert torch.equal(again, cache)

    gk, gv = fa2.fa2_kv4_gather(cache, i32(table), i32(lens), dk, dv, N, d, starts=i32(starts), dtype=DT[dtype])
    ok(fa2)
    for out, part, ds in ((gk, 0, kd), (gv, 1, vd)):
        t = kv4.scale32(nsc, ds[None, :, None, None, None])
        want = (kv4.E2M1[nc].astype(np.float32) * np.repeat(t, 16, -1)).astype(np.float32)
        ref = torch.zeros(B, H, N, d)
        for b in range(B):
            for i in range(counts[b]):
                pg, row = divmod(int(slots[b, i]), page)
                ref[b, :, i] = torch.tensor(want[pg, :, part, row])
        assert torch.equal(out.cpu(), ref.to(DT[dtype]))


def test_append_ties_go_to_the_even_code(gpu_lib):
    """All seven midpoints of the codes, and scales at midpoints of e4m3."""
    fa2 = gpu_lib
    one = torch.ones(1, device="cuda")
    cache = torch.zeros(fa2.fa2_kv4_cache_shape(1, 1, 16, 64), dtype=torch.uint8, device="cuda")
    x = torch.zeros(1, 1, 2, 64)
    x[0, 0, 0, :9] = torch.tensor([6.0, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, -0.25])
    x[0, 0, 1, 0] = 6.0 * 1.0625     # between scales 1 and 1.125: 1 is even
    x[0, 0, 1, 16] = 6.0 * 1.1875    # between 1.125 and 1.25: 1.25 is even
    x = x.to(torch.bfloat16).cuda()
    fa2.fa2_kv4_append(x, x, i32([[0, 1]]), cache, one, one)
    ok(fa2)
    codes, scales = kv4.split(cache.cpu().numpy(), 64)
    assert list(codes[0, 0, 0, 0, :8]) == [7, 0, 2, 8 + 2, 4, 4, 8 + 6, 6] and codes[0, 0, 0, 0, 8] & 7 == 0
    assert kv4.E4M3[scales[0, 0, 0, 1, 0]] == 1.0 and kv4.E4M3[scales[0, 0, 0, 1, 1]] == 1.25


def test_append_of_values_that_are_not_finite(gpu_lib):
    fa2 = gpu_lib
    one = torch.ones(2, device="cuda")
    cache = torch.zeros(fa2.fa2_kv4_cache_shape(2, 2, 16, 128), dtype=torch.uint8, device="cuda")
    k = torch.randn(1, 2, 3, 128).to(torch.bfloat16).cuda()
    k[0, 1, 1, 20] = float("inf")
    k[0, 0, 2, 127] = float("nan")
    fa2.fa2_kv4_append(k, k, i32([[3, 4, 20]]), cache, one, one)
    table = i32([[0, 1]])
    gk, _ = fa2.fa2_kv4_gather(cache, table, i32([32]), one, one, 32, 128)
    ok(fa2)
    bad = torch.zeros(2, 32, 128, dtype=torch.bool)
    bad[1, 4, 16:32] = True
    bad[0, 20, 112:] = True
    assert torch.equal(gk[0].isnan().cpu(), bad)


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("B,N,page,W,seed,tight", [
    (1, 1, 16, 4, 0, False), (7, 1, 16, 5, 1, False), (40, 1, 64, 30, 2, True), (300, 1, 16, 8, 3, True),
    (5, 100, 16, 9, 4, False), (33, 257, 32, 20, 5, True), (2100, 3, 16, 3, 6, False), (2100, 3, 16, 3, 7, True),
    (64, 64, 128, 2, 8, True), (20, 1000, 16, 80, 9, False), (70, 515, 64, 12, 10, True), (1100, 300, 128, 5, 11, True),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(gpu_lib, B, N, page, W, seed, tight, in_place):
    fa2 = gpu_lib
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, W * page + 1, B)
    new = rng.integers(-1, N + 2, B)       # ends, nothing, tokens, one too many
    have = -(-lens // page)
    P = int(have.sum()) + B + 5
    ids = rng.permutation(P)
    table = np.full((B, W), -7)
    at = 0
    for b in range(B):
        table[b, : have[b]] = ids[at: at + have[b]]
        at += have[b]
    free = (P - at) // (4 if tight else 1)
    first = int(rng.integers(0, P))
    ring = np.full(P, -9)
    ring[(first + np.arange(free)) % P] = ids[at: at + free]
    want = kv4.plan(lens, new, table, ring, [first, free], page, N)
    t, r, ln, st = i32(table), i32(ring), i32(lens), i32([first, free])
    keep_l, keep_s = ln.clone(), st.clone()
    kw = {"seq_lens_out": ln, "free_state_out": st} if in_place else {}
    got = fa2.fa2_kv4_plan(ln, i32(new), t, r, st, page, N, **kw)
    ok(fa2)
    for x, y in zip((*got, t, r), want):
        assert np.array_equal(x.cpu().numpy(), np.asarray(y))
    if not in_place:
        assert torch.equal(ln, keep_l) and torch.equal(st, keep_s)


def test_plan_reports_what_is_no_length_or_ring(gpu_lib):
    fa2 = gpu_lib
    stream = torch.cuda.current_stream().cuda_stream
    t, r = i32(np.full((2, 2), -1)), i32(np.arange(8))
    lens, acc, slots, st = fa2.fa2_kv4_plan(i32([-3, 33]), i32([1, 1]), t, r, i32([0, 8]), 16, 1)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    assert lens.tolist() == [1, 1] and slots.tolist() == [[0], [16]]
    for state in ([-1, 3], [8, 1], [0, 9], [0, -1]):
        lens, acc, slots, st = fa2.fa2_kv4_plan(i32([0, 5]), i32([1, 1]), i32([[-1, -1], [3, -1]]), r, i32(state), 16, 1)
        assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
        assert acc.tolist() == [0, 1] and slots.tolist() == [[-1], [3 * 16 + 5]]


# ------------------------------------------------------------------ as a program uses them

def serve(fa2, steps, B, Hq, Hkv, d, page, dtype, seed):
    """A small serving loop; yields what a step's checks need."""
    rng = np.random.default_rng(seed)
    W, P = 6, 4 * B
    dev = "cuda"
    cache = torch.full(fa2.fa2_kv4_cache_shape(P, Hkv, page, d), 0xFF, dtype=torch.uint8, device=dev)
    kd, vd = torch.full((Hkv,), 0.002, device=dev), torch.full((Hkv,), 0.003, device=dev)
    lens, state = i32(np.zeros(B)), i32([0, P])
    table, ring = i32(np.full((B, W), -1)), i32(rng.permutation(P))
    kept = [[] for _ in range(B)]
    for step in range(steps):
        N = 40 if step % 4 == 0 else 3
        new = rng.integers(0, N + 1, B)
        if step:
            new[rng.random(B) < 0.2] = -1
        _, acc, slots, _ = fa2.fa2_kv4_plan(lens, i32(new), table, ring, state, page, N, seq_lens_out=lens,
                                            free_state_out=state)
        k, v = (torch.tensor(rng.standard_normal((B, Hkv, N, d))).to(DT[dtype]).to(dev) for _ in range(2))
        fa2.fa2_kv4_append(k, v, slots, cache, kd, vd)
        q = torch.tensor(rng.standard_normal((B, Hq, N, d))).to(DT[dtype]).to(dev)
        o, lse = fa2.fa2_fwd_kv4(q, cache, table, lens, kd, vd, causal=True)
        ok(fa2)
        for b, (a, n) in enumerate(zip(acc.tolist(), new.tolist())):
            kept[b] = [] if n < 0 else kept[b] + [(step, b, i) for i in range(a)]
            assert len(kept[b]) == int(lens[b])
        yield cache, table, lens, kd, vd, q, o, lse, kept, (k, v)


@pytest.mark.parametrize("d,page,dtype", [(128, 16, "bf16"), (64, 32, "fp16")])
def test_plan_append_attend_together(gpu_lib, d, page, dtype):
    """Lengths, pages given back and reused, appended tokens and attention
    over them agree with the oracle step by step, and gather plus fa2_fwd_ex
    gives the same attention to within both bounds."""
    fa2 = gpu_lib
    used = set()
    for cache, table, lens, kd, vd, q, o, lse, kept, _ in serve(fa2, 9, 5, 4, 2, d, page, dtype, 77):
        n = lens.tolist()
        tb = table.cpu().numpy()
        live = [p for b in range(5) for p in tb[b, : -(-n[b] // page)]]
        assert len(set(live)) == len(live)          # no page is handed out twice
        used |= set(live)
        c = cache.cpu().numpy()
        keys, values = context(c, tb, n, d, kd.cpu().numpy(), vd.cpu().numpy())
        check_attention(o, lse, q, keys, values, d ** -0.5, True, n, dtype)
        b = int(np.argmax(n))
        if n[b] == 0:
            continue
        k, v = fa2.fa2_kv4_gather(cache, table[b: b + 1], lens[b: b + 1], kd, vd, n[b], d, dtype=DT[dtype])
        o2, l2 = fa2.fa2_fwd_ex(q[b: b + 1], k, v, causal=True)
        ok(fa2)
        tol = 4 * U[dtype]
        seen = torch.isfinite(lse[b])
        assert torch.equal(seen, torch.isfinite(l2[0]))
        assert torch.allclose(l2[0][seen], lse[b][seen], atol=16 * U[dtype], rtol=U[dtype])
        assert torch.allclose(o2[0].float(), o[b].float(), atol=8 * U[dtype], rtol=tol)
    assert len(used) > 5


def test_appended_tokens_are_what_is_attended(gpu_lib):
    """From the new tokens themselves: quantised in 64 bits, attended in 64 bits."""
    fa2 = gpu_lib
    rng = np.random.default_rng(21)
    B, Hq, Hkv, N, d, page = 2, 4, 2, 45, 128, 16
    lens = [45, 30]
    table, P = make_tables(rng, lens, page)
    slots = np.full((B, N), -1)
    for b in range(B):
        for i in range(lens[b]):
            slots[b, i] = table[b, i // page] * page + i % page
    k, v = (torch.tensor(rng.standard_normal((B, Hkv, N, d))).to(torch.bfloat16) for _ in range(2))
    cache = torch.zeros(fa2.fa2_kv4_cache_shape(P, Hkv, page, d), dtype=torch.uint8, device="cuda")
    one = torch.full((Hkv,), 2.0 ** -9, device="cuda")
    fa2.fa2_kv4_append(k.cuda(), v.cuda(), i32(slots), cache, one, one)
    q = torch.tensor(rng.standard_normal((B, Hq, 1, d))).to(torch.bfloat16)
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), cache, i32(table), i32(lens), one, one)
    ok(fa2)

    keys, values = ([kv4.rounded(x[b, :, : lens[b]].double().numpy(), 2.0 ** -9) for b in range(B)] for x in (k, v))
    check_attention(o, lse, q, keys, values, d ** -0.5, False, lens, "bf16")


def test_captured_step_replays_with_new_lengths(gpu_lib):
    """plan, append and attention in one CUDA graph; every replay goes on
    from the lengths that the last one left."""
    fa2 = gpu_lib
    rng = np.random.default_rng(31)
    B, Hq, Hkv, d, page, W, P = 3, 8, 2, 128, 16, 8, 40
    dev = "cuda"

    def fresh():
        cache = torch.zeros(fa2.fa2_kv4_cache_shape(P, Hkv, page, d), dtype=torch.uint8, device=dev)
        return cache, i32([0, 0, 0]), i32(np.full((B, W), -1)), i32(np.arange(P)), i32([0, P])

    ds = torch.full((Hkv,), 0.002, device=dev)
    toks = torch.tensor(rng.standard_normal((6, 3, B, Hkv, 1, d))).to(torch.bfloat16).to(dev)
    qs = torch.tensor(rng.standard_normal((6, B, Hq, 1, d))).to(torch.bfloat16).to(dev)
    k, v, q = torch.empty_like(toks[0, 0]), torch.empty_like(toks[0, 1]), torch.empty_like(qs[0])
    new = i32([1, 1, 1])
    acc, slots = torch.empty_like(new), torch.empty((B, 1), dtype=torch.int32, device=dev)
    ws = torch.empty(fa2.fa2_fwd_kv4_workspace(B, Hq, Hkv, 1, d, W, page), dtype=torch.uint8, device=dev)
    o, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device=dev)

    def step(s):
        cache, lens, table, ring, state = s
        fa2.fa2_kv4_plan(lens, new, table, ring, state, page, 1, lens, acc, slots, state)
        fa2.fa2_kv4_append(k, v, slots, cache, ds, ds)
        fa2.fa2_fwd_kv4(q, cache, table, lens, ds, ds, o, lse, ws)

    s = fresh()
    want = []
    for i in range(6):
        k.copy_(toks[i, 0]), v.copy_(toks[i, 1]), q.copy_(qs[i])
        step(s)
        want.append((o.clone(), lse.clone(), s[1].clone()))
    s = fresh()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(s)
    for i in range(6):
        k.copy_(toks[i, 0]), v.copy_(toks[i, 1]), q.copy_(qs[i])
        g.replay()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) and torch.equal(s[1], want[i][2])
    ok(fa2)


def test_two_calls_on_two_streams(gpu_lib):
    fa2 = gpu_lib
    rng = np.random.default_rng(41)
    lens, d, page = [5000, 1200], 128, 64
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, 2, page, d)).cuda()
    one = torch.ones(2, device="cuda")
    t, ln = i32(table), i32(lens)
    q = [torch.tensor(rng.standard_normal((2, 8, 1, d))).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [fa2.fa2_fwd_kv4(x, cache, t, ln, one, one) for x in q]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        got.append(fa2.fa2_fwd_kv4(q[i % 2], cache, t, ln, one, one, stream=st[i % 2]))
    for s in st:
        assert fa2.fa2_check_status(s.cuda_stream) == fa2.FA2_OK
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_cache_behind_four_gigabytes(gpu_lib):
    """Pages whose byte offsets pass 32 bits."""
    fa2 = gpu_lib
    rng = np.random.default_rng(51)
    Hkv, d, page = 8, 128, 128
    shape = fa2.fa2_kv4_cache_shape(1, Hkv, page, d)
    size = int(np.prod(shape))
    P = (1 << 32) // size + 200
    cache = torch.empty((P, *shape[1:]), dtype=torch.uint8, device="cuda")
    n = 300
    table = np.array([[P - 1, P - 7, P - 3, -1]])
    part = make_cache(rng, 3, Hkv, page, d)
    for j in range(3):
        cache[int(table[0, j])] = torch.tensor(part[j]).cuda()
    one = np.ones(Hkv, np.float32)
    q = torch.tensor(rng.standard_normal((1, 8, 1, d))).to(torch.float16)
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), cache, i32(table), i32([n]), torch.tensor(one).cuda(), torch.tensor(one).cuda())
    keys, values = context(part, np.array([[0, 1, 2]]), [n], d, one, one)
    check_attention(o, lse, q, keys, values, d ** -0.5, False, [n], "fp16")
    # written and read back at the far end
    k = torch.tensor(rng.standard_normal((1, Hkv, 2, d))).to(torch.bfloat16).cuda()
    fa2.fa2_kv4_append(k, k, i32([[(P - 1) * page + 5, (P - 3) * page + 43]]), cache, torch.tensor(one).cuda(),
                       torch.tensor(one).cuda())
    gk, gv = fa2.fa2_kv4_gather(cache, i32(table), i32([n]), torch.tensor(one).cuda(), torch.tensor(one).cuda(), n, d)
    ok(fa2)
    for pos, i in ((5, 0), (299, 1)):
        step = k[0, :, i].float().reshape(Hkv, -1, 16).abs().amax(-1, keepdim=True) / 6
        assert ((gk[0, :, pos] - k[0, :, i]).float().reshape(Hkv, -1, 16).abs() <= 1.2 * step).all()
        assert torch.equal(gk[0, :, pos], gv[0, :, pos])


def test_results_repeat_bit_for_bit(gpu_lib):
    fa2 = gpu_lib
    rng = np.random.default_rng(61)
    lens, d, page = [9000, 0, 333, 4097], 64, 32
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, 2, page, d)).cuda()
    one = torch.ones(2, device="cuda")
    q = torch.tensor(rng.standard_normal((4, 16, 3, d))).to(torch.bfloat16).cuda()
    a = [fa2.fa2_fwd_kv4(q, cache, i32(table), i32(lens), one, one, causal=True) for _ in range(5)]
    ok(fa2)
    assert all(torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1]) for x in a)


def test_refusals_on_the_device(gpu_lib):
    fa2 = gpu_lib
    dev = "cuda"
    cache = torch.zeros(fa2.fa2_kv4_cache_shape(4, 2, 16, 64), dtype=torch.uint8, device=dev)
    ds, table, lens = torch.ones(2, device=dev), i32(np.zeros((1, 4))), i32([5])
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device=dev)
    good = (q, cache, table, lens, ds, ds)
    fa2.fa2_fwd_kv4(*good)
    for i, bad in ((0, q.float()), (0, q[:, :3].contiguous()), (0, q[..., :32].contiguous()), (0, q.transpose(1, 2)[:, ::1].expand(1, 4, 4, 64)),
                   (1, cache[:, :1]), (1, cache.int()), (1, cache[..., :-1]), (2, table.long()), (2, table[:, ::2]),
                   (3, lens.cpu()), (3, i32([5, 5])), (4, ds[:1]), (5, ds.double())):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
            fa2.fa2_fwd_kv4(*args)
    wide = list(good)
    wide[2] = i32(np.zeros((1, 400)))
    with pytest.raises(fa2.FA2Error):
        fa2.fa2_fwd_kv4(*wide, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    fa2.fa2_fwd_kv4(*wide)
    with pytest.raises(ValueError):
        fa2.fa2_fwd_kv4(*good, o=torch.empty(1, 4, 1, 64, device=dev))
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device=dev)
    slots = i32(np.zeros((1, 3)))
    for a in ((k.transpose(2, 3), k.transpose(2, 3), slots), (k, k.half(), slots), (k, k, slots[:, :2]),
              (torch.zeros(1, 2, 3, 68, dtype=torch.bfloat16, device=dev)[..., :64],) * 2 + (slots,),
              (torch.zeros(1, 2, 3, 72, dtype=torch.bfloat16, device=dev)[..., 4:68],) * 2 + (slots,)):
        with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
            fa2.fa2_kv4_append(*a, cache, ds, ds)
    ok(fa2)


# ------------------------------------------------------------------ many query rows a KV head

ROWS = [  # Hq, Hkv, Nq: 12 to 24 rows a head in one pass of mma.sync, above on tcgen05, above 64 in blocks
    (12, 1, 1), (4, 1, 4), (6, 2, 8), (25, 1, 1), (8, 1, 4), (12, 1, 3), (6, 2, 16), (4, 2, 32), (13, 1, 5), (8, 1, 16),
]


@pytest.mark.parametrize("d,page,dtype,causal", [(128, 64, "bf16", True), (64, 16, "fp16", False), (64, 128, "bf16", True),
                                                 (128, 32, "fp16", False)])
@pytest.mark.parametrize("Hq,Hkv,Nq", ROWS)
def test_many_rows_long_and_short_together(gpu_lib, Hq, Hkv, Nq, d, page, dtype, causal):
    """A context that several CTAs share and join, beside empty and short ones."""
    run_case(gpu_lib, 100 * Hq + Nq + d, [6001, 0, 2, 127, 129, 1500], Hq, Hkv, Nq, d, page, causal, dtype)


@pytest.mark.parametrize("Hq,Nq", [(16, 1), (24, 1), (32, 1), (16, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_and_a_table_that_needs_no_workspace(gpu_lib, Hq, Nq, d):
    """As many CTAs as segments, each with one of its own, or 125 short requests."""
    for lens, Hkv in (([500, 1, 0, 130], 3), ([33, 0, 140, 7, 128] * 25, 1)):
        W = -(-max(lens) // 16) + 2
        assert gpu_lib.fa2_fwd_kv4_workspace(len(lens), Hq * Hkv, Hkv, Nq, d, W, 16) == 0
        run_case(gpu_lib, Hq + d + len(lens), lens, Hq * Hkv, Hkv, Nq, d, 16, True, "bf16")


@pytest.mark.parametrize("step", [1.0, 6.0, 40.0])
@pytest.mark.parametrize("rows", [10, 20, 32, 48, 64])
def test_running_maximum_of_many_rows(gpu_lib, rows, step):
    """Rows whose scores grow from tile to tile by less, about and more than
    the slack, beside rows whose scores fall or stay."""
    fa2 = gpu_lib
    d, page, n = 128, 32, 2560
    rng = np.random.default_rng(int(step) + rows)
    table, P = make_tables(rng, [n], page)
    cache = make_cache(rng, P, 1, page, d)
    codes, scales = cache[..., : page * d // 2], cache[..., page * d // 2:]
    scales = scales.reshape(P, 1, 2, page, d // 16)
    codes = codes.reshape(P, 1, 2, page, d // 2)
    for j in range(n):
        codes[table[0, j // page], 0, 0, j % page] = 0x22      # 1.0
        level = int(np.searchsorted(kv4.E4M3[:127], (1 + j // 128) * step / 64.0))
        scales[table[0, j // page], 0, 0, j % page] = min(level, 126)
    ck = np.concatenate([codes.reshape(P, 1, 2, -1), scales.reshape(P, 1, 2, -1)], -1)
    q = torch.full((1, rows, 1, d), 64.0 * math.log(2) / d)
    q *= torch.tensor([1.0, 0.25, -1.0, 0.0, 0.5]).repeat(rows)[:rows].reshape(1, rows, 1, 1)
    q = q.to(torch.bfloat16)
    one = np.ones(1, np.float32)
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), torch.tensor(ck).cuda(), i32(table), i32([n]), torch.tensor(one).cuda(),
                             torch.tensor(one).cuda(), scale=1.0)
    ok(fa2)
    keys, values = context(ck, table, [n], d, one, one)
    check_attention(o, lse, q, keys, values, 1.0, False, [n], "bf16")


@pytest.mark.parametrize("dtype,mag", [("bf16", 1e-38), ("bf16", 1e30), ("fp16", 6e-8), ("fp16", 3e4)])
@pytest.mark.parametrize("Hq", [16, 40])
def test_many_query_rows_of_any_magnitude(gpu_lib, Hq, dtype, mag):
    fa2 = gpu_lib
    rng = np.random.default_rng(8)
    lens, d, page = [177], 64, 16
    table, P = make_tables(rng, lens, page)
    cache = make_cache(rng, P, 1, page, d)
    q = torch.tensor(np.clip(rng.standard_normal((1, Hq, 1, d)), -2, 2)).to(DT[dtype])
    q[0, 1::3] = (q[0, 1::3].float() * mag).to(DT[dtype])
    one = np.ones(1, np.float32)
    scale = 0.1 if mag < 1 else 1.0 / mag
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), torch.tensor(cache).cuda(), i32(table), i32(lens), torch.tensor(one).cuda(),
                             torch.tensor(one).cuda(), scale=scale)
    ok(fa2)
    keys, values = context(cache, table, lens, d, one, one)
    check_attention(o, lse, q, keys, values, scale, False, lens, dtype)


@pytest.mark.parametrize("Hq,Nq", [(4, 4), (12, 4), (16, 8)])
def test_what_is_not_finite_stays_with_its_rows(gpu_lib, Hq, Nq):
    """NaN scales of the last new token reach the last query row of each head;
    a query row with a NaN or an infinity leaves the others as they were."""
    fa2 = gpu_lib
    rng = np.random.default_rng(10)
    n, d, page = 270, 128, 16
    table, P = make_tables(rng, [n], page)
    t, ln, one = i32(table), i32([n]), torch.ones(1, device="cuda")
    q = torch.tensor(rng.standard_normal((1, Hq, Nq, d))).to(torch.float16).cuda()
    cache = make_cache(rng, P, 1, page, d)
    clean = torch.tensor(cache).cuda()
    o, lse = fa2.fa2_fwd_kv4(q, clean, t, ln, one, one, causal=True)
    for part in (0, 1):
        c = cache.copy()
        c[table[0, (n - 1) // page], 0, part, page * d // 2 + (n - 1) % page * (d // 16) + 3] = 0xFF
        o2, lse2 = fa2.fa2_fwd_kv4(q, torch.tensor(c).cuda(), t, ln, one, one, causal=True)
        ok(fa2)
        assert torch.equal(o2[:, :, :-1], o[:, :, :-1]) and torch.equal(lse2[:, :, :-1], lse[:, :, :-1])
        if part:
            assert o2[:, :, -1, 48:64].isnan().all()
            assert torch.equal(o2[:, :, -1, :48], o[:, :, -1, :48]) and torch.equal(o2[:, :, -1, 64:], o[:, :, -1, 64:])
        else:
            assert o2[:, :, -1].isnan().all() and lse2[:, :, -1].isnan().all()
    q2 = q.clone()
    q2[0, 1, 2, 5], q2[0, Hq - 1, 0, 100] = float("nan"), float("inf")
    o2, lse2 = fa2.fa2_fwd_kv4(q2, clean, t, ln, one, one, causal=True)
    ok(fa2)
    keep = torch.ones(1, Hq, Nq, dtype=torch.bool)
    keep[0, 1, 2] = keep[0, Hq - 1, 0] = False
    assert o2[~keep].isnan().all()
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])


@pytest.mark.parametrize("Hq", [4, 16, 40])
def test_bad_pages_of_many_rows(gpu_lib, Hq):
    """In a first, a middle and a last tile, a whole tile among them."""
    fa2 = gpu_lib
    rng = np.random.default_rng(13)
    n, d, page = 5000, 128, 16
    table, P = make_tables(rng, [n], page)
    cache = make_cache(rng, P, 1, page, d)
    one = np.ones(1, np.float32)
    q = torch.tensor(rng.standard_normal((1, Hq, 1, d))).to(torch.bfloat16)
    bad = table.copy()
    out = [0, 3, *range(24, 32), 100, 101, 312]
    bad[0, out] = rng.choice([-1, P, 2 ** 31 - 1, -2 ** 31], len(out))
    c, ones = torch.tensor(cache).cuda(), torch.ones(1, device="cuda")
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), c, i32(bad), i32([n]), ones, ones)
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_ERR_BOUNDS
    keys, values = context(cache, table, [n], d, one, one)
    seen = np.concatenate([np.arange(j * page, min((j + 1) * page, n)) for j in range(-(-n // page)) if j not in out])
    check_attention(o, lse, q, [keys[0][:, seen]], [values[0][:, seen]], d ** -0.5, False, [len(seen)], "bf16")
    bad[0] = -1   # no token at all is left
    o, lse = fa2.fa2_fwd_kv4(q.cuda(), c, i32(bad), i32([n]), ones, ones)
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_ERR_BOUNDS
    assert not o.any() and lse.isneginf().all()


@pytest.mark.parametrize("Hq,Nq", [(8, 1), (16, 1), (8, 3), (12, 4), (16, 8)])
def test_graphs_that_share_a_workspace(gpu_lib, Hq, Nq):
    """Two captured calls of different shapes, replayed in turn on one stream
    with one workspace that held anything before, while eager calls use it too."""
    fa2 = gpu_lib
    rng = np.random.default_rng(71)
    d, page = 128, 64
    one = torch.ones(2, device="cuda")
    calls, need = [], 0
    for lens in ([7000, 300, 0], [90, 12000]):
        table, P = make_tables(rng, lens, page)
        cache = torch.tensor(make_cache(rng, P, 2, page, d)).cuda()
        q = torch.tensor(rng.standard_normal((len(lens), 2 * Hq, Nq, d))).to(torch.bfloat16).cuda()
        args = (q, cache, i32(table), i32(lens), one, one)
        want = fa2.fa2_fwd_kv4(*args, causal=True)
        need = max(need, fa2.fa2_fwd_kv4_workspace(len(lens), 2 * Hq, 2, Nq, d, table.shape[1], page))
        calls.append((args, want, torch.empty_like(want[0]), torch.empty_like(want[1])))
    assert need > 0
    ws = torch.tensor(rng.integers(0, 256, need, dtype=np.uint8)).cuda()
    torch.cuda.synchronize()
    graphs = []
    for args, _, o, lse in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa2.fa2_fwd_kv4(*args, o, lse, ws, causal=True)
        graphs.append(g)
    for _ in range(3):
        for i in (0, 0, 1, 0, 1, 1):
            args, want, o, lse = calls[i]
            o.fill_(7), lse.fill_(7)
            graphs[i].replay()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            args, want, _, _ = calls[1 - i]
            got = fa2.fa2_fwd_kv4(*args, None, None, ws, causal=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok(fa2)


@pytest.mark.parametrize("Hq,Nq,d", [(16, 1, 128), (24, 1, 64), (32, 1, 128), (16, 4, 64), (16, 8, 128)])
def test_many_rows_repeat_bit_for_bit(gpu_lib, Hq, Nq, d):
    fa2 = gpu_lib
    rng = np.random.default_rng(62)
    lens, page = [9000, 0, 333, 4097], 32
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, 2, page, d)).cuda()
    one = torch.ones(2, device="cuda")
    q = torch.tensor(rng.standard_normal((4, 2 * Hq, Nq, d))).to(torch.bfloat16).cuda()
    a = [fa2.fa2_fwd_kv4(q, cache, i32(table), i32(lens), one, one, causal=True) for _ in range(8)]
    ok(fa2)
    assert all(torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1]) for x in a)


def test_calls_on_a_given_stream_allocate_from_it(gpu_lib):
    """What a call with `stream` allocates belongs to that stream: memory given
    back there is reused behind the work queued on it, without a wait."""
    fa2 = gpu_lib
    rng = np.random.default_rng(63)
    lens, d, page = [12000, 3], 128, 64
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, 2, page, d)).cuda()
    one, t, ln = torch.ones(2, device="cuda"), i32(table), i32(lens)
    q = torch.tensor(rng.standard_normal((2, 16, 1, d))).to(torch.bfloat16).cuda()
    want = fa2.fa2_fwd_kv4(q, cache, t, ln, one, one)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(30):
        got = fa2.fa2_fwd_kv4(q, cache, t, ln, one, one, stream=side)
        kv = fa2.fa2_kv4_gather(cache, t, ln, one, one, 500, d, stream=side.cuda_stream)
        with torch.cuda.stream(side):
            same = torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert same and not kv[0][1, :, 3:].any()
        del kv
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    again = fa2.fa2_fwd_kv4(q, cache, t, ln, one, one, stream=0)   # the default stream's handle
    assert torch.equal(again[0], want[0])
    ok(fa2)


@pytest.mark.parametrize("d", [64, 128])
def test_watchdog_of_many_rows(gpu_lib, d):
    """A wait that runs out ends the call with a status; the context and the
    workspace stay usable."""
    fa2 = gpu_lib
    rng = np.random.default_rng(64)
    lens, page = [6000, 20], 64
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, 1, page, d)).cuda()
    one, t, ln = torch.ones(1, device="cuda"), i32(table), i32(lens)
    q = torch.tensor(rng.standard_normal((2, 32, 1, d))).to(torch.bfloat16).cuda()
    ws = torch.zeros(fa2.fa2_fwd_kv4_workspace(2, 32, 1, 1, d, table.shape[1], page), dtype=torch.uint8, device="cuda")
    want = fa2.fa2_fwd_kv4(q, cache, t, ln, one, one, workspace=ws)
    ok(fa2)
    old_limit = fa2.fa2_set_wait_limit_ns(20_000_000)
    old_flags = fa2.fa2_set_debug_flags(1)
    try:
        fa2.fa2_fwd_kv4(q, cache, t, ln, one, one, workspace=ws)
        rc = fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream)
    finally:
        fa2.fa2_set_debug_flags(old_flags)
        fa2.fa2_set_wait_limit_ns(old_limit)
    assert rc == fa2.FA2_ERR_TIMEOUT
    ok(fa2)
    got = fa2.fa2_fwd_kv4(q, cache, t, ln, one, one, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok(fa2)


@pytest.mark.parametrize("Hq,Hkv,Nq,d", [(8, 2, 1, 128), (8, 2, 700, 64), (16, 1, 16, 128), (32, 8, 300, 128)])
def test_padded_batch_with_idle_requests(gpu_lib, Hq, Hkv, Nq, d):
    """Requests of length 0 and below it: O = 0, LSE = -inf on every row."""
    fa2 = gpu_lib
    rng = np.random.default_rng(65)
    lens, page = [0, 40, -3, 0, 0], 16
    table, P = make_tables(rng, lens, page)
    cache = torch.tensor(make_cache(rng, P, Hkv, page, d)).cuda()
    one = torch.ones(Hkv, device="cuda")
    q = torch.tensor(rng.standard_normal((5, Hq, Nq, d))).to(torch.bfloat16).cuda()
    for sel in ([0, 1, 2, 3, 4], [2], [0, 3]):
        o, lse = torch.full_like(q[sel], 7), torch.full((len(sel), Hq, Nq), 7.0, device="cuda")
        fa2.fa2_fwd_kv4(q[sel], cache, i32(table[sel]), i32(np.array(lens)[sel]), one, one, o, lse)
        ok(fa2)
        for j, b in enumerate(sel):
            if lens[b] <= 0:
                assert not o[j].any() and lse[j].isneginf().all()
            else:
                alone = fa2.fa2_fwd_kv4(q[b: b + 1], cache, i32(table[b: b + 1]), i32(lens[b: b + 1]), one, one)
                assert torch.equal(o[j], alone[0][0]) and torch.equal(lse[j], alone[1][0])


def test_idle_request_of_more_elements_than_32_bits_count(gpu_lib):
    """2^27 + 64 rows of 64: their pieces of four pass 2^31."""
    fa2 = gpu_lib
    Hq, Nq, d, page = 64, 2 ** 21 + 1, 64, 16
    q = torch.zeros((1, Hq, Nq, d), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(q, 7), torch.full((1, Hq, Nq), 7.0, device="cuda")
    cache = torch.zeros(fa2.fa2_kv4_cache_shape(1, 1, page, d), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    fa2.fa2_fwd_kv4(q, cache, i32([[0]]), i32([0]), one, one, o, lse)
    ok(fa2)
    del q
    assert lse.isneginf().all()
    assert all(not part.any() for part in o[0])


@pytest.mark.parametrize("B,Hkv,n,page", [(1, 1, 300011, 128), (1, 2, 40000, 16), (2, 3, 33000, 64)])
@pytest.mark.parametrize("Hq,Nq,d", [(1, 1, 64), (8, 1, 128), (16, 1, 64), (20, 1, 128), (8, 5, 128), (13, 7, 64)])
def test_parts_joined_in_groups(gpu_lib, B, Hkv, n, page, Hq, Nq, d):
    """Contexts so long that a row block has dozens of parts, 292 at most.
    All tokens lie in one page that every table entry names, so that 64 bits are
    quick: the softmax's sums run over its tokens, each counted."""
    fa2 = gpu_lib
    rng = np.random.default_rng(B + n + Hq + Nq + d)
    cache = make_cache(rng, 1, Hkv, page, d)
    lens = [n - 777 * b for b in range(B)]
    table = np.zeros((B, -(-n // page)), np.int64)
    q = torch.tensor(rng.standard_normal((B, Hq * Hkv, Nq, d))).to(torch.bfloat16)
    one = np.ones(Hkv, np.float32)
    args = (q.cuda(), torch.tensor(cache).cuda(), i32(table), i32(lens), torch.tensor(one).cuda(), torch.tensor(one).cuda())
    o, lse = fa2.fa2_fwd_kv4(*args, causal=True)
    again = fa2.fa2_fwd_kv4(*args, causal=True)
    ok(fa2)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    o, lse, qd = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    keys, values = context(cache, np.zeros((1, 1), int), [page], d, one, one)
    for b in range(B):
        for h in range(Hq * Hkv):
            k, v = keys[0][h // Hq], values[0][h // Hq]
            for i in range(Nq):
                m = lens[b] + i + 1 - Nq
                count = m // page + (np.arange(page) < m % page)
                s = d ** -0.5 * (k @ qd[b, h, i])
                w = count * np.exp(s - s.max())
                ref, lref = w @ v / w.sum(), s.max() + math.log(w.sum())
                A = w @ np.abs(v) / w.sum()
                big = d ** -0.5 * (np.abs(k) @ np.abs(qd[b, h, i])).max()
                e = (d + 8) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * abs(lref) + 2.0 ** -21
                r = (m / 8 + 64) * 2.0 ** -23
                bound = (2.0 ** -11 + 2 * e + r) * A + 2.0 ** -32 * m * np.abs(v).max() + U["bf16"] * np.abs(ref)
                assert np.all(np.abs(o[b, h, i] - ref) <= bound)
                assert abs(lse[b, h, i] - lref) <= e + r + 2.0 ** -22 * abs(lref)


@pytest.mark.parametrize("Hq,Nq", [(2, 1), (20, 1), (13, 3)])
def test_longest_table_and_context(gpu_lib, Hq, Nq):
    """Positions just below 2^31, all in one page of equal tokens: O is their
    value, LSE their score and the logarithm of their number. Every weight is 2^7
    up to 2^-21 of it, and fewer than 2^24 of them go into a sum one by one, so
    sums are as good."""
    fa2 = gpu_lib
    page, d, W = 128, 64, 2 ** 24 - 3
    n = W * page - 41
    cache = np.zeros((1, 1, 2, page * (d // 2 + d // 16)), np.uint8)
    cache[..., : page * d // 2] = 0x22                   # 1.0
    cache[..., page * d // 2:] = 0x38                    # 1.0
    q = torch.full((1, Hq, Nq, d), 0.125)
    q[:, ::2] *= -1
    table = torch.zeros((1, W), dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    o, lse = fa2.fa2_fwd_kv4(q.bfloat16().cuda(), torch.tensor(cache).cuda(), table, i32([n]), one, one * 3, scale=0.25,
                             causal=True)
    ok(fa2)
    assert torch.all(o == 3)
    m = n + torch.arange(Nq, dtype=torch.float64) + 1 - Nq
    want = m.log() + torch.where(torch.arange(Hq) % 2 == 0, -2.0, 2.0).double()[:, None]
    assert (lse[0].double().cpu() - want).abs().max() <= 8 * 2.0 ** -23 * 24


def test_table_rows_of_millions_of_pages(gpu_lib):
    """The second row of a table lies 64 MB behind the first; a table that would
    need more tiles than are counted is refused."""
    fa2 = gpu_lib
    rng = np.random.default_rng(66)
    page, d, W, lens = 128, 128, 2 ** 24 - 3, [300, 170]
    small, P = make_tables(rng, lens, page)
    table = torch.full((2, W), -1, dtype=torch.int32, device="cuda")
    table[:, : small.shape[1]] = i32(small)
    for Hkv, G in ((4, 1), (2, 20)):
        cache = torch.tensor(make_cache(rng, P, Hkv, page, d)).cuda()
        one = torch.ones(Hkv, device="cuda")
        q = torch.tensor(rng.standard_normal((2, Hkv * G, 1, d))).to(torch.bfloat16).cuda()
        a = fa2.fa2_fwd_kv4(q, cache, table, i32(lens), one, one)
        b = fa2.fa2_fwd_kv4(q, cache, i32(small), i32(lens), one, one)
        ok(fa2)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ka, kb = (fa2.fa2_kv4_gather(cache, t, i32(lens), one, one, 300, d)[0] for t in (table, i32(small)))
        assert torch.equal(ka, kb)
    many = torch.zeros(fa2.fa2_kv4_cache_shape(1, 32, page, d), dtype=torch.uint8, device="cuda")
    with pytest.raises(fa2.FA2Error):
        fa2.fa2_fwd_kv4(torch.zeros(2, 32, 1, d, dtype=torch.bfloat16, device="cuda"), many, table, i32(lens),
                        torch.ones(32, device="cuda"), torch.ones(32, device="cuda"))
