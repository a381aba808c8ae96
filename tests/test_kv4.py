"""The paged 4-bit KV cache on the host: argument checks before any device is
touched, refusals of the torch binding, and the oracle's own pins (CPU only)."""
import math

import numpy as np
import pytest
import torch

from attention_fa2_forward_03_gb300 import build, fa2
from oracle import kv4

A = 1 << 20  # a 16-byte aligned fake address: never dereferenced on these paths
BAD, UNS = 1, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa2.load()


def swap(args, i, x):
    out = list(args)
    out[i] = x
    return out


PLAN = [A] * 9 + [4, 8, 10, 64, 100]   # ..., B, N, max_pages, page_size, num_pages


@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in range(9)], *[(j, A + 2, BAD) for j in range(9)],
    (9, 0, BAD), (10, 0, BAD), (11, 0, BAD), (12, 0, BAD), (13, -1, BAD),
    (12, 48, UNS), (12, 256, UNS), (12, 8, UNS), (13, 1 << 26, UNS), (11, 1 << 26, UNS), (9, 1 << 29, UNS),
])
def test_plan_host_validation(i, x, want):
    assert fa2.fa2_kv4_plan_ptr(*swap(PLAN, i, x)) == want


APPEND = [A] * 6 + [2, 8, 5, 128, (8, 8, 8), (0, 1024, 128), 64, 100, 0]


@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in range(6)], (0, A + 8, BAD), (1, A + 8, BAD), (3, A + 8, BAD), (2, A + 2, BAD),
    (4, A + 2, BAD), (5, A + 1, BAD), (6, 0, BAD), (7, -1, BAD), (8, 0, BAD), (9, 0, BAD),
    (10, (8, 8, 4), BAD), (11, (-8, 8, 8), BAD), (12, 0, BAD), (13, 0, BAD), (14, 3, BAD),
    (9, 96, UNS), (9, 256, UNS), (12, 24, UNS), (13, 1 << 25, UNS), (8, 1 << 30, UNS),
])
def test_append_host_validation(i, x, want):
    assert fa2.fa2_kv4_append_ptr(*swap(APPEND, i, x)) == want


GATHER = [A] * 8 + [2, 8, 5, 64, 10, 32, 100, 1]


@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in (0, 1, 2, 4, 5, 6, 7)], (0, A + 8, BAD), (6, A + 8, BAD), (7, A + 8, BAD), (1, A + 2, BAD),
    (2, A + 2, BAD), (3, A + 2, BAD), (4, A + 2, BAD), (8, 0, BAD), (9, 0, BAD), (10, 0, BAD), (11, -64, BAD),
    (12, 0, BAD), (13, 0, BAD), (14, 0, BAD), (15, 2, BAD), (11, 80, UNS), (13, 1, UNS), (10, 1 << 30, UNS),
])
def test_gather_host_validation(i, x, want):
    assert fa2.fa2_kv4_gather_ptr(*swap(GATHER, i, x)) == want


FWD = [A] * 9 + [1 << 40, 2, 32, 8, 1, 128, 99, 64, 100, 0.1, 0, 0]


@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in range(9)], *[(j, A + 8, BAD) for j in (0, 1, 6, 7, 8)],
    *[(j, A + 2, BAD) for j in (2, 3, 4, 5)],
    (9, 100, BAD), (9, -1, BAD), (10, 0, BAD), (11, 0, BAD), (11, 20, BAD), (12, 0, BAD), (13, 0, BAD), (14, 0, BAD),
    (15, 0, BAD), (16, 0, BAD), (17, 0, BAD), (18, 0.0, BAD), (18, float("nan"), BAD), (18, float("inf"), BAD),
    (19, 2, BAD), (20, 9, BAD), (14, 96, UNS), (16, 20, UNS), (17, 1 << 25, UNS), (15, 1 << 25, UNS),
    (13, 1 << 26, UNS),
])
def test_forward_host_validation(i, x, want):
    assert fa2.fa2_fwd_kv4_ptr(*swap(FWD, i, x)) == want


def test_workspace_is_checked_exactly():
    for Hq, Hkv, Nq, d in ((32, 8, 1, 128), (32, 8, 5, 128), (8, 1, 2, 64), (16, 16, 700, 64)):
        n = fa2.fa2_fwd_kv4_workspace(2, Hq, Hkv, Nq, d, 99, 64)
        args = FWD[:]
        args[9:15] = [n - 1, 2, Hq, Hkv, Nq, d]
        assert n > 0 and fa2.fa2_fwd_kv4_ptr(*args) == BAD
    # short sequences are never split: no workspace, and none is asked for
    assert fa2.fa2_fwd_kv4_workspace(2, 32, 8, 1, 128, 36, 64) == 0 < fa2.fa2_fwd_kv4_workspace(2, 32, 8, 1, 128, 37, 64)
    assert fa2.fa2_fwd_kv4_workspace(32, 32, 8, 1, 128, 36, 64) == 0 < fa2.fa2_fwd_kv4_workspace(33, 32, 8, 1, 128, 36, 64)
    for bad in ((2, 0, 8, 1, 128, 10, 64), (2, 32, 0, 1, 128, 10, 64), (2, 32, 5, 1, 128, 10, 64),
                (2, 32, 8, 0, 128, 10, 64), (2, 32, 8, 1, 96, 10, 64), (0, 32, 8, 1, 128, 10, 64),
                (2, 32, 8, 1, 128, 0, 64), (2, 32, 8, 1, 128, 10, 48)):
        assert fa2.fa2_fwd_kv4_workspace(*bad) == -1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    cache = torch.zeros(fa2.fa2_kv4_cache_shape(4, 2, 16, 64), dtype=torch.uint8)
    ds = torch.ones(2)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    slots = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa2.fa2_fwd_kv4(q, cache, table, lens, ds, ds)
    with pytest.raises(ValueError):
        fa2.fa2_fwd_kv4(q[0], cache, table, lens, ds, ds)
    with pytest.raises(ValueError):
        fa2.fa2_kv4_append(k, k, slots, cache, ds, ds)
    with pytest.raises(ValueError):
        fa2.fa2_kv4_append(k, k[:, :1], slots, cache, ds, ds)
    with pytest.raises(ValueError):
        fa2.fa2_kv4_gather(cache, table, lens, ds, ds, 3, 64)
    with pytest.raises(ValueError):
        fa2.fa2_kv4_plan(lens, lens, table, lens, torch.zeros(2, dtype=torch.int32), 16, 3)


# ------------------------------------------------------------------ the oracle's pins

def test_e4m3_table_matches_torch():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv4.E4M3, want, equal_nan=True)


def test_every_product_of_code_and_scale_is_exact_in_fp16():
    p = kv4.E2M1[:8, None] * kv4.E4M3[None, :127]
    assert np.array_equal(p, p.astype(np.float16).astype(np.float64))


def test_oracle_rounding_by_hand():
    x = np.zeros((2, 16))
    x[0, :9] = [6.0, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 0.26]
    x[1, :2] = [6.0 * 1.0625, 3.0]      # scale between 1 and 1.125: 1; 3 is a code
    want = np.zeros((2, 16))
    want[0, :9] = [6.0, 0.0, 1.0, -1.0, 2.0, 2.0, -4.0, 4.0, 0.5]
    want[1, :2] = [6.0, 3.0]
    assert np.array_equal(kv4.rounded(x, 1.0), want)
    y = torch.rand(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(2)) * 500
    assert np.array_equal(kv4.E4M3[kv4.nearest(kv4.E4M3[:127], y.numpy())],
                          y.float().clamp(max=448).to(torch.float8_e4m3fn).double().numpy())


def test_oracle_layout_by_hand():
    """One page of 16, one head, d = 64: element 5 of token 3 has code 0b1110 (-4) and scale byte 0x40 (2)."""
    c = np.zeros((1, 1, 2, 16 * 36), np.uint8)
    c[0, 0, 1, 3 * 32 + 2] = 0xE0
    c[0, 0, 1, 16 * 32 + 3 * 4 + 0] = 0x40
    v = kv4.tokens(c, 64, [0], 4, 0, 1, 0.25)
    assert v[3, 5] == -2.0 and np.count_nonzero(v) == 1
    assert not kv4.tokens(c, 64, [0], 4, 0, 0, 0.25).any()


def test_oracle_attention_against_torch():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((1, 4, 3, 64), (1, 2, 9, 64), (1, 2, 9, 64)))
    o, lse, _, _ = kv4.attention(q.numpy(), [k[0].numpy()], [v[0].numpy()], 0.125, True, [9])
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    mask = torch.arange(9) >= torch.arange(3)[:, None] + 7
    s = (q @ kk.transpose(2, 3) * 0.125).masked_fill(mask, -math.inf)
    assert np.allclose(o, (torch.softmax(s, -1) @ vv).numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-12)


def test_oracle_plan_by_hand():
    table = np.full((3, 3), -1)
    table[1, 0], table[2, 0] = 7, 5
    ring = np.array([9, 8, 4, 0, 0, 0, 0, 0, 0, 0])
    lens, acc, slots, state, t2, r2 = kv4.plan([0, 10, 16], [20, -1, 1], table, ring, [0, 3], 16, 20)
    assert lens == [20, 0, 17] and acc == [20, 0, 1] and state == [3, 1]
    assert list(t2[0]) == [9, 8, -1] and list(t2[2]) == [5, 4, -1] and r2[3] == 7
    assert list(slots[0, :17]) == list(range(144, 160)) + [128] and slots[2, 0] == 64 and (slots[1] == -1).all()
