"""Rotary positions and the paged 16-bit KV cache on the host: argument checks
before any device is touched, refusals of the torch binding, and the oracle's
own pins (CPU only)."""
import math

import numpy as np
import pytest
import torch

from attention_fa2_forward_03_gb300 import build, fa2
from oracle import kv16

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


def strides(i, x, n=12):
    s = [64 * (j + 1) for j in range(n)]
    s[i] = x
    return s


# q, k, q_out, k_out, positions, inv_freq, axes, B, H_q, H_kv, N, d, rot_dim, n_axes, interleaved, strides, dtype
ROPE = [A] * 7 + [2, 8, 4, 5, 128, 128, 3, 0, strides(0, 64), 0]


@pytest.mark.parametrize("call", ["fa2_rope_ptr", "fa2_rope_bwd_ptr"])
@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in (0, 1, 2, 3, 4, 5)], *[(j, A + 8, BAD) for j in (0, 1, 2, 3)], *[(j, A + 2, BAD) for j in (4, 5, 6)],
    (7, 0, BAD), (8, 0, BAD), (9, 0, BAD), (9, -1, BAD), (10, 0, BAD), (11, 0, BAD), (12, 0, BAD), (12, -16, BAD), (13, 0, BAD),
    (14, 2, BAD), (15, strides(3, 4), BAD), (15, strides(0, -8), BAD), (15, strides(6, 0), BAD), (15, strides(10, 0), BAD), (16, 2, BAD),
    (11, 96, UNS), (11, 256, UNS), (12, 144, UNS), (12, 24, UNS), (13, 9, UNS), (10, 1 << 30, UNS), (7, 1 << 30, UNS),
    (15, strides(2, 1 << 31), UNS), (8, 1 << 25, UNS),
])
def test_rope_host_validation(call, i, x, want):
    assert getattr(fa2, call)(*swap(ROPE, i, x)) == want


def test_rope_without_k_does_not_read_its_strides():
    args = swap(swap(swap(ROPE, 1, 0), 3, 0), 9, 0)
    s = [3 if (j // 3) % 2 else 64 for j in range(12)]
    assert fa2.fa2_rope_ptr(*swap(swap(args, 15, s), 12, 24)) == UNS       # past the strides, to the sizes
    assert fa2.fa2_rope_ptr(*swap(args, 15, [7] * 12)) == BAD
    with pytest.raises(ValueError):
        fa2.fa2_rope_ptr(*swap(ROPE, 15, [64] * 11))


# q, k, v, slots, positions, inv_freq, axes, cache, q_out, T, H_q, H_kv, d, rot_dim, n_axes, interleaved, strides, page_size, num_pages, dtype
APPEND = [A] * 9 + [5, 8, 4, 128, 64, 1, 0, strides(0, 64, 6), 64, 100, 1]


@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in (0, 1, 2, 3, 5, 7, 8)], (4, 0, BAD), *[(j, A + 8, BAD) for j in (0, 1, 2, 7, 8)],
    *[(j, A + 2, BAD) for j in (3, 4, 5, 6)], (9, 0, BAD), (10, 0, BAD), (11, 0, BAD), (12, 0, BAD), (13, 0, BAD), (14, 0, BAD), (15, 2, BAD),
    (16, strides(2, 4, 6), BAD), (16, strides(5, -8, 6), BAD), (17, 0, BAD), (18, 0, BAD), (19, 5, BAD),
    (12, 96, UNS), (13, 40, UNS), (14, 9, UNS), (16, strides(1, 1 << 31, 6), UNS), (17, 48, UNS), (18, 1 << 26, UNS), (9, (1 << 31) - 1, UNS),
    (11, 1 << 24, UNS),
])
def test_append_host_validation(i, x, want):
    assert fa2.fa2_kv16_append_ptr(*swap(APPEND, i, x)) == want


def test_append_without_positions_or_q():
    plain = [0, A, A, A, 0, 0, 0, A, 0, 5, 0, 4, 128, 0, 0, 0, strides(0, 3, 6), 64, 100, 1]   # q's strides are not read
    assert fa2.fa2_kv16_append_ptr(*swap(plain, 12, 96)) == UNS            # all else is accepted
    assert fa2.fa2_kv16_append_ptr(*swap(plain, 13, 64)) == BAD            # nothing says by how much to rotate
    assert fa2.fa2_kv16_append_ptr(*swap(plain, 10, 8)) == BAD             # heads without q
    assert fa2.fa2_kv16_append_ptr(*swap(plain, 19, 2)) == BAD


# q, cache, block_table, seq_lens, q_starts, q_lens, o, lse, workspace, workspace_bytes, T, B, H_q, H_kv, d, stride_t, stride_h,
# max_pages, page_size, num_pages, scale, causal, dtype
FWD = [A] * 9 + [1 << 40, 50, 4, 32, 8, 128, 4096, 128, 99, 64, 100, 0.1, 1, 0]


@pytest.mark.parametrize("i,x,want", [
    *[(j, 0, BAD) for j in range(9)], *[(j, A + 8, BAD) for j in (0, 1, 6, 7, 8)], *[(j, A + 2, BAD) for j in (2, 3, 4, 5)],
    (9, 100, BAD), (9, -1, BAD), (10, 0, BAD), (11, 0, BAD), (12, 0, BAD), (12, 30, BAD), (13, 0, BAD), (14, 0, BAD), (15, 0, BAD), (15, 12, BAD),
    (16, -128, BAD), (16, 4, BAD), (17, 0, BAD), (18, 0, BAD), (19, 0, BAD), (20, 0.0, BAD), (20, math.nan, BAD), (20, math.inf, BAD), (21, 2, BAD),
    (22, 9, BAD), (14, 96, UNS), (18, 20, UNS), (19, 1 << 25, UNS), (17, 1 << 25, UNS), (10, 1 << 26, UNS), (15, 1 << 32, UNS), (12, 8 * 129, UNS),
    (13, 1 << 20, BAD),
])
def test_forward_host_validation(i, x, want):
    assert fa2.fa2_fwd_kv16_ptr(*swap(FWD, i, x)) == want


def test_workspace_is_checked_exactly():
    sizes = (50, 4, 32, 8, 128, 99, 64)
    need = fa2.fa2_fwd_kv16_workspace(*sizes)
    assert need > 0 and need % 16 == 0
    assert fa2.fa2_fwd_kv16_ptr(*swap(FWD, 9, need - 1)) == BAD


@pytest.mark.parametrize("T,B,H_q,H_kv,d,max_pages,page", [
    (0, 4, 32, 8, 128, 99, 64), (50, 0, 32, 8, 128, 99, 64), (50, 4, 30, 8, 128, 99, 64), (50, 4, 32, 8, 96, 99, 64), (50, 4, 32, 8, 128, 0, 64),
    (50, 4, 32, 8, 128, 99, 48), (1 << 26, 4, 32, 8, 128, 99, 64), (50, 4, 256, 1, 128, 99, 64), (1 << 20, 1 << 20, 64, 64, 64, 1 << 18, 128),
    (50, 2 ** 31 - 1, 32, 8, 128, 99, 64),
])
def test_workspace_says_no_to_what_the_call_refuses(T, B, H_q, H_kv, d, max_pages, page):
    assert fa2.fa2_fwd_kv16_workspace(T, B, H_q, H_kv, d, max_pages, page) == -1
    args = list(FWD)
    args[10:15], args[17], args[18] = [T, B, H_q, H_kv, d], max_pages, page
    assert fa2.fa2_fwd_kv16_ptr(*args) in (BAD, UNS)


def test_tensors_off_the_gpu_are_refused():
    q, k = torch.zeros(1, 4, 5, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16)
    pos, f = torch.zeros(1, 5, dtype=torch.int32), torch.zeros(32)
    for call in (fa2.fa2_rope, fa2.fa2_rope_bwd):
        with pytest.raises(ValueError):
            call(q, k, pos, f)
        with pytest.raises(TypeError):
            call(None, k, pos, f)
    cache = torch.zeros(fa2.fa2_kv16_cache_shape(3, 2, 16, 64), dtype=torch.bfloat16)
    t, i = torch.zeros(5, 2, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa2.fa2_kv16_append(t, t, i, cache)
    with pytest.raises(ValueError):
        fa2.fa2_fwd_kv16(t, cache, i[None], i[:1], i[:1], i[:1])


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("inter", [False, True])
def test_oracle_rotation_is_a_complex_product(inter):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 7, 10))
    pos, f, axes = rng.integers(-50, 50, (2, 3, 7)), rng.random(4).astype(np.float32), np.array([0, 1, 1, 0])
    y = kv16.rotate(x, pos, f, axes, inter)
    pairs = (lambda t: t[..., 0:8:2] + 1j * t[..., 1:8:2]) if inter else (lambda t: t[..., :4] + 1j * t[..., 4:8])
    angle = np.moveaxis(pos[axes], 0, -1) * f.astype(float)
    assert np.allclose(pairs(y), pairs(x) * np.exp(1j * angle), rtol=0, atol=1e-12)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(kv16.rotate(y, pos, f, axes, inter, inverse=True), x, rtol=0, atol=1e-12)


def test_oracle_rotation_at_far_positions():
    """2^31 - 1 times a frequency of 24 bits does not fit 53: against integers."""
    from fractions import Fraction

    f = np.array([0.7391], np.float32)
    n = 2 ** 31 - 1
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    angle = Fraction(float(f[0])) * n
    angle = float(angle - int(angle / (2 * pi)) * 2 * pi)
    y = kv16.rotate(np.array([[1.0, 0.0]]), np.array([[n]]), f)
    assert abs(y[0, 0] - math.cos(angle)) < 1e-8 and abs(y[0, 1] - math.sin(angle)) < 1e-8


def test_oracle_attention_against_a_loop():
    rng = np.random.default_rng(1)
    n, Hq, H, L, d = 4, 4, 2, 6, 3
    q, k, v = rng.standard_normal((n, Hq, d)), rng.standard_normal((H, L, d)), rng.standard_normal((H, L, d))
    for causal in (False, True):
        o, lse, _, _ = kv16.attention(q, k, v, 0.5, causal)
        for i in range(n):
            for h in range(Hq):
                m = L - n + 1 + i if causal else L
                s = [0.5 * sum(q[i, h, e] * k[h // 2, j, e] for e in range(d)) for j in range(m)]
                z = sum(math.exp(t) for t in s)
                assert abs(lse[i, h] - math.log(z)) < 1e-12
                assert np.allclose(o[i, h], sum(math.exp(s[j]) / z * v[h // 2, j] for j in range(m)))
    o, lse, _, _ = kv16.attention(q, k[:, :2], v[:, :2], 0.5, True)   # two rows without a key
    assert np.isneginf(lse[:2]).all() and not o[:2].any() and np.isfinite(lse[2:]).all()
