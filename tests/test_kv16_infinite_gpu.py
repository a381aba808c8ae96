"""Attention over the paged 16-bit KV cache where keys and values are infinite or
NaN, against the same formula in fp64 over the keys that each row sees: an
infinite value comes out as that infinity, wherever its token lies in the chunk and
however the prompt was cut into chunks.

The inputs are normal and the scale d^-0.5, so scores lie within some ten of one
another and no weight rounds to zero in 16 bits. Finite elements within the
bounds of test_kv16_gpu.py, whose terms are made from the finite keys and values.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}
INF, NAN = math.inf, math.nan


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Prompt:
    """One request of L tokens, all its queries, keys and values; pages in no order."""

    def __init__(self, seed, L, Hq, Hkv, d, page, dtype):
        rng = np.random.default_rng(seed)
        self.L, self.G, self.d, self.page, self.dtype = L, Hq // Hkv, d, page, dtype
        self.q, self.k, self.v = (torch.tensor(rng.standard_normal((L, h, d))).to(DT[dtype]) for h in (Hq, Hkv, Hkv))
        self.ids = rng.permutation(-(-L // page))

    def run(self, fa2, chunks):
        """The last sum(chunks) tokens in calls of these sizes: o, lse of those rows."""
        P, H = len(self.ids), self.k.shape[1]
        rows = torch.full((P * self.page, 2, H, self.d), NAN, dtype=DT[self.dtype])   # in the request's order
        rows[: self.L, 0], rows[: self.L, 1] = self.k, self.v
        cache = torch.empty(P, H, 2, self.page, self.d, dtype=DT[self.dtype])
        cache[torch.tensor(self.ids)] = rows.view(P, self.page, 2, H, self.d).permute(0, 3, 2, 1, 4)
        cache, table = cache.cuda(), i32(self.ids[None])
        at, out = self.L - sum(chunks), []
        for n in chunks:
            out.append(fa2.fa2_fwd_kv16(self.q[at: at + n].cuda(), cache, table, i32([at + n]), i32([0]), i32([n]), causal=True))
            at += n
        assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_OK
        return tuple(torch.cat([x[i] for x in out]).double().cpu().numpy() for i in (0, 1))

    def check(self, o, lse, n):
        """o, lse of the last n tokens."""
        q, k, v = (x.double().numpy() for x in (self.q, self.k, self.v))
        u, scale = U[self.dtype], self.d ** -0.5
        kf, vf = (np.where(np.isfinite(x), x, 0.0) for x in (k, v))
        for i in range(n):
            seen = self.L - n + 1 + i
            for h in range(q.shape[1]):
                x = q[seen - 1, h]
                with np.errstate(invalid="ignore"):
                    s = scale * (k[:seen, h // self.G] @ x)
                    p = np.exp(s - s.max())
                    want, z = p @ v[:seen, h // self.G] / p.sum(), s.max() + np.log(p.sum())
                got, lgot = o[i, h], lse[i, h]
                if np.isneginf(s).all():   # as a row without a key
                    assert not got.any() and np.isneginf(lgot), (i, h)
                    continue
                assert np.array_equal(np.isnan(got), np.isnan(want)), (i, h)
                assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want)), (i, h)
                assert np.isnan(lgot) == np.isnan(z), (i, h)
                if np.isnan(z):
                    continue
                big = scale * (np.abs(kf[:seen, h // self.G]) @ np.abs(x)).max()
                e = (self.d + 8) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * abs(z) + 2.0 ** -21
                r = (seen / 8 + 64) * 2.0 ** -23
                A = p @ np.abs(vf[:seen, h // self.G]) / p.sum()
                f = np.isfinite(want)
                bound = (u + 2 * e + r) * A + SUB[self.dtype] * (seen * np.abs(vf).max() + 1) + u * np.abs(np.where(f, want, 0))
                assert np.all(np.abs(got[f] - want[f]) <= bound[f]), (i, h)
                assert abs(lgot - z) <= e + r + 2.0 ** -22 * abs(z), (i, h)


# tokens, how many of them are new, query heads, KV heads, d, page, dtype
SHAPES = [
    (300, 300, 2, 1, 128, 16, "fp16"), (300, 70, 8, 2, 128, 64, "bf16"), (413, 200, 4, 2, 64, 32, "bf16"), (129, 5, 8, 1, 128, 128, "bf16"),
    (140, 40, 8, 2, 64, 16, "fp16"),
]


def places(L, n):
    """In front of the new tokens' first tile, in it, in the middle, at the end."""
    return sorted({0, max(L - n - 130, 0), max(L - n - 1, 0), L - n + 1, L - n // 2, L - 1})


@pytest.mark.parametrize("L,n,Hq,Hkv,d,page,dtype", SHAPES)
@pytest.mark.parametrize("value", [INF, -INF])
def test_infinite_values(gpu_lib, L, n, Hq, Hkv, d, page, dtype, value):
    """A column for each place, one with the same infinity twice, one with both, one with a NaN behind an infinity."""
    s = Prompt(1 + L + d, L, Hq, Hkv, d, page, dtype)
    at = places(L, n)
    for i, pos in enumerate(at):
        s.v[pos, i % Hkv, 3 * i] = value
    s.v[at[0], 0, d - 1] = s.v[at[-2], 0, d - 1] = value
    s.v[at[-3], 0, d - 2], s.v[at[-1], 0, d - 2] = value, -value
    s.v[at[-3], 0, d - 3], s.v[at[-1], 0, d - 3] = value, NAN
    s.check(*s.run(gpu_lib, [n]), n)


@pytest.mark.parametrize("L,n,Hq,Hkv,d,page,dtype", SHAPES)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_infinite_keys(gpu_lib, L, n, Hq, Hkv, d, page, dtype, value):
    """A score of -inf is no weight (and a row with no others one without a key),
    one of +inf or NaN is a row of NaN, and rows that do not see the key have neither."""
    for pos in places(L, n):
        s = Prompt(2 + L + d, L, Hq, Hkv, d, page, dtype)
        s.k[pos, Hkv - 1, 7] = value
        s.check(*s.run(gpu_lib, [n]), n)


@pytest.mark.parametrize("chunks", [[260], [1, 259], [130, 130], [64, 1, 195], [3, 200, 57]])
def test_chunks_make_no_difference_to_what_is_infinite(gpu_lib, chunks):
    s = Prompt(5, 500, 8, 2, 128, 16, "bf16")
    for i, pos in enumerate((10, 239, 240, 300, 383, 384, 430, 499)):
        s.v[pos, i % 2, 5 * i] = INF if i % 3 else -INF
    s.check(*s.run(gpu_lib, chunks), 260)


@pytest.mark.parametrize("d,page,dtype", [(128, 64, "bf16"), (64, 16, "fp16")])
def test_infinite_values_of_a_long_context(gpu_lib, d, page, dtype):
    """The rows are split over many CTAs and joined."""
    s = Prompt(6 + d, 9000, 4, 1, d, page, dtype)
    for i, pos in enumerate((100, 4500, 8975, 8985, 8999)):
        s.v[pos, 0, 3 * i] = -INF if i % 2 else INF
    s.v[200, 0, d - 1], s.v[8990, 0, d - 1] = INF, -INF
    s.check(*s.run(gpu_lib, [30]), 30)
