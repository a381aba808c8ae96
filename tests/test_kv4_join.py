"""How the attention over the 4-bit KV cache joins the partial results of
contexts that several CTAs share: which counter each of them counts on (CPU, by
the kernel's own Split), and results of lines that are not padded, where one
CTA ends a segment and begins the next (GPU)."""
import math
import os
import random
import subprocess

import numpy as np
import pytest
import torch

from attention_fa2_forward_03_gb300 import build
from oracle import kv4

# Reads "ctas c0 c1" a line; writes, for each CTA of the segment, the counters
# on which it may count: level, word, the count at which all are there, and the
# group's first CTA.
PROGRAM = r"""
#include <cstdio>
#include "fa2_kv4_sm103.cuh"
int main() {
    int ctas, c0, c1;
    while (std::scanf("%d %d %d", &ctas, &c0, &c1) == 3) {
        for (int c = c0; c <= c1; ++c) {
            const fa2::kv4::Split s(c0, c1, c);
            for (int level = s.begins(); level < 2; ++level)
                std::printf("%d %d %d %d ", level, s.word(level, ctas), s.count(level), level ? c0 : s.first);
            std::printf(";");
        }
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    """[(ctas, c0, c1)] -> for each, for each of its CTAs, [(level, word, count, group)]."""
    at = tmp_path_factory.mktemp("split")
    src, exe = str(at / "split.cu"), str(at / "split")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-o", exe, src], check=True)

    def run(segments):
        text = subprocess.run([exe], input="".join("%d %d %d\n" % s for s in segments), capture_output=True, text=True,
                              check=True).stdout
        out = []
        for line in text.splitlines():
            ctas = [[int(x) for x in c.split()] for c in line.split(";")[:-1]]
            out.append([[tuple(c[i: i + 4]) for i in range(0, len(c), 4)] for c in ctas])
        return out

    return run


def line(lens, hrs, ctas, tile, warps):
    """The segments of a launch that more than one CTA shares, [(c0, c1)], as
    `locate` cuts the line of tiles (32 or 128 tokens, by 8 or 1) into runs."""
    least, spare = 32 // (tile // 32), 40 // (tile // 32)
    tiles = [-(-n // tile) for n in lens]
    total = sum(tiles) * hrs
    per = max(-(-total // ctas), least)
    per = -(-per // warps) * warps
    pad = 1
    if len(lens) * hrs <= ctas:
        if max(tiles) <= per + spare:
            per = max(per, -(-max(tiles) // warps) * warps)
        if sum(-(-t // per) for t in tiles) * hrs <= ctas:
            pad = per
    out, at = [], 0
    for t in tiles:
        for _ in range(hrs if t else 0):
            end = at + -(-t // pad) * pad
            if (end - 1) // per > at // per:
                out.append((at // per, (end - 1) // per))
            at = end
    return out, pad


# 152 SMs: a CTA an SM for 9 to 24 rows a head, two otherwise.
KERNELS = [(304, 32, 8), (152, 32, 8), (304, 128, 1)]   # CTAs, tokens of a tile, warps that share a run


def shared_counters(split, launches):
    """Of launches [(ctas, [(c0, c1)])]: those in which two groups count on one word."""
    flat = [(ctas, c0, c1) for ctas, segments in launches for c0, c1 in segments]
    got, at, bad = split(flat), 0, []
    for ctas, segments in launches:
        words = {}
        for c0, c1 in segments:
            per_cta, at = got[at], at + 1
            members = {}
            for cta, levels in zip(range(c0, c1 + 1), per_cta):
                assert levels[-1][0] == 1
                for level, word, count, group in levels:
                    assert 0 <= word < 2 * ctas
                    words.setdefault(word, set()).add((c0, level, group))
                    if level == 0:
                        members.setdefault((level, word, count), set()).add(cta)
            # a level-0 counter is counted on by as many CTAs as it waits for,
            # and level 1 by one CTA of each group and all that begin there
            for (_, _, count), ctas_in in members.items():
                assert len(ctas_in) == count
            tops = {levels[-1][1:3] for levels in per_cta}
            assert len(tops) == 1
            assert tops.pop()[1] == len(members) + sum(len(levels) == 1 for levels in per_cta)
        bad += [(ctas, segments, w, g) for w, g in words.items() if len(g) > 1]
    return bad


def test_every_pair_of_neighbouring_segments(split):
    """Segments of every number of parts, the second begun by the CTA that ends the first."""
    launches = [(304, [(0, a), (a, a + b)]) for a in range(1, 152) for b in (1, 11, 12, 13, 30, 151)]
    assert not shared_counters(split, launches)


@pytest.mark.parametrize("ctas,tile,warps", KERNELS)
def test_no_two_groups_of_a_launch_share_a_counter(split, ctas, tile, warps):
    rng = random.Random(ctas + tile)
    launches, unpadded = [], 0
    while len(launches) < 3000:
        B, hrs = (int(2 ** rng.uniform(0, top)) for top in (6, 4))
        top = int(2 ** rng.uniform(10, 17))
        lens = [top] + [rng.randint(0 if rng.random() < 0.1 else top // 3, top) for _ in range(B - 1)]
        segments, pad = line(lens, hrs, ctas, tile, warps)
        unpadded += pad == 1 and any(b - a > 11 for a, b in segments)
        launches.append((ctas, segments))
    assert unpadded > 100   # lines with segments of more parts than are joined at once
    # equal and ragged requests of neighbouring parts 13, 21, 31, ...
    for lens, hrs in (([131072] * 6, 4), ([131072] * 3, 8), ([65536, 48435, 55679, 25679], 8)):
        launches.append((ctas, line(lens, hrs, ctas, tile, warps)[0]))
    assert not shared_counters(split, launches)


# ------------------------------------------------------------------ on the GPU

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
RAGGED = [65536, 48435, 55679, 25679]
# lens, KV heads, query rows a KV head as (heads, tokens), d, dtype. One token or
# a few; 8, 20, 32 or 40 rows. With 152 SMs these lines are not padded.
LINES = [
    (RAGGED, 8, (8, 1), 128, "bf16"), (RAGGED, 8, (8, 5), 128, "bf16"), (RAGGED, 8, (4, 5), 128, "fp16"),
    ([131072] * 6, 4, (8, 1), 64, "fp16"), ([131072] * 3, 8, (8, 1), 128, "bf16"), ([131072] * 3, 8, (32, 1), 64, "bf16"),
    ([131072] * 6, 4, (8, 8), 128, "fp16"), ([131072, 0, 99000, 131072, 127, 70001], 3, (20, 1), 128, "bf16"),
]


def in_one_page(fa2, lens, Hkv, rows, d, dtype, page=64):
    """A call whose tokens all lie in one page that every table entry names,
    so that 64 bits are quick; and (O, LSE, their bounds) in 64 bits. The bounds are
    those of tests/test_kv4_gpu.py: each token of the page counts as often as
    it is seen."""
    G, Nq = rows
    rng = np.random.default_rng(sum(lens) + Hkv + G + Nq + d)
    cache = rng.integers(0, 256, (1, Hkv, 2, page * (d // 2 + d // 16)), dtype=np.uint8)
    cache[..., page * d // 2:] = rng.integers(0x28, 0x48, (1, Hkv, 2, page * d // 16), dtype=np.uint8)   # 0.25 .. 3.75
    q = torch.tensor(rng.standard_normal((len(lens), G * Hkv, Nq, d))).to(DT[dtype])
    table = torch.zeros((len(lens), -(-max(lens) // page)), dtype=torch.int32, device="cuda")
    one = torch.ones(Hkv, device="cuda")
    args = (q.cuda(), torch.tensor(cache).cuda(), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), one, one)

    k, v = (np.stack([kv4.tokens(cache, d, [0], page, h, part, 1.0) for h in range(Hkv)]) for part in (0, 1))
    k, v = (np.repeat(x, G, 0)[None, :, None] for x in (k, v))                       # [1, Hq, 1, page, d]
    n = np.array(lens)[:, None, None]
    m = np.maximum(n + np.arange(Nq) + 1 - Nq, 0)                                    # tokens that a row sees
    seen = m[..., None] // page + (np.arange(page) < m[..., None] % page)            # [B, 1, Nq, page]
    qd = q.double().numpy()[..., None, :]
    s = d ** -0.5 * (k * qd).sum(-1)
    top = np.where(seen > 0, s, -np.inf).max(-1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    w = seen * np.exp(np.where(seen > 0, s - top, 0.0))
    z = w.sum(-1)
    some = z > 0
    w = w / np.where(some, z, 1)[..., None]
    ref, A = (np.einsum("bhnp,bhnpd->bhnd", w, np.broadcast_to(x, (*w.shape, d))) for x in (v, np.abs(v)))
    lref = np.where(some, top[..., 0] + np.log(np.where(some, z, 1)), -np.inf)
    big = d ** -0.5 * (np.abs(k) * np.abs(qd)).sum(-1).max(-1)
    e = (d + 8) * 2.0 ** -23 * big + 4 * 2.0 ** -23 * np.abs(np.where(some, lref, 0)) + 2.0 ** -21
    r = (m / 8 + 64) * 2.0 ** -23
    bound = (2.0 ** -11 + 2 * e + r)[..., None] * A + (2.0 ** -32 * m * np.abs(v).max())[..., None] + U[dtype] * np.abs(ref)
    # fp16 results below 2^-14 are multiples of 2^-24
    bound = bound + (2.0 ** -25 if dtype == "fp16" else 0.0)
    return args, (ref, lref, bound, e + r + 2.0 ** -22 * np.abs(np.where(some, lref, 0)))


def check(o, lse, want):
    ref, lref, bound, lbound = want
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    some = np.isfinite(lref)
    assert np.array_equal(np.isneginf(lse), ~some) and not o[~some].any()
    assert np.all(np.abs(o - ref) <= bound)
    assert np.all(np.abs(lse[some] - lref[some]) <= lbound[some])


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hkv,rows,d,dtype", LINES)
def test_lines_that_are_not_padded(gpu_lib, lens, Hkv, rows, d, dtype):
    """A CTA ends one segment of many parts and begins another: every call
    writes every row, and the same bits, alone and while calls on another stream
    delay its CTAs."""
    fa2 = gpu_lib
    args, want = in_one_page(fa2, lens, Hkv, rows, d, dtype)
    ws = [torch.empty(fa2.fa2_fwd_kv4_workspace(len(lens), rows[0] * Hkv, Hkv, rows[1], d, args[2].shape[1], 64),
                      dtype=torch.uint8, device="cuda") for _ in range(2)]
    first = fa2.fa2_fwd_kv4(*args, causal=True)
    check(*first, want)
    o, lse = (torch.empty_like(x) for x in first)
    for _ in range(100):
        o.fill_(math.nan), lse.fill_(math.nan)
        fa2.fa2_fwd_kv4(*args, o, lse, ws[0], causal=True)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            one = [torch.full_like(x, math.nan) for x in first]
            fa2.fa2_fwd_kv4(*args, *one, ws[i % 2], causal=True)
            outs.append(one)
    for st in streams:
        assert fa2.fa2_check_status(st.cuda_stream) == fa2.FA2_OK
    assert all(torch.equal(x[0], first[0]) and torch.equal(x[1], first[1]) for x in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hkv,rows,d,dtype", LINES[:2] + LINES[4:6])
def test_lines_that_are_not_padded_in_a_graph(gpu_lib, lens, Hkv, rows, d, dtype):
    """Replays carry the same launch's number: each finds the counters clean."""
    fa2 = gpu_lib
    args, want = in_one_page(fa2, lens, Hkv, rows, d, dtype)
    ws = torch.full((fa2.fa2_fwd_kv4_workspace(len(lens), rows[0] * Hkv, Hkv, rows[1], d, args[2].shape[1], 64),), 0x5A,
                    dtype=torch.uint8, device="cuda")
    first = fa2.fa2_fwd_kv4(*args, causal=True)
    check(*first, want)
    o, lse = (torch.empty_like(x) for x in first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa2.fa2_fwd_kv4(*args, o, lse, ws, causal=True)
    for _ in range(100):
        o.fill_(math.nan), lse.fill_(math.nan)
        g.replay()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_OK
