"""Rotary positions and the append to the 16-bit KV cache on the GPU against the
fp64 oracle (oracle/kv16.py).

Bound of an element y of a pair (x1, x2): an angle is off by 2^-32 of a turn, by
half a step (2^-24 of at most pi) when it becomes a float, and sine and cosine by
two of their steps (2^-23); two products and a sum round once each (2^-24 of
|x1| + |x2|). Together less than 2^-20 (|x1| + |x2|), then one rounding of y: half
a step of the type, u |y|, or of fp16's smallest, 2^-25.
"""
import numpy as np
import pytest
import torch

from oracle import kv16

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}


def ok(fa2):
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_OK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def freqs(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def sections(rot):
    P = rot // 2
    a = P // 4
    return np.array([0] * a + [1] * ((P - a) // 2) + [2] * (P - a - (P - a) // 2), np.int32)


def check(got, x, positions, f, axes, inter, inverse, dtype):
    """got, x [..., d] with positions [A, ...] of the leading sizes."""
    x = x.double().cpu().numpy()
    want = kv16.rotate(x, positions, f, axes, inter, inverse)
    P = len(f)
    i = np.arange(P)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + P)
    size = np.zeros_like(x)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    err = np.abs(got.double().cpu().numpy() - want)
    bound = 2.0 ** -20 * size + U[dtype] * np.abs(want) + SUB[dtype]
    bound[..., 2 * P:] = 0   # copied
    assert np.all(err <= bound), np.nanmax(err / np.maximum(bound, 1e-300))


def spread(positions, heads):
    """[A, B, N] to [A, B, heads, N]."""
    return np.broadcast_to(positions[:, :, None], positions.shape[:2] + (heads,) + positions.shape[2:])


def some_positions(rng, A, B, N, kind):
    if kind == "near":
        return rng.integers(0, 3, (A, B, 1)) + np.arange(N) * np.arange(1, A + 1)[:, None, None]
    if kind == "far":
        return rng.integers(2 ** 19, 2 ** 21, (A, B, N))
    x = rng.integers(-2 ** 31, 2 ** 31, (A, B, N))   # any int32, the ends among them
    x[0, 0, 0] = -2 ** 31
    x[0, -1, -1] = 2 ** 31 - 1
    return x


CASES = [
    # B, Hq, Hkv, N, d, rot, A, interleaved, dtype, positions
    (1, 1, 0, 1, 128, 128, 1, False, "bf16", "near"),
    (1, 1, 1, 1, 64, 16, 1, True, "fp16", "any"),
    (2, 4, 2, 37, 128, 128, 1, False, "bf16", "far"),
    (2, 4, 2, 37, 128, 128, 3, False, "fp16", "far"),
    (3, 3, 1, 11, 64, 64, 3, True, "bf16", "any"),
    (1, 7, 1, 130, 128, 64, 1, False, "fp16", "near"),
    (1, 2, 2, 65, 128, 96, 2, False, "bf16", "any"),
    (2, 2, 2, 33, 64, 48, 8, True, "fp16", "far"),
    (1, 5, 0, 5003, 64, 64, 3, False, "bf16", "near"),     # eight tokens a block
    (3, 3, 1, 1700, 128, 80, 1, True, "fp16", "far"),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,A,inter,dtype,kind", CASES)
def test_rope_every_element(gpu_lib, B, Hq, Hkv, N, d, rot, A, inter, dtype, kind, inverse):
    fa2 = gpu_lib
    rng = np.random.default_rng(B + N + rot)
    pos = some_positions(rng, A, B, N, kind)
    f = freqs(rot)
    axes = rng.integers(0, A, rot // 2).astype(np.int32) if A > 1 else None
    q = torch.tensor(rng.standard_normal((B, Hq, N, d))).to(DT[dtype]).cuda()
    k = torch.tensor(rng.standard_normal((B, Hkv, N, d))).to(DT[dtype]).cuda() if Hkv else None
    call = fa2.fa2_rope_bwd if inverse else fa2.fa2_rope
    p = i32(pos if A > 1 else pos[0])
    yq, yk = call(q, k, p, torch.tensor(f).cuda(), None if axes is None else i32(axes), inter)
    ok(fa2)
    check(yq, q, spread(pos, Hq), f, axes, inter, inverse, dtype)
    if k is None:
        assert yk is None
    else:
        check(yk, k, spread(pos, Hkv), f, axes, inter, inverse, dtype)


def test_frequencies_of_every_size(gpu_lib):
    """Frequencies from far below to far above a radian, of both signs, zero."""
    fa2 = gpu_lib
    rng = np.random.default_rng(4)
    f = np.concatenate([2.0 ** np.arange(-40, 20), [0.0, -0.25, -3e-5, 1e-30]]).astype(np.float32)
    pos = rng.integers(-1000, 1000, (1, 1, 50))
    q = torch.tensor(rng.standard_normal((1, 2, 50, 128))).to(torch.float16).cuda()
    y, _ = fa2.fa2_rope(q, None, i32(pos[0]), torch.tensor(f).cuda())
    ok(fa2)
    check(y, q, spread(pos, 2), f, None, False, False, "fp16")


@pytest.mark.parametrize("inter", [False, True])
def test_views_in_place_and_back(gpu_lib, inter):
    """From a projection's output to dense tensors, into a projection's layout,
    and in place: the same bits; rotating back gives the input again."""
    fa2 = gpu_lib
    rng = np.random.default_rng(5)
    B, Hq, Hkv, N, d = 2, 6, 2, 70, 128
    x = torch.tensor(rng.standard_normal((B, N, Hq + 2 * Hkv, d))).to(torch.bfloat16).cuda()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq: Hq + Hkv].transpose(1, 2)
    pos, f = i32(rng.integers(0, 9000, (3, B, N))), torch.tensor(freqs(128)).cuda()
    axes = i32(sections(128))
    yq, yk = fa2.fa2_rope(q, k, pos, f, axes, inter)
    assert yq.is_contiguous() and yk.is_contiguous()
    zq, zk = fa2.fa2_rope(q.contiguous(), k.contiguous(), pos, f, axes, inter)
    assert torch.equal(yq, zq) and torch.equal(yk, zk)
    to = torch.full((B, N, Hq + Hkv + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fa2.fa2_rope(q, k, pos, f, axes, inter, q_out=to[:, :, :Hq].transpose(1, 2), k_out=to[:, :, Hq: Hq + Hkv].transpose(1, 2))
    assert torch.equal(to[:, :, :Hq].transpose(1, 2), yq) and torch.equal(to[:, :, Hq: Hq + Hkv].transpose(1, 2), yk)
    assert (to[:, :, -1] == 7).all()
    before = x.clone()
    a, b = fa2.fa2_rope(q, k, pos, f, axes, inter, q_out=q, k_out=k)
    assert a is not None and torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(x[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])
    fa2.fa2_rope_bwd(q, k, pos, f, axes, inter, dq=q, dk=k)
    ok(fa2)
    # two roundings, each half a step of a value no larger than its pair
    i = torch.arange(64, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + 64)
    pair = torch.empty_like(before, dtype=torch.float32)
    pair[..., ia] = pair[..., ib] = (before[..., ia].float() ** 2 + before[..., ib].float() ** 2).sqrt()
    assert ((x - before).float().abs()[:, :, : Hq + Hkv] <= 4 * 2.0 ** -8 * pair[:, :, : Hq + Hkv]).all()


def test_gradient_against_differences(gpu_lib):
    """<dy, rope(x + h e) - rope(x - h e)> / 2h in 64 bits is the gradient's
    element: the rotation is linear, so any h gives it to rounding."""
    fa2 = gpu_lib
    rng = np.random.default_rng(6)
    B, H, N, d, rot = 1, 2, 3, 64, 48
    pos, f = rng.integers(0, 5000, (3, B, N)), freqs(rot)
    axes = sections(rot)
    x, dy = rng.standard_normal((B, H, N, d)), torch.tensor(rng.standard_normal((B, H, N, d))).to(torch.float16)
    g, _ = fa2.fa2_rope_bwd(dy.cuda(), None, i32(pos), torch.tensor(f).cuda(), i32(axes))
    ok(fa2)
    g, w = g.double().cpu().numpy(), dy.double().numpy()
    for e in np.ndindex(B, H, N, d):
        h = np.zeros_like(x)
        h[e] = 0.5
        up, down = (kv16.rotate(x + s * h, spread(pos, H), f, axes) for s in (1, -1))
        want = float((w * (up - down)).sum())
        assert abs(g[e] - want) <= 2.0 ** -11 * abs(want) + 2.0 ** -19 * np.abs(w[e[:3]]).max() + 2.0 ** -25


def test_an_axis_that_is_none_is_reported(gpu_lib):
    fa2 = gpu_lib
    q = torch.randn(1, 1, 2, 64, device="cuda").to(torch.bfloat16)
    f = torch.tensor(freqs(32)).cuda()
    axes = np.zeros(16, np.int32)
    axes[3], axes[7] = 2, -1
    pos = np.array([[[5, 9]], [[1, 2]]])
    y, _ = fa2.fa2_rope(q, None, i32(pos), f, i32(axes))
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_ERR_BOUNDS
    g = freqs(32)
    g[[3, 7]] = 0
    axes[[3, 7]] = 0
    check(y, q, spread(pos, 1), g, axes, False, False, "bf16")
    ok(fa2)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("T,Hq,Hkv,d,rot,A,inter,page,dtype", [
    (1, 4, 1, 128, 128, 1, False, 16, "bf16"),
    (130, 0, 2, 64, 64, 3, True, 32, "fp16"),
    (77, 6, 3, 128, 64, 3, False, 64, "bf16"),
    (300, 0, 2, 128, 0, 0, False, 128, "fp16"),           # nothing is rotated
    (5001, 2, 1, 64, 32, 1, False, 16, "bf16"),
])
def test_append_every_element(gpu_lib, T, Hq, Hkv, d, rot, A, inter, page, dtype):
    fa2 = gpu_lib
    rng = np.random.default_rng(T + d)
    x = torch.tensor(rng.standard_normal((T, Hq + 2 * Hkv + 1, d))).to(DT[dtype]).cuda()
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv: Hq + 2 * Hkv]
    P = -(-T // page) + 3
    slots = rng.permutation(P * page)[:T]
    slots[rng.random(T) < 0.1] = -1
    cache = torch.full(fa2.fa2_kv16_cache_shape(P, Hkv, page, d), 7.0, dtype=DT[dtype], device="cuda")
    kw = {}
    if rot:
        pos, f = some_positions(rng, A, 1, T, "far")[:, 0], freqs(rot)
        axes = rng.integers(0, A, rot // 2).astype(np.int32) if A > 1 else None
        kw = dict(positions=i32(pos), inv_freq=torch.tensor(f).cuda(), axes=None if axes is None else i32(axes), interleaved=inter)
    if Hq:
        kw["q"] = q
    c, q_out = fa2.fa2_kv16_append(k, v, i32(slots), cache, **kw)
    ok(fa2)
    assert c is cache
    rows = cache.permute(0, 3, 2, 1, 4).reshape(P * page, 2, Hkv, d)   # by slot
    live = slots >= 0
    at = torch.tensor(slots[live]).cuda()
    assert torch.equal(rows[at, 1], v[torch.tensor(live).cuda()])
    rest = np.ones(P * page, bool)
    rest[slots[live]] = False
    assert (rows[torch.tensor(rest).cuda()] == 7).all()
    if not rot:
        assert q_out is None and torch.equal(rows[at, 0], k[torch.tensor(live).cuda()])
        return
    heads = lambda p, h: np.broadcast_to(p[:, :, None], p.shape + (h,))
    check(rows[at, 0], k[torch.tensor(live).cuda()], heads(pos[:, live], Hkv), f, axes, inter, False, dtype)
    if Hq:
        check(q_out, q, heads(pos, Hq), f, axes, inter, False, dtype)


def test_slots_outside_the_cache_are_reported(gpu_lib):
    fa2 = gpu_lib
    cache = torch.zeros(fa2.fa2_kv16_cache_shape(2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    fa2.fa2_kv16_append(k, k, i32([32, 2 ** 31 - 1, 31]), cache)
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_ERR_BOUNDS
    assert (cache[1, 0, :, 15] == 1).all() and float(cache.float().sum()) == 128
    ok(fa2)


# ------------------------------------------------------------------ as a training step uses them

@pytest.mark.parametrize("inter", [False, True])
def test_rotation_attention_and_their_gradients(gpu_lib, inter):
    """rope, fa2_fwd_ex, fa2_bwd and rope_bwd in turn, against the gradients of
    the same function in 64 bits on the same projection's output."""
    fa2 = gpu_lib
    rng = np.random.default_rng(9)
    B, Hq, Hkv, N, d = 2, 4, 2, 150, 64
    x = torch.tensor(rng.standard_normal((B, N, Hq + 2 * Hkv, d))).to(torch.bfloat16).cuda()
    dout = torch.tensor(rng.standard_normal((B, Hq, N, d))).to(torch.bfloat16).cuda()
    pos, f = rng.integers(0, 3000, (3, B, N)), freqs(d)
    axes = sections(d)
    P, F, A = i32(pos), torch.tensor(f).cuda(), i32(axes)
    y = x.transpose(1, 2)
    v = y[:, Hq + Hkv:].contiguous()
    q, k = fa2.fa2_rope(y[:, :Hq], y[:, Hq: Hq + Hkv], P, F, A, inter)
    o, lse = fa2.fa2_fwd_ex(q, k, v, causal=True)
    dq, dk, dv = fa2.fa2_bwd(q, k, v, o, lse, dout, causal=True)
    dx = torch.zeros_like(x)
    to = dx.transpose(1, 2)
    fa2.fa2_rope_bwd(dq, dk, P, F, A, inter, dq=to[:, :Hq], dk=to[:, Hq: Hq + Hkv])
    to[:, Hq + Hkv:] = dv
    ok(fa2)
    # 64 bits, by autograd on elementary operations
    z = x.double().cpu().requires_grad_()
    i = np.arange(d // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + d // 2)
    angle = torch.tensor(pos[axes].transpose(1, 2, 0) * f.astype(np.float64))[:, :, None]
    c, s = angle.cos(), angle.sin()

    def turn(t):
        out = torch.empty_like(t)
        out[..., ia] = t[..., ia] * c - t[..., ib] * s
        out[..., ib] = t[..., ib] * c + t[..., ia] * s
        return out.transpose(1, 2)

    qq, kk, vv = turn(z[:, :, :Hq]), turn(z[:, :, Hq: Hq + Hkv]), z[:, :, Hq + Hkv:].transpose(1, 2)
    kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in (kk, vv))
    sc = (qq @ kk.transpose(2, 3)) * d ** -0.5
    sc = sc.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -torch.inf)
    (sc.softmax(-1) @ vv * dout.double().cpu()).sum().backward()
    want = z.grad
    err = (dx.double().cpu() - want).abs()
    # q, k, o, weights, their gradients and the results are rounded to bf16, each half a step of a
    # term no larger than the largest: eight of them
    scale = want.abs().amax()
    assert err.max() <= 8 * U["bf16"] * scale
    assert err.pow(2).mean().sqrt() <= 2 * U["bf16"] * want.pow(2).mean().sqrt()


def test_captured_rotation_and_its_gradient(gpu_lib):
    fa2 = gpu_lib
    rng = np.random.default_rng(10)
    x = torch.tensor(rng.standard_normal((2, 6, 90, 128))).to(torch.float16).cuda()
    pos, f = i32(rng.integers(0, 999, (2, 90))), torch.tensor(freqs(128)).cuda()
    y, z, g = torch.empty_like(x), torch.empty_like(x), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        fa2.fa2_rope(x, None, pos, f, q_out=y)
        fa2.fa2_rope_bwd(y, None, pos, f, dq=z)
    for _ in range(3):
        x.copy_(torch.randn(x.shape, device="cuda"))
        pos.add_(17)
        g.replay()
        a, _ = fa2.fa2_rope(x, None, pos, f)
        b, _ = fa2.fa2_rope_bwd(a, None, pos, f)
        assert torch.equal(a, y) and torch.equal(b, z)
    ok(fa2)


def test_refusals(gpu_lib):
    fa2 = gpu_lib
    dev = "cuda"
    q, k = torch.zeros(2, 4, 5, 64, dtype=torch.bfloat16, device=dev), torch.zeros(2, 2, 5, 64, dtype=torch.bfloat16, device=dev)
    pos, f = torch.zeros(2, 5, dtype=torch.int32, device=dev), torch.zeros(32, device=dev)
    good = [q, k, pos, f]
    fa2.fa2_rope(*good)
    bad = [(0, q.float()), (0, q[0]), (0, q.transpose(2, 3)), (0, torch.zeros(2, 4, 5, 96, dtype=torch.bfloat16, device=dev)),
           (0, torch.zeros(2, 4, 5, 68, dtype=torch.bfloat16, device=dev)[..., :64]),
           (0, torch.zeros(2, 4, 5, 72, dtype=torch.bfloat16, device=dev)[..., 4:68]), (0, q.cpu()), (1, k.half()), (1, k[:1]), (1, k[:, :, :4]),
           (1, k.cpu()), (2, pos.long()), (2, pos[:, :4]), (2, pos.cpu()), (2, torch.zeros(9, 2, 5, dtype=torch.int32, device=dev)),
           (3, f.double()), (3, f[:7]), (3, torch.zeros(40, device=dev)), (3, f[:0]), (3, f.cpu())]
    for i, x in bad:
        args = list(good)
        args[i] = x
        for call in (fa2.fa2_rope, fa2.fa2_rope_bwd):
            with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
                call(*args)
    for kw in (dict(axes=torch.zeros(31, dtype=torch.int32, device=dev)), dict(axes=torch.zeros(32, device=dev)),
               dict(q_out=torch.zeros(2, 4, 5, 64, device=dev)), dict(q_out=q[:, :3]), dict(k_out=q),
               dict(q_out=torch.zeros(1, 4, 5, 64, dtype=torch.bfloat16, device=dev).expand(2, 4, 5, 64))):
        with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
            fa2.fa2_rope(*good, **kw)
    with pytest.raises(ValueError):
        fa2.fa2_rope(q, None, pos, f, k_out=k)
    c = torch.zeros(fa2.fa2_kv16_cache_shape(2, 2, 16, 64), dtype=torch.bfloat16, device=dev)
    t, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev), i32([0, 1, 2])
    for args, kw in (((t, t, slots.long(), c), {}), ((t, t.half(), slots, c), {}), ((t, t[:2], slots, c), {}), ((t, t, slots[:2], c), {}),
                     ((t, t, slots, c[:, :1]), {}), ((t, t, slots, c.half()), {}), ((t[None], t[None], slots, c), {}),
                     ((t, t, slots, c), dict(q=t)), ((t, t, slots, c), dict(inv_freq=f)), ((t, t, slots, c), dict(q_out=t)),
                     ((t, t, slots, c), dict(positions=slots)), ((t, t, slots, c), dict(positions=slots[:2], inv_freq=f)),
                     ((t, t, slots, c), dict(q=t[:2], positions=slots, inv_freq=f)),
                     ((t, t, slots, c), dict(q=t, positions=slots, inv_freq=f, q_out=t.float()))):
        with pytest.raises((ValueError, TypeError, fa2.FA2Error)):
            fa2.fa2_kv16_append(*args, **kw)
    ok(fa2)
