"""Cases for rotary positions and for a paged KV cache held in 16 bits.

The cache is one 16-bit tensor [num_pages, H_kv, 2, page_size, d]: of a page
and KV head first the keys, then the values of page_size tokens. A token's
place is its slot, page * page_size + offset.

Operators:
  rope      rotates q and k [B, H, N, d] by their positions (several axes:
            time, height, width), from a projection's output to the dense
            tensors that attention takes
  rope_bwd  the gradient of it, from attention's gradients back to the
            projection's layout
  append    rotates new keys and queries and writes keys and values into
            their slots
  attend    attention of each request's new tokens (one for a decoding
            request, a chunk for a prompt) over its cached tokens
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One user, one token, a short conversation: launch latency is what counts.
        {"name": "attend_one_short", "op": "attend", "chunks": 0, "chunk": 0, "singles": 1, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "max_len": 517, "dtype": "bf16"},
        # A server's decode step: a token of each request, ragged contexts.
        {"name": "attend_decode", "op": "attend", "chunks": 0, "chunk": 0, "singles": 64, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "max_len": 16384, "dtype": "bf16"},
        # A mixed step: prompts' chunks beside decoding requests, small pages.
        {"name": "attend_mixed", "op": "attend", "chunks": 3, "chunk": 512, "singles": 24, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 16, "max_len": 8192, "dtype": "fp16"},
        # Whole prompts of a model with heads of 64, ungrouped.
        {"name": "attend_prompts_d64", "op": "attend", "chunks": 2, "chunk": 4096, "singles": 0, "Hq": 32, "Hkv": 32, "d": 64,
         "page": 32, "max_len": 4096, "dtype": "fp16"},
        # The largest: the last chunk of a long document.
        {"name": "attend_chunk_long", "op": "attend", "chunks": 1, "chunk": 2048, "singles": 0, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "max_len": 32768, "dtype": "bf16"},
        # The cache write of a decode step of 128 requests.
        {"name": "append_step", "op": "append", "T": 128, "axes": 1, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "inter": False,
         "page": 64, "dtype": "bf16"},
        # The cache write of a step of prompts with images: positions in time, height and width.
        {"name": "append_prompts", "op": "append", "T": 8191, "axes": 3, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "page": 64, "dtype": "bf16"},
        # A short text, neighbouring pairs, heads of 64.
        {"name": "rope_short", "op": "rope", "B": 1, "N": 517, "axes": 1, "Hq": 16, "Hkv": 16, "d": 64, "rot": 64,
         "inter": True, "dtype": "fp16"},
        # A training step's batch of texts.
        {"name": "rope_text", "op": "rope", "B": 4, "N": 4096, "axes": 1, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16"},
        # A training step's batch of videos, three axes, ungrouped heads, a length of no round number.
        {"name": "rope_video", "op": "rope", "B": 2, "N": 8191, "axes": 3, "Hq": 16, "Hkv": 16, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16"},
        # Gradients of a short text, half of each head rotated.
        {"name": "rope_bwd_short", "op": "rope_bwd", "B": 1, "N": 1000, "axes": 1, "Hq": 8, "Hkv": 2, "d": 128, "rot": 64,
         "inter": False, "dtype": "bf16"},
        # Gradients of a training step's batch.
        {"name": "rope_bwd_text", "op": "rope_bwd", "B": 4, "N": 4096, "axes": 1, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "rope", "rope_bwd"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "attend":
        G = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
        max_len = _log_int(rng, 1, 32768)
        chunks = rng.choice([0, 0, 1, 1, 2, 4])
        chunk = _log_int(rng, 2, max(2, min(max_len, 4096))) if chunks and max_len > 1 else 0
        chunks = chunks if chunk else 0
        most = 2048 * 32768 * 32   # (row, key) pairs of the largest listed case
        while chunks > 1 and chunks * chunk * max_len * G * Hkv > most:
            chunks -= 1
        chunk = max(1, min(chunk, most // (max_len * G * Hkv))) if chunks else 0
        singles = _log_int(rng, 1, max(1, min(128, 2 ** 23 // (max_len * Hkv)))) if not chunks or rng.random() < 0.5 else 0
        return {"op": op, "chunks": chunks, "chunk": chunk, "singles": singles, "Hq": G * Hkv, "Hkv": Hkv, "d": d,
                "page": rng.choice([16, 32, 64, 128]), "max_len": max_len, "dtype": dtype}
    G = rng.choice([1, 1, 2, 4, 7, 8])
    rot = rng.choice([d, d, d // 2])
    inter = rng.random() < 0.3
    axes = rng.choice([1, 1, 3])
    most = 16384 * 40 * 128 // ((G + 1) * Hkv * d)
    if op == "append":
        return {"op": op, "T": _log_int(rng, 1, max(1, min(16384, most // 2))), "axes": axes, "Hq": G * Hkv, "Hkv": Hkv, "d": d,
                "rot": rot, "inter": inter, "page": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    N = _log_int(rng, 1, min(16384, most))
    return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most // N))), "N": N, "axes": axes, "Hq": G * Hkv, "Hkv": Hkv, "d": d,
            "rot": rot, "inter": inter, "dtype": dtype}


def _requests(case):
    """New and cached tokens of each request of a step, the new ones among the
    cached: plain numbers of the case alone. A request's first chunk finds
    nothing before it, a later one the tokens of those before it."""
    rng = random.Random(",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))
    top, out = case["max_len"], []
    for i in range(case["chunks"]):
        n = case["chunk"] if i == 0 else rng.randint((case["chunk"] + 1) // 2, case["chunk"])
        out.append((n, top if i == 0 else rng.randint(n, top)))
    for i in range(case["singles"]):
        out.append((1, top if i == 0 and not case["chunks"] else rng.randint(max(1, top // 3), top)))
    rng.shuffle(out)
    return out


# ------------------------------------------------------------------ inputs

def _inv_freq(rot, dev):
    return (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)).float()


def _axes(case, dev):
    """The axis of each pair: runs of pairs in the shares 2 : 3 : 3."""
    P = case["rot"] // 2
    a = P // 4
    b = (P - a) // 2
    return torch.tensor([0] * a + [1] * b + [2] * (P - a - b), dtype=torch.int32, device=dev)


def _positions(case, shape, g, dev):
    """Texts count up from somewhere in a long document. Of three axes, runs
    of text have all three equal and images a grid of rows and columns."""
    B, N = shape
    first = torch.randint(0, 1 << 17, (B, 1), generator=g, device=dev)
    n = torch.arange(N, device=dev)
    t = first + n
    if case["axes"] == 1:
        return t[None].to(torch.int32).contiguous()
    frame = n // 1024 * 1024
    image = (n // 1024 % 2 == 1)
    grid = torch.stack([first + frame, first + frame + n % 1024 // 32, first + frame + n % 32])
    return torch.where(image, grid, t[None]).to(torch.int32).contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case)
    dtype = DT[case["dtype"]]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    if case["op"] == "attend":
        page = case["page"]
        new, lens = zip(*_requests(case))
        need = [-(-n // page) for n in lens]
        total, width = sum(need), max(need)
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        have = torch.tensor(need, device=dev)
        j = torch.arange(width, device=dev)
        at = ((have.cumsum(0) - have)[:, None] + j).clamp(max=total - 1)
        s["block_table"] = torch.where(j < have[:, None], ids[at], -1).to(torch.int32).contiguous()
        cache = torch.empty(total, Hkv, 2, page, d, dtype=dtype, device=dev)
        for p0 in range(0, total, 1024):
            x = torch.randn(min(1024, total - p0), Hkv, 2, page, d, generator=g, device=dev)
            x[:, :, 0, :, :: d // 4] *= 2.5   # keys have a few strong channels
            cache[p0: p0 + 1024] = x.to(dtype)
        s["cache"] = cache
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q_lens"] = torch.tensor(new, dtype=torch.int32, device=dev)
        s["q_starts"] = (s["q_lens"].cumsum(0) - s["q_lens"]).to(torch.int32)
        s["new"], s["lens"] = list(new), list(lens)
        s["q"] = randn(sum(new), Hq, d)
        s["scale"] = d ** -0.5
        return s
    s["inv_freq"] = _inv_freq(case["rot"], dev)
    s["axis"] = _axes(case, dev) if case["axes"] == 3 else None
    if case["op"] == "append":
        T, page = case["T"], case["page"]
        x = randn(T, Hq + 2 * Hkv, d)   # a projection's output
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
        s["positions"] = _positions(case, (1, T), g, dev)[:, 0].contiguous()
        # runs of tokens on pages in no order (a step's requests), a few places of a padded batch left out
        pages = -(-T // page) + 8
        ids = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        slots = ids[t // page] * page + t % page
        s["slots"] = torch.where(t % 61 == 60, -1, slots).to(torch.int32)
        s["cache"] = torch.zeros(pages, Hkv, 2, page, d, dtype=dtype, device=dev)
        return s
    B, N = case["B"], case["N"]
    s["positions"] = _positions(case, (B, N), g, dev)
    if case["op"] == "rope":
        x = randn(B, N, Hq + 2 * Hkv, d).transpose(1, 2)
        s["q"], s["k"] = x[:, :Hq], x[:, Hq: Hq + Hkv]
    else:
        s["dq"], s["dk"] = randn(B, Hq, N, d), randn(B, Hkv, N, d)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"rope": _rope, "rope_bwd": _rope_bwd, "append": _append, "attend": _attend}[s["op"]](s)


def _angles(positions, inv_freq, axis):
    """positions [A, ...] to angles [..., pairs], in 64 bits: far positions
    leave few of 24 bits for the angle in a turn."""
    p = positions.double()
    p = p[0][..., None].expand(*p.shape[1:], inv_freq.shape[0]) if axis is None else p[axis.long()].movedim(0, -1)
    return p * inv_freq.double()


def _rotate(x, cos, sin, rot, inter):
    """x [..., d] with cos, sin [..., rot / 2] broadcast to it, in 32 bits."""
    x = x.float()
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _rope(s):
    q, k = s["q"], s["k"]
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        return fa2.fa2_rope(q, k, s["positions"], s["inv_freq"], axes=s["axis"], interleaved=s["inter"])
    a = _angles(s["positions"], s["inv_freq"], s["axis"])[:, None]
    cos, sin = a.cos().float(), a.sin().float()
    return tuple(_rotate(x, cos, sin, s["rot"], s["inter"]).to(x.dtype).contiguous() for x in (q, k))


def _rope_bwd(s):
    """The gradients go into the layout of the projection's output, where the
    projection's own gradient is taken."""
    dq, dk = s["dq"], s["dk"]
    B, N, Hq, Hkv = s["B"], s["N"], s["Hq"], s["Hkv"]
    dx = torch.empty(B, N, Hq + Hkv, s["d"], dtype=dq.dtype, device=dq.device)
    to = dx.transpose(1, 2)
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        fa2.fa2_rope_bwd(dq, dk, s["positions"], s["inv_freq"], axes=s["axis"], interleaved=s["inter"], dq=to[:, :Hq],
                         dk=to[:, Hq:])
        return dx
    a = _angles(s["positions"], s["inv_freq"], s["axis"])[:, None]
    cos, sin = a.cos().float(), -a.sin().float()
    to[:, :Hq] = _rotate(dq, cos, sin, s["rot"], s["inter"]).to(dq.dtype)
    to[:, Hq:] = _rotate(dk, cos, sin, s["rot"], s["inter"]).to(dk.dtype)
    return dx


def _append(s):
    q, k, v, slots, cache = s["q"], s["k"], s["v"], s["slots"], s["cache"]
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        _, q_out = fa2.fa2_kv16_append(k, v, slots, cache, q=q, positions=s["positions"], inv_freq=s["inv_freq"],
                                       axes=s["axis"], interleaved=s["inter"])
        return cache, q_out
    a = _angles(s["positions"], s["inv_freq"], s["axis"])[:, None]
    cos, sin = a.cos().float(), a.sin().float()
    page = s["page"]
    keep = (slots >= 0).nonzero()[:, 0]
    at = slots[keep].long()
    cache[at // page, :, 0, at % page] = _rotate(k, cos, sin, s["rot"], s["inter"]).to(k.dtype)[keep]
    cache[at // page, :, 1, at % page] = v[keep]
    return cache, _rotate(q, cos, sin, s["rot"], s["inter"]).to(q.dtype)


def _attend(s):
    q, cache, table = s["q"], s["cache"], s["block_table"]
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        return fa2.fa2_fwd_kv16(q, cache, table, s["seq_lens"], s["q_starts"], s["q_lens"], scale=s["scale"], causal=True)
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    G = Hq // Hkv
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        pages = table[b, : -(-L // s["page"])].long()
        kv = cache[pages].permute(2, 1, 0, 3, 4).reshape(2, Hkv, -1, d)[:, :, :L].float()
        step = max(1, 2 ** 29 // (Hq * L))   # rows at a time: 2 GB of scores
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            x = q[at + i0: at + i1].float().reshape(i1 - i0, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
            x = torch.matmul(x, kv[0].transpose(1, 2)) * s["scale"]
            x = x.reshape(Hkv, G, i1 - i0, L)
            if n > 1:
                end = L - n + 1 + torch.arange(i0, i1, device=q.device)
                x = x.masked_fill(torch.arange(L, device=q.device) >= end[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            x = torch.exp(x - m)
            total = x.sum(-1, keepdim=True)
            y = torch.matmul(x.reshape(Hkv, -1, L), kv[1]).reshape(Hkv, G, i1 - i0, d) / total
            o[at + i0: at + i1] = y.permute(2, 0, 1, 3).reshape(i1 - i0, Hq, d).to(q.dtype)
            lse[at + i0: at + i1] = (m + total.log())[..., 0].permute(2, 0, 1).reshape(i1 - i0, Hq)
        at += n
    return o, lse


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "attend":
        pairs = rows = tokens = pages = 0
        for n, L in _requests(case):
            pairs += n * L - n * (n - 1) // 2   # row i sees L - n + 1 + i keys
            rows += n
            tokens += L
            pages += -(-L // case["page"])
        return {"bytes": 4.0 * tokens * Hkv * d + rows * Hq * (4.0 * d + 4) + 4.0 * pages, "flops": 4.0 * pairs * Hq * d}
    T = case["T"] if case["op"] == "append" else case["B"] * case["N"]
    heads = Hq + Hkv + (Hkv if case["op"] == "append" else 0)
    return {"bytes": 4.0 * T * heads * d + 4.0 * T * (case["axes"] + (case["op"] == "append")),
            "flops": 3.0 * T * (Hq + Hkv) * case["rot"]}


# ------------------------------------------------------------------ 64 bits

def _turned(x, positions, inv_freq, axis, rot, inter, sign):
    """x [..., H, N, d] of a batch entry with positions [A, N]: each pair as a
    complex number times exp(i * sign * angle)."""
    out = x.double().clone()
    pairs = torch.arange(rot // 2, device=x.device)
    i, j = (2 * pairs, 2 * pairs + 1) if inter else (pairs, pairs + rot // 2)
    which = torch.zeros_like(pairs) if axis is None else axis.long()
    angle = positions.double().index_select(0, which).T * inv_freq.double()     # [N, pairs]
    z = torch.complex(out[..., i], out[..., j]) * torch.polar(torch.ones_like(angle), sign * angle)
    out[..., i], out[..., j] = z.real, z.imag
    return out


def exact(case, seed):
    op = case["op"]
    if op == "attend":
        flops = work(case)["flops"]
        if flops > 3e12:
            return None
        return _exact_attend(prepare(case, seed))
    s = prepare(case, seed)
    rot, inter = case["rot"], case["inter"]
    if op == "append":
        q, k = (_turned(x.transpose(0, 1), s["positions"], s["inv_freq"], s["axis"], rot, inter, 1.0).transpose(0, 1)
                for x in (s["q"], s["k"]))
        cache = s["cache"].double()
        H, page = case["Hkv"], case["page"]
        rows = cache.permute(0, 3, 2, 1, 4).reshape(-1, 2, H, case["d"]).clone()     # by slot
        live = s["slots"] >= 0
        at = s["slots"].long()[live]
        rows[at, 0] = k[live]
        rows[at, 1] = s["v"].double()[live]
        return rows.reshape(-1, page, 2, H, case["d"]).permute(0, 3, 2, 1, 4).contiguous(), q.contiguous()
    sign = 1.0 if op == "rope" else -1.0
    names = ("q", "k") if op == "rope" else ("dq", "dk")
    out = [torch.stack([_turned(s[n][b], s["positions"][:, b], s["inv_freq"], s["axis"], rot, inter, sign)
                        for b in range(case["B"])]) for n in names]
    return tuple(out) if op == "rope" else torch.cat(out, 1).transpose(1, 2).contiguous()


def _exact_attend(s):
    Hq, Hkv, d, page = s["Hq"], s["Hkv"], s["d"], s["page"]
    G, dev = Hq // Hkv, s["q"].device
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=dev)
    first = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        pos = torch.arange(L, device=dev)
        pg = s["block_table"][b].long()[pos // page]
        for h in range(Hkv):
            k = s["cache"][pg, h, 0, pos % page].double()
            v = s["cache"][pg, h, 1, pos % page].double()
            heads = slice(h * G, (h + 1) * G)
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                x = torch.einsum("ngd,ld->ngl", s["q"][first + i0: first + i1, heads].double(), k) * s["scale"]
                last = L - n + torch.arange(i0, i1, device=dev)                  # the last key that a row sees
                x = torch.where(pos[None, None] <= last[:, None, None], x, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[first + i0: first + i1, heads] = z
                o[first + i0: first + i1, heads] = torch.einsum("ngl,ld->ngd", torch.exp(x - z[..., None]), v)
        first += n
    return o, lse
