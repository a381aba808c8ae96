"""Cases for the operators around a paged KV cache held in 4 bits.

The cache is one uint8 tensor [num_pages, H_kv, 2, page_size * (d/2 + d/16)].
Part 0 of a (page, KV head) holds the keys of page_size tokens, part 1 the
values: first the e2m1 codes [page_size, d/2] (element 2i of a token in the
low four bits of byte i), then one e4m3 scale for each 16 elements
[page_size, d/16]. An element stands for code * scale * descale[head].

Four operators work on it:
  plan    pages and slots of a step's new tokens, from the request lengths
  append  quantises new keys and values into their slots
  gather  reads tokens back as 16-bit tensors (for a prompt's own attention)
  decode  attention of N_q new tokens a request over its cached tokens
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One user, a short conversation: launch latency is what counts.
        {"name": "decode_one_short", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 1, "d": 128, "page": 64,
         "max_len": 517, "causal": False, "dtype": "bf16"},
        # A server's ordinary decode step: grouped heads, ragged contexts, some idle rows of a padded batch.
        {"name": "decode_batch", "op": "decode", "B": 32, "Hq": 32, "Hkv": 8, "Nq": 1, "d": 128, "page": 64,
         "max_len": 8192, "causal": False, "dtype": "bf16"},
        # One very long document, few KV heads: the long axis has to be split.
        {"name": "decode_one_long", "op": "decode", "B": 1, "Hq": 32, "Hkv": 4, "Nq": 1, "d": 128, "page": 128,
         "max_len": 262139, "causal": False, "dtype": "bf16"},
        # The largest step: many long contexts.
        {"name": "decode_large", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "d": 128, "page": 64,
         "max_len": 32768, "causal": False, "dtype": "bf16"},
        # Scoring five drafted tokens a request, causal among themselves.
        {"name": "decode_drafts", "op": "decode", "B": 16, "Hq": 32, "Hkv": 8, "Nq": 5, "d": 128, "page": 32,
         "max_len": 8192, "causal": True, "dtype": "fp16"},
        # Ungrouped heads of 64, small pages.
        {"name": "decode_mha_d64", "op": "decode", "B": 8, "Hq": 32, "Hkv": 32, "Nq": 1, "d": 64, "page": 16,
         "max_len": 2048, "causal": False, "dtype": "fp16"},
        # The cache write of one decode step of 128 requests.
        {"name": "append_step", "op": "append", "B": 128, "Hkv": 8, "N": 1, "d": 128, "page": 64, "start": 2048,
         "dtype": "bf16"},
        # The cache write of four prompts, padded to the longest.
        {"name": "append_prompts", "op": "append", "B": 4, "Hkv": 8, "N": 8191, "d": 128, "page": 64, "start": 0,
         "dtype": "bf16"},
        # A short context read back for the next chunk of its prompt.
        {"name": "gather_short", "op": "gather", "B": 1, "Hkv": 32, "d": 64, "page": 16, "max_len": 777,
         "dtype": "fp16"},
        # Two long contexts read back for chunked prompts.
        {"name": "gather_long", "op": "gather", "B": 2, "Hkv": 8, "d": 128, "page": 64, "max_len": 65536,
         "dtype": "bf16"},
        # The scheduler's step for 256 decoding requests, some of which end.
        {"name": "plan_step", "op": "plan", "B": 256, "N": 1, "page": 64, "max_len": 8192, "tight": False},
        # Admission of 48 prompts with too few free pages for all of them.
        {"name": "plan_prompts", "op": "plan", "B": 48, "N": 16384, "page": 16, "max_len": 16384, "tight": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "append", "gather", "plan"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        N = 1 if rng.random() < 0.5 else _log_int(rng, 2, 16384)
        return {"op": op, "B": _log_int(rng, 1, max(1, min(512, 700000 // N))), "N": N, "page": page,
                "max_len": max(N, _log_int(rng, 128, 16384)), "tight": rng.random() < 0.4}
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        N = 1 if rng.random() < 0.4 else _log_int(rng, 2, 16384)
        B = _log_int(rng, 1, max(1, min(256, 32768 // N * 8 // Hkv)))
        return {"op": op, "B": B, "Hkv": Hkv, "N": N, "d": d, "page": page,
                "start": 0 if rng.random() < 0.3 else _log_int(rng, 1, 4096), "dtype": dtype}
    if op == "gather":
        max_len = _log_int(rng, 1, 65536)
        B = _log_int(rng, 1, max(1, min(32, 131072 // max_len * 8 // Hkv)))
        return {"op": op, "B": B, "Hkv": Hkv, "d": d, "page": page, "max_len": max_len, "dtype": dtype}
    G = rng.choice([1, 2, 3, 4, 4, 7, 8, 8, 12, 16])
    Nq = 1 if rng.random() < 0.6 else rng.randint(2, 16)
    max_len = _log_int(rng, 1, 131072)
    B = _log_int(rng, 1, max(1, min(128, 64 * 8 * 32768 // (max_len * Hkv * max(1, G * Nq // 8)))))
    return {"op": op, "B": B, "Hq": G * Hkv, "Hkv": Hkv, "Nq": Nq, "d": d, "page": page, "max_len": max_len,
            "causal": Nq > 1 and rng.random() < 0.7, "dtype": dtype}


def _lengths(case):
    """Cached tokens of each request (decode, gather), or new tokens and the
    tokens before them (append): plain numbers of the case alone."""
    rng = random.Random(",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))
    B = case["B"]
    if case["op"] == "append":
        N, start = case["N"], case["start"]
        new = [N] + [N if N == 1 else rng.randint((N + 1) // 2, N) for _ in range(B - 1)]
        return new, [start] + [rng.randint(start // 2, start) for _ in range(B - 1)]
    top = case["max_len"]
    lens = [top] + [rng.randint(max(1, top // 3), top) for _ in range(B - 1)]
    if case["op"] == "decode":
        for b in range(11, B, 16):  # idle rows of a padded batch
            lens[b] = 0
    return lens, None


# ------------------------------------------------------------------ inputs

def _quantise(x, descale):
    """x [..., d] fp32, descale broadcast to x[..., 0]: the code bytes
    [..., d/2] and scale bytes [..., d/16] of an append."""
    d = x.shape[-1]
    xb = x.reshape(*x.shape[:-1], d // 16, 16)
    ds = descale[..., None]
    s8 = (xb.abs().amax(-1) / (6.0 * ds)).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = (s8.float() * ds)[..., None]
    q = torch.where(t > 0, xb / t, torch.zeros((), device=x.device))
    a = q.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code |= (q < 0).to(torch.uint8) << 3
    code = code.reshape(*x.shape[:-1], d // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s8.view(torch.uint8)


def _descales(Hkv, g, dev):
    # what calibration gives: a head's largest magnitude over the largest value a code and a scale stand for
    return tuple((4.0 + 4.0 * torch.rand(Hkv, generator=g, device=dev)) / (6.0 * 448.0) for _ in range(2))


def _filled_cache(num_pages, case, kd, vd, g, dev):
    """A cache whose every slot holds quantised values (slots past a
    request's last token hold what former requests left there). Keys have a
    few strong channels, as they do after a rotary embedding."""
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    chan = torch.ones(d, device=dev)
    chan[:: d // 4] = 2.5
    parts = []
    for descale, w in ((kd, chan), (vd, None)):
        x = torch.randn(num_pages, Hkv, page, d, generator=g, device=dev)
        x = x * w if w is not None else x
        codes, scales = _quantise(x, descale[None, :, None])
        del x
        parts.append(torch.cat([codes.reshape(num_pages, Hkv, -1), scales.reshape(num_pages, Hkv, -1)], -1))
        del codes, scales
    return torch.stack(parts, 2)


def _tables(lens, page, g, dev):
    """Pages of each request in no order, and how many there are."""
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    total = max(1, sum(need))
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    have = torch.tensor(need, device=dev)
    j = torch.arange(width, device=dev)
    first = have.cumsum(0) - have
    at = (first[:, None] + j[None, :]).clamp(max=total - 1)
    table = torch.where(j[None, :] < have[:, None], perm[at], -1)
    return table.to(torch.int32).contiguous(), total


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case)
    page = case["page"]
    if case["op"] == "plan":
        B, N, top = case["B"], case["N"], case["max_len"]
        width = -(-(top + N) // page)
        prompts = N > 1
        # decoding requests are anywhere in their context; prompts start from nothing or from a cached prefix
        lens = torch.randint(1, top + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        if prompts:
            lens = lens // 4 * (torch.rand(B, generator=g, device=dev) < 0.5)
        new = torch.randint(max(1, N // 2), N + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        u = torch.rand(B, generator=g, device=dev)
        new = torch.where(u < 0.06, -1, torch.where(u < 0.1, 0, new)).to(torch.int32)
        have = -(-lens // page)
        used = int(have.sum())
        need = int((-(-(lens + new.clamp(min=0)) // page) - have).sum())
        pages = B * width
        free = max(1, need * 3 // 4) if case["tight"] else pages - used
        ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        j = torch.arange(width, device=dev)
        at = ((have.cumsum(0) - have)[:, None] + j).clamp(max=pages - 1)
        s["block_table"] = torch.where(j < have[:, None], ids[at], -1).to(torch.int32).contiguous()
        head = int(torch.randint(0, pages, (1,), generator=g, device=dev))
        ring = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        ring[(head + torch.arange(free, device=dev)) % pages] = ids[used: used + free]
        s.update(seq_lens=lens.to(torch.int32), new_lens=new, free_pages=ring,
                 free_state=torch.tensor([head, free], dtype=torch.int32, device=dev))
        return s
    d, Hkv = case["d"], case["Hkv"]
    s["k_descale"], s["v_descale"] = kd, vd = _descales(Hkv, g, dev)
    if case["op"] == "append":
        new, start = _lengths(case)
        lens = [a + b for a, b in zip(new, start)]
        s["block_table"], total = _tables(lens, page, g, dev)
        s["cache"] = torch.zeros(total, Hkv, 2, page * (d // 2 + d // 16), dtype=torch.uint8, device=dev)
        s["k"], s["v"] = _new_tokens(case, g, dev)
        s["starts"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        i = torch.arange(case["N"], device=dev)
        pos = s["starts"][:, None] + i
        live = pos < s["seq_lens"][:, None]
        at = (pos // page).clamp(max=s["block_table"].shape[1] - 1)
        slots = s["block_table"].gather(1, at.long()) * page + pos % page
        s["slots"] = torch.where(live, slots, -1).to(torch.int32).contiguous()
        return s
    lens, _ = _lengths(case)
    s["block_table"], total = _tables(lens, page, g, dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cache"] = _filled_cache(total, case, kd, vd, g, dev)
    if case["op"] == "decode":
        q = torch.randn(case["B"], case["Hq"], case["Nq"], d, generator=g, device=dev)
        s["q"] = q.to(DT[case["dtype"]])
        s["scale"] = d ** -0.5
    return s


def _new_tokens(case, g, dev):
    shape = (case["B"], case["Hkv"], case["N"], case["d"])
    k = torch.randn(shape, generator=g, device=dev)
    k[..., :: case["d"] // 4] *= 2.5
    return k.to(DT[case["dtype"]]), torch.randn(shape, generator=g, device=dev).to(DT[case["dtype"]])


# ------------------------------------------------------------------ one pass

def run(s):
    return {"decode": _decode, "append": _append, "gather": _gather, "plan": _plan}[s["op"]](s)


def _values(part, descale, page, d):
    """[..., H, page * (d/2 + d/16)] bytes to fp32 [..., H, page, d]."""
    codes = part[..., : page * d // 2].reshape(*part.shape[:-1], page, d // 2)
    scales = part[..., page * d // 2:].contiguous().view(torch.float8_e4m3fn).float()
    t = scales.reshape(*part.shape[:-1], page, d // 16) * descale[:, None, None]
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                       device=part.device)
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(-1).int()
    c = lut.index_select(0, c).reshape(*part.shape[:-1], page, d // 16, 16)
    return (c * t[..., None]).reshape(*part.shape[:-1], page, d)


def _context(s, part):
    """Every request's cached keys (0) or values (1): fp32 [B, H, width * page, d]."""
    page, d, table = s["page"], s["d"], s["block_table"]
    x = s["cache"][:, :, part][table.clamp(min=0).long()]
    x = _values(x, s["k_descale"] if part == 0 else s["v_descale"], page, d)
    B, W, H = x.shape[:3]
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, W * page, d)


def _decode(s):
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        return fa2.fa2_fwd_kv4(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["k_descale"], s["v_descale"],
                               scale=s["scale"], causal=s["causal"])
    q, lens = s["q"], s["seq_lens"]
    B, Hq, Nq, d = q.shape
    Hkv = s["Hkv"]
    k = _context(s, 0)
    L = k.shape[2]
    x = torch.matmul(q.float().reshape(B, Hkv, (Hq // Hkv) * Nq, d), k.transpose(2, 3)) * s["scale"]
    del k
    j = torch.arange(L, device=q.device)
    i = torch.arange(Nq, device=q.device)
    end = lens[:, None].expand(B, Nq)
    end = torch.minimum(end, i + 1 + end - Nq) if s["causal"] else end
    seen = (j < end[..., None])[:, None, None]                                  # [B, 1, 1, Nq, L]
    x = x.reshape(B, Hkv, Hq // Hkv, Nq, L).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    del x
    total = p.sum(-1, keepdim=True)
    v = _context(s, 1).masked_fill(~(j < lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.reshape(B, Hkv, -1, L), v).reshape(B, Hkv, Hq // Hkv, Nq, d)
    o = torch.where(total > 0, o / total, 0.0).reshape(B, Hq, Nq, d)
    lse = (m + total.log()).reshape(B, Hq, Nq)
    return o.to(q.dtype), lse


def _append(s):
    """The write, and the new tokens as the cache now has them (what a
    prompt's own attention reads)."""
    k, v, slots, cache = s["k"], s["v"], s["slots"], s["cache"]
    N, page, d = s["N"], s["page"], s["d"]
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        fa2.fa2_kv4_append(k, v, slots, cache, s["k_descale"], s["v_descale"])
        return fa2.fa2_kv4_gather(cache, s["block_table"], s["seq_lens"], s["k_descale"], s["v_descale"], N, d,
                                  starts=s["starts"], dtype=k.dtype)
    flat = slots.reshape(-1)
    keep = (flat >= 0).nonzero()[:, 0]
    at = flat[keep].long()
    pg, row = at // page, at % page
    i, g = torch.arange(d // 2, device=k.device), torch.arange(d // 16, device=k.device)
    for part, x, descale in ((0, k, s["k_descale"]), (1, v, s["v_descale"])):
        x = x.transpose(1, 2).reshape(-1, s["Hkv"], d)[keep].float()
        codes, scales = _quantise(x, descale[None, :])
        to = cache[:, :, part].permute(0, 2, 1)                                 # [pages, bytes, H]
        to[pg[:, None], row[:, None] * (d // 2) + i] = codes.transpose(1, 2)
        to[pg[:, None], page * (d // 2) + row[:, None] * (d // 16) + g] = scales.transpose(1, 2)
    return _read(s, s["starts"], N, k.dtype)


def _read(s, starts, N, dtype):
    page = s["page"]
    pos = starts[:, None] + torch.arange(N, device=starts.device)
    live = pos < s["seq_lens"][:, None]
    table = s["block_table"]
    at = (pos // page).clamp(max=table.shape[1] - 1).long()
    pg = table.gather(1, at).clamp(min=0).long()                                # [B, N]
    row = (pos % page).long()
    H, d = s["Hkv"], s["d"]
    out = []
    i, g = torch.arange(d // 2, device=pos.device), torch.arange(d // 16, device=pos.device)
    for part, descale in ((0, s["k_descale"]), (1, s["v_descale"])):
        src = s["cache"][:, :, part].permute(0, 2, 1)                           # [pages, bytes, H]
        codes = src[pg[..., None], row[..., None] * (d // 2) + i]               # [B, N, d/2, H]
        scales = src[pg[..., None], page * (d // 2) + row[..., None] * (d // 16) + g]
        one = torch.cat([codes, scales], 2).permute(0, 3, 1, 2).contiguous()    # [B, H, N, d/2 + d/16]
        one = one.transpose(1, 2).reshape(*pos.shape, H, -1)
        x = _values(one, descale, 1, d)[..., 0, :].transpose(1, 2)              # [B, H, N, d]
        out.append(x.masked_fill(~live[:, None, :, None], 0.0).to(dtype).contiguous())
    return out[0], out[1]


def _gather(s):
    dtype = DT[s["dtype"]]
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        return fa2.fa2_kv4_gather(s["cache"], s["block_table"], s["seq_lens"], s["k_descale"], s["v_descale"],
                                  s["max_len"], s["d"], dtype=dtype)
    N = s["max_len"]
    live = (torch.arange(N, device=s["seq_lens"].device) < s["seq_lens"][:, None])[:, None, :, None]
    k = _context(s, 0)[:, :, :N].masked_fill(~live, 0.0).to(dtype)
    return k, _context(s, 1)[:, :, :N].masked_fill(~live, 0.0).to(dtype)


def _plan(s):
    lens, new, table, ring, state = (s[n] for n in ("seq_lens", "new_lens", "block_table", "free_pages",
                                                    "free_state"))
    page, N = s["page"], s["N"]
    if own:
        from attention_fa2_forward_03_gb300 import fa2
        lens_out, accepted, slots, state_out = fa2.fa2_kv4_plan(lens, new, table, ring, state, page, N)
        return lens_out, accepted, slots, state_out, table, ring
    W, P = table.shape[1], ring.shape[0]
    lens, new = lens.long(), new.long()
    head, count = state[0].long(), state[1].long()
    have = (lens + page - 1) // page
    ends = new < 0
    fits = ~ends & (new <= N) & (lens + new <= W * page)
    need = torch.where(fits, (lens + new + page - 1) // page - have, 0)
    upto = need.cumsum(0)
    granted = fits & ((need == 0) | (upto <= count))
    accepted = torch.where(granted, new, 0)
    lens_out = torch.where(ends, 0, lens + accepted)
    j = torch.arange(W, device=lens.device)
    # pages of requests that end go behind the ring's last page
    rel = torch.where(ends, have, 0)
    at = (head + count + (rel.cumsum(0) - rel)[:, None] + j) % P
    back = ends[:, None] & (j < have[:, None])
    ring[at[back]] = table[back]
    at = (head + (upto - need)[:, None] + j - have[:, None]) % P
    fresh = granted[:, None] & (j >= have[:, None]) & (j < (have + need)[:, None])
    table.copy_(torch.where(fresh, ring[at], table))
    taken = torch.where(granted, need, 0).sum()
    state_out = torch.stack([(head + taken) % P, count - taken + rel.sum()]).int()
    i = torch.arange(N, device=lens.device)
    pos = lens[:, None] + i
    slot = table.gather(1, (pos // page).clamp(max=W - 1)).long() * page + pos % page
    slots = torch.where(i < accepted[:, None], slot, -1).int()
    return lens_out.int(), accepted.int(), slots, state_out, table, ring


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, B = case["op"], case["B"]
    if op == "plan":
        W = -(-(case["max_len"] + case["N"]) // case["page"])
        new = 1 if case["N"] == 1 else case["N"] * 3 // 4
        pages = -(-new // case["page"])
        # lengths in and out, slots out, the entries of the last and of the new pages
        return {"bytes": 4.0 * B * (4 + case["N"] + min(W, 1 + 2 * pages)), "flops": 0.0}
    H, d = case["Hkv"], case["d"]
    token = 2 * H * (d // 2 + d // 16)
    lens, _ = _lengths(case)
    if op == "append":
        n = sum(lens)
        # new tokens in, their cache bytes out and back, padded values out
        return {"bytes": 4.0 * n * H * d + 2.0 * n * token + 4.0 * B * case["N"] * (H * d + 1),
                "flops": 6.0 * n * H * d}
    if op == "gather":
        return {"bytes": 1.0 * sum(lens) * token + 4.0 * B * case["max_len"] * H * d, "flops": 4.0 * sum(lens) * H * d}
    rows = B * case["Hq"] * case["Nq"]
    return {"bytes": 1.0 * sum(lens) * token + rows * (4.0 * d + 4) + 4.0 * sum(-(-n // case["page"]) for n in lens),
            "flops": 4.0 * sum(lens) * case["Hq"] * case["Nq"] * d}


# ------------------------------------------------------------------ 64 bits

def _round_to(x, lowest, most, bits, top):
    """x >= 0 to the nearest of a format with `bits` fraction bits and
    exponents from `lowest` to `most`, ties to even, at most `top`."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** (lowest - 4)))).clamp(lowest, most)
    e = torch.where(x >= 2.0 ** (e + 1), e + 1, torch.where(x < 2.0 ** e, e - 1, e)).clamp(lowest, most)
    step = 2.0 ** (e - bits)
    return (torch.round(x / step) * step).clamp(max=top)


def _exact_codes(x, descale):
    """fp64 [..., d] as append's definition keeps it."""
    b = x.unflatten(-1, (-1, 16))
    s = _round_to(b.abs().amax(-1) / 6 / descale[..., None], -6, 8, 3, 448.0)[..., None]
    t = s * descale[..., None, None]
    y = torch.where(t > 0, b.abs() / t.clamp(min=1e-300), 0.0)
    return (_round_to(y, 0, 2, 1, 6.0) * b.sign() * t).flatten(-2)


def _exact_tokens(s, b, n, part):
    """fp64 [H, n, d]: request b's first n cached tokens, byte by byte."""
    page, d = s["page"], s["d"]
    pages = s["block_table"][b, : -(-n // page)].long()
    raw = s["cache"][pages, :, part].transpose(0, 1)                            # [H, pages, bytes]
    split = page * d // 2
    codes = raw[..., :split].reshape(raw.shape[0], -1, d // 2)[:, :n].to(torch.int16)
    sc = raw[..., split:].reshape(raw.shape[0], -1, d // 16)[:, :n].to(torch.int16)
    e, f = (sc >> 3) & 15, (sc & 7).double()
    scale = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e.double() - 7))
    out = torch.empty(raw.shape[0], n, d, dtype=torch.float64, device=raw.device)
    for odd in (0, 1):
        c = (codes >> (4 * odd)) & 15
        e, f = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e.double() - 1))
        out[..., odd::2] = torch.where(c > 7, -mag, mag)
    descale = (s["k_descale"], s["v_descale"])[part].double()
    return out * scale.repeat_interleave(16, -1) * descale[:, None, None]


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    dev, B = s["cache"].device, case["B"]
    if op == "append":
        new, _ = _lengths(case)
        out = []
        for x, descale in ((s["k"], s["k_descale"]), (s["v"], s["v_descale"])):
            y = torch.zeros(x.shape, dtype=torch.float64, device=dev)
            for b in range(B):
                y[b, :, : new[b]] = _exact_codes(x[b, :, : new[b]].double(), descale.double()[:, None])
            out.append(y)
        return out[0], out[1]
    lens, _ = _lengths(case)
    if op == "gather":
        out = []
        for part in (0, 1):
            y = torch.zeros(B, case["Hkv"], case["max_len"], case["d"], dtype=torch.float64, device=dev)
            for b in range(B):
                y[b, :, : lens[b]] = _exact_tokens(s, b, lens[b], part)
            out.append(y)
        return out[0], out[1]
    Hkv, Nq, d = case["Hkv"], case["Nq"], case["d"]
    G = case["Hq"] // Hkv
    o = torch.zeros(B, case["Hq"], Nq, d, dtype=torch.float64, device=dev)
    lse = torch.full((B, case["Hq"], Nq), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        k, v = _exact_tokens(s, b, n, 0), _exact_tokens(s, b, n, 1)
        x = torch.einsum("hgqd,hnd->hgqn", s["q"][b].double().reshape(Hkv, G, Nq, d), k) * s["scale"]
        for i in range(Nq):
            m = min(n, i + 1 + n - Nq) if case["causal"] else n
            if m <= 0:
                continue
            w = x[:, :, i, :m]
            z = torch.logsumexp(w, -1)
            lse[b, :, i] = z.reshape(-1)
            o[b, :, i] = torch.einsum("hgn,hnd->hgd", torch.exp(w - z[..., None]), v[:, :m]).reshape(-1, d)
    return o, lse
