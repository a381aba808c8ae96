"""Pages that ended requests give back, ids outside the cache among them."""
import numpy as np
import pytest
import torch

from oracle import kv4


def test_oracle_leaves_bad_ids_out_of_the_ring():
    table = np.array([[9, -1, 7], [3, 12, 2]])
    ring = np.array([4, 5, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0])
    lens, acc, slots, state, _, r = kv4.plan([33, 48], [-1, -1], table, ring, [0, 2], 16, 1)
    assert lens == [0, 0] and state == [0, 6] and list(r[:6]) == [4, 5, 9, 7, 3, 2]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,page,W,seed", [
    (1, 1, 16, 300, 0), (40, 1, 64, 30, 1), (300, 1, 16, 8, 2), (2100, 3, 16, 3, 3), (33, 257, 32, 140, 4),
    (1100, 300, 128, 5, 5), (70, 515, 64, 12, 6),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_bad_ids_of_requests_that_end(gpu_lib, B, N, page, W, seed, in_place):
    """They are reported by the call that ends their request and none joins the
    ring; the next call hands out pages of the cache only, without a report."""
    fa2 = gpu_lib
    rng = np.random.default_rng(seed)
    stream = torch.cuda.current_stream().cuda_stream
    lens = rng.integers(1, W * page + 1, B)
    new = np.where(rng.random(B) < 0.4, -1, rng.integers(0, N + 1, B))
    new[B // 2] = -1
    have = -(-lens // page)
    P = int(have.sum()) + B + 5
    ids = rng.permutation(P)
    table = np.full((B, W), -7)
    at = 0
    for b in range(B):
        table[b, : have[b]] = ids[at: at + have[b]]
        at += have[b]
    ends = np.flatnonzero(new < 0)
    for b in ends[:: 2] if len(ends) > 1 else ends:
        bad = rng.permutation(have[b])[: rng.integers(1, have[b] + 1)]
        table[b, bad] = rng.choice([-1, P, 2 ** 31 - 1, -2 ** 31], len(bad))
    free, first = P - at, int(rng.integers(0, P))
    ring = np.full(P, -9)
    ring[(first + np.arange(free)) % P] = ids[at: at + free]
    want = kv4.plan(lens, new, table, ring, [first, free], page, N)
    t, r, ln, st = i32(table), i32(ring), i32(lens), i32([first, free])
    kw = {"seq_lens_out": ln, "free_state_out": st} if in_place else {}
    got = fa2.fa2_kv4_plan(ln, i32(new), t, r, st, page, N, **kw)
    assert fa2.fa2_check_status(stream) == fa2.FA2_ERR_BOUNDS
    for x, y in zip((*got, t), want):
        assert np.array_equal(x.cpu().numpy(), np.asarray(y))
    live = (want[3][0] + np.arange(want[3][1])) % P      # the other places hold nothing that is read
    assert np.array_equal(r.cpu().numpy()[live], want[5][live])
    # everything that is free is handed out, and every id is a page of its own
    count = int(got[3][1])
    t2 = torch.full((count, 1), -1, dtype=torch.int32, device="cuda")
    fa2.fa2_kv4_plan(i32(np.zeros(count)), i32(np.ones(count)), t2, r, got[3], page, 1)
    assert fa2.fa2_check_status(stream) == fa2.FA2_OK
    out = t2.cpu().numpy()[:, 0]
    assert len(set(out.tolist())) == count and out.min() >= 0 and out.max() < P
