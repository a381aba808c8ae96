"""What bf16 query rows of the attention over the 4-bit cache lose: nothing
down to 2^-31 of a row's largest element, 2^-39 of that below."""
import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 20, 40])
@pytest.mark.parametrize("low,off", [(-31, 0.0), (-38, 2.0 ** -39)])
def test_elements_far_below_their_rows_largest(gpu_lib, rows, low, off):
    """The largest element, 1 to 2, meets keys of 0, so that the scores come
    from those down to 2^low of it alone. One token: LSE is its score. The sum of 48
    products in fp32 is off by 48 * 2^-23 of their magnitudes, the factors by 2^-21 of the
    score."""
    fa2 = gpu_lib
    rng = np.random.default_rng(rows - low)
    d, page = 64, 16
    cache = rng.integers(0, 256, (1, 1, 2, page * (d // 2 + d // 16)), dtype=np.uint8)
    cache[..., page * d // 2:] = rng.integers(0x28, 0x48, page * d // 16, dtype=np.uint8)
    cache[..., 0, : 8] = 0                               # codes of elements 0 .. 15 of the first token
    q = np.exp2(rng.uniform(low, low + 4, (1, rows, 1, d))) * rng.choice([-1.0, 1.0], (1, rows, 1, d))
    q[..., 0] = rng.uniform(1, 2, (1, rows, 1))
    q = torch.tensor(q).to(torch.bfloat16)
    q[..., 1:] = torch.where(q[..., 1:].abs() < q[..., :1] * 2.0 ** low, q[..., 1:] * 2, q[..., 1:])
    scale = 2.0 ** (-low - 4)
    one, table = torch.ones(1, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    _, lse = fa2.fa2_fwd_kv4(q.cuda(), torch.tensor(cache).cuda(), table, table[0] + 1, one, one, scale=scale)
    assert fa2.fa2_check_status(torch.cuda.current_stream().cuda_stream) == fa2.FA2_OK
    k = kv4.tokens(cache, d, [0], 1, 0, 0, 1.0)[0]
    assert not k[:16].any() and k[16:].any()
    x = q.double().numpy()[0, :, 0]
    want, size = scale * (x @ k), scale * (np.abs(x) @ np.abs(k))
    bound = 48 * 2.0 ** -23 * size + 2.0 ** -21 * np.abs(want) + 2.0 ** -21 + scale * off * x[:, 0] * np.abs(k).sum()
    assert np.all(np.abs(lse[0, :, 0].double().cpu().numpy() - want) <= bound)
