"""Sizes that the attention over the 4-bit cache refuses: fa2_fwd_kv4 and
fa2_fwd_kv4_workspace say the same, before any device is touched; and those that
the plan refuses (CPU only)."""
import pytest

from attention_fa2_forward_03_gb300 import build, fa2

A = 1 << 20   # a 16-byte aligned fake address: never dereferenced on these paths
UNS = 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa2.load()


@pytest.mark.parametrize("B,Hq,Hkv,Nq,d,max_pages,page", [
    (1, 1, 1, 2 ** 31 - 64, 64, 10, 16), (2 ** 16, 2 ** 15, 2 ** 14, 1, 64, 10, 16),   # rows
    (2 ** 31 - 1, 2 ** 15 - 1, 2 ** 15 - 1, 2 ** 31 - 1, 128, 2 ** 24 - 3, 128),   # products of four sizes
    (1, 2 ** 15, 2 ** 15, 1, 64, 10, 16),                     # heads whose page passes 32 bits
    (2, 32, 32, 1, 128, 2 ** 24 - 3, 128),                    # tiles of all segments
    (2 ** 15, 2 ** 10, 2 ** 10, 1, 128, 33, 32),              # 33 tiles for 2^25 segments
    (1, 1, 1, 2 ** 20 * 64, 128, 2 ** 9 + 1, 64),             # 2^20 blocks of rows, 1026 tiles each
    (1, 8, 8, 1, 96, 10, 64), (1, 8, 8, 1, 128, 10, 48), (1, 8, 8, 1, 128, 2 ** 26, 64),
])
def test_what_the_forward_refuses_needs_no_workspace(B, Hq, Hkv, Nq, d, max_pages, page):
    assert fa2.fa2_fwd_kv4_workspace(B, Hq, Hkv, Nq, d, max_pages, page) == -1
    args = [A] * 9 + [1 << 62, B, Hq, Hkv, Nq, d, max_pages, page, 100, 0.1, 0, 0]
    assert fa2.fa2_fwd_kv4_ptr(*args) == UNS


@pytest.mark.parametrize("B,Hq,Hkv,Nq,d,max_pages,page", [
    (1, 1, 1, 2 ** 31 - 65, 64, 2, 16), (1, 2 ** 15 - 1, 2 ** 15 - 1, 1, 64, 10, 16), (1, 16, 16, 1, 128, 2 ** 24 - 3, 128),
    (2 ** 15, 2 ** 10, 2 ** 10, 1, 128, 32, 32), (1, 1, 1, 2 ** 20 * 64, 128, 2 ** 9, 64),
])
def test_the_largest_sizes_have_a_workspace(B, Hq, Hkv, Nq, d, max_pages, page):
    assert fa2.fa2_fwd_kv4_workspace(B, Hq, Hkv, Nq, d, max_pages, page) >= 0


@pytest.mark.parametrize("B,N", [(2 ** 31 - 1, 1), (2 ** 31 - 1023, 1), (1, 2 ** 31 - 1), (1, 2 ** 31 - 1023), (2, 2 ** 30 - 511)])
def test_plan_refuses_counts_that_its_steps_would_carry_past_32_bits(B, N):
    """The kernel counts requests by up to 1024 and slots by 256 in 32 bits."""
    assert fa2.fa2_kv4_plan_ptr(*[A] * 9, B, N, 10, 64, 100) == UNS
