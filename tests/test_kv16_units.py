"""The sums by which attention over the paged 16-bit KV cache cuts its work, compiled
for the host from the kernel's source and compared with counting (CPU only)."""
import ctypes
import os
import random
import re
import subprocess

import pytest

from attention_fa2_forward_03_gb300 import build

HOST = """
#include <algorithm>
#define __device__
#define __forceinline__ static
#define __popc __builtin_popcount
using std::min;
constexpr int kBN = 128;
%s
extern "C" int tiles(int n, int keys, int step) { return tiles_of_blocks(n, keys, step); }
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    with open(os.path.join(build.CSRC, "fa2_kv16_sm103.cuh")) as f:
        body = re.search(r"__device__ __forceinline__ int tiles_of_blocks\(.*?\n}\n", f.read(), re.S)[0]
    at = tmp_path_factory.mktemp("units")
    (at / "u.cpp").write_text(HOST % body)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-o", at / "u.so", at / "u.cpp"], check=True)
    return ctypes.CDLL(str(at / "u.so")).tiles


def counted(n, keys, step):
    return sum((keys + i * step + 127) // 128 for i in range(n))


STEPS = sorted({2 * (128 // group) for group in range(1, 129)})


@pytest.mark.parametrize("step", STEPS)
def test_tiles_of_every_step(tiles, step):
    rng = random.Random(step)
    for keys in [*range(1, 260), *(rng.randrange(1, 1 << 20) for _ in range(20))]:
        for n in (1, 2, 3, rng.randrange(1, 200), 63, 64, 65, 128):
            assert tiles(n, keys, step) == counted(n, keys, step)


@pytest.mark.parametrize("step,n,keys", [
    (256, 13000, 1), (256, 20, (1 << 31) - 257 - 20 * 256), (2, 200000, 5), (2, 1 << 17, 127), (84, 26000, 77), (50, 40000, 3),
    (254, 9, (1 << 31) - 257 - 9 * 254), (128, 19000, 128),
])
def test_tiles_of_the_longest(tiles, step, n, keys):
    """Up to what the host lets through: 2^30 units, three a tile, and 2^31 - 256 tokens."""
    want = counted(n, keys, step)
    assert 3 * want <= 2 ** 30 and keys + (n - 1) * step < 2 ** 31 - 256   # the host's bounds
    assert tiles(n, keys, step) == want
