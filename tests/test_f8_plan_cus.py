"""The choice of e4m3 kernel on devices and partitions of fewer CUs, asked on the host."""

import math
import random

import pytest

from tests.f8_plan import compiled

LAUNCH = {"few2": (32, 64, 512), "small": (64, 64, 192), "tall": (128, 64, 256), "square": (128, 128, 512),
          "wide": (256, 128, 512), "turns": (256, 256, 512)}     # rows, tokens and threads of a block


@pytest.fixture(scope="module")
def both(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("f8_plan_cus")))


def _threads(both, t, n, k, cut, cus):
    kernel = both[0](t, n, k, cut, cus)
    rows, tokens, threads = (both[1](t, n, cus), 64, 512) if kernel == "few1" else LAUNCH[kernel]
    return (-(-n // rows) * -(-t // tokens) + 8) * threads


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("cus", [1, 32, 64, 128, 256, 304])
def test_launches_fit(both, cus, cut):
    """Fewer than 2^32 threads in any launch that T <= 2^24, N <= 2^26, T * N <= 2^36 and
    N * K <= 2^38 allow: the borders, sizes that passed 2^32 once, and sizes even over the logarithm."""
    rng = random.Random(cus)
    sizes = [(1029, 65673803, 448), (16373863, 568, 127296), (1 << 24, 1 << 12, 131072), (1 << 10, 1 << 26, 4096)]
    for n in (1, 7, 16, 40, 130, 568, 1000, 4097, 8192, 1 << 20, 1 << 26):
        for t in (1, 16, 17, 32, 33, 64, 65, 1000, 1 << 14, 1 << 20, 1 << 24, (1 << 36) // n):
            sizes += [(t, n, k) for k in (16, 128, 2560, 28672, 131072)]
    for _ in range(20000):
        n = int(2 ** rng.uniform(0, 26))
        sizes.append((int(2 ** rng.uniform(0, min(24, 36 - math.log2(n)))), n, 16 * int(2 ** rng.uniform(0, 13))))
    for t, n, k in sizes:
        if t <= 1 << 24 and t * n <= 1 << 36 and n * k <= 1 << 38:
            assert _threads(both, t, n, k, cut, cus) < 1 << 32, (t, n, k)


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("t,n,k", [(2048, 6912, 2560), (250, 28672, 8192), (512, 8192, 28672), (128, 13942, 5136)])
def test_many_tokens_take_tiles_on_any_device(both, t, n, k, cut):
    """Both kinds of kernel take rounds over the CUs there are."""
    for cus in (32, 64, 128, 256):
        assert not both[0](t, n, k, cut, cus).startswith("few")
