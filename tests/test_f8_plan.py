"""Which kernel an e4m3 product takes, asked on the host."""

import pytest

from tests.f8_cases import SHAPES
from tests.f8_plan import KERNELS, compiled

CUS = 256


@pytest.fixture(scope="module")
def both(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("f8_plan")))


@pytest.fixture(scope="module")
def plan(both):
    return both[0]


def test_cases_reach_every_kernel(both):
    """Both output types, whole and partial last blocks of K; of the streaming
    kernel every number of token tiles and of rows per block."""
    plan, rows = both
    seen = set()
    for t, n, k in SHAPES:
        for bf16 in (False, True):
            kernel = plan(t, n, k, bf16, CUS)
            seen.add((kernel, bf16, k % 128 != 0))
            if kernel.startswith("few"):
                tiles = 1 if t <= 16 else 2 if t <= 32 else 4
                seen.add((kernel, bf16, tiles))
                if kernel == "few1":
                    seen.add((bf16, tiles, rows(t, n, CUS)))
    for bf16 in (False, True):
        for kernel in KERNELS[:7 if bf16 else 6]:
            for tail in (False, True):
                assert (kernel, bf16, tail) in seen, (kernel, bf16, tail)
        for few in (("few1", 1), ("few1", 2), ("few1", 4), ("few2", 2)):
            assert (few[0], bf16, few[1]) in seen, (few, bf16)
        for tiles in (1, 2, 4):
            # (bfloat16 outputs of more than 32 tokens take tiles from about 2000 rows on)
            for per in (4, 8) if bf16 and tiles == 4 else (4, 8, 12, 16):
                assert (bf16, tiles, per) in seen, (bf16, tiles, per)


KS = (16, 128, 2560, 28672, 131072)


def test_binary32_outputs_never_take_the_e4m3_only_kernel(plan):
    for t in (1, 33, 64, 200, 1024, 4096, 1 << 24):
        for n in (1, 100, 2560, 28672, 128256, 1 << 26):
            for k in KS:
                assert plan(t, n, k, False, CUS) != "turns"


def test_few_tokens_stream(plan):
    for t in range(1, 17):
        for n in (1, 640, 128256, 1 << 26):
            for k in KS:
                assert plan(t, n, k, True, CUS) == plan(t, n, k, False, CUS) == "few1"


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [1, 7, 16, 40, 130, 1000, 4097, 8192, 1 << 20, 1 << 26])
def test_launches_fit(both, n, bf16):
    """Fewer than 2^32 threads in any launch that T * N <= 2^36 allows."""
    plan, few_rows = both
    for t in (1, 16, 17, 32, 33, 64, 65, 1000, 1 << 14, 1 << 20, 1 << 24):
        if t * n > 1 << 36:
            continue
        for k in KS:
            kernel = plan(t, n, k, bf16, CUS)
            rows, tokens, threads = {"few1": (few_rows(t, n, CUS), 64, 512), "few2": (32, 64, 512), "small": (64, 64, 192),
                                     "tall": (128, 64, 256), "square": (128, 128, 512),
                                     "wide": (256, 128, 512), "turns": (256, 256, 512)}[kernel]
            assert (-(-n // rows) * -(-t // tokens) + 8) * threads < 1 << 32, (kernel, t, n, k)


def test_rows_per_block(both):
    """Multiples of four, no more blocks than CUs below 16 rows."""
    for cus in (1, 64, 256):
        for n in (1, 4, 1024, 1025, 2048, 2049, 4095, 4096, 1 << 26):
            for t in (1, 64, 65, 1000, 1 << 24):
                lots, rows = -(-t // 64), both[1](t, n, cus)
                assert rows in (4, 8, 12, 16) and (rows == 16 or -(-n // rows) * lots <= cus)
                assert rows == 4 or -(-n // (rows - 4)) * lots > cus
