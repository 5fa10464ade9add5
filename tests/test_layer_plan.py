"""How a whole routed layer runs, asked on the host: the GPU tests' sizes reach
every kernel and both sides of every choice."""

import pytest

from tests.layer_cases import DOWN, GATE, LIMITS
from tests.layer_plan import compiled

CUS = 256
RAW = (0, 2, 4)


@pytest.fixture(scope="module")
def both(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("layer_plan")))


def _quads(k):
    return "words" if k < 64 else "short" if k % 64 else "whole"


def test_gate_cases_reach_every_kernel(both):
    plan, depth = both
    seen = set()
    for case in GATE:
        for raw in RAW:
            p = plan(*case, raw, CUS)
            assert p.two and not p.own_quant, case
            seen.add((raw, p.pairs, p.gate_waves, _quads(case[4]), depth(case[4])))
    rows = [("words", 2)] + [(q, d) for q in ("short", "whole") for d in (2, 4, 6, 8, 10)]
    assert seen == {(raw, *blocks, *row) for raw in RAW for blocks in ((0, 4), (0, 8), (1, 4)) for row in rows}


def test_down_cases_reach_every_kernel(both):
    plan, _ = both
    seen, ends, teams = set(), set(), set()
    for case in DOWN:
        p, f, n = plan(*case, 0, CUS), case[3], case[5]
        assert p.two, case
        seen.add((p.down_tiles, _quads(f), p.team > 1))
        if p.down_tiles == 2:
            ends.add((_quads(f), p.team > 1, 0 if n % 32 == 0 else 1 if n % 32 <= 16 else 2))
            teams.add(p.team)
    for q, team in (("words", False), ("short", False), ("whole", False), ("short", True), ("whole", True)):
        assert (2, q, team) in seen
        assert {e for a, b, e in ends if (a, b) == (q, team)} == {0, 1, 2}, (q, team)
    for q in ("short", "whole"):
        assert (1, q, True) in seen or q == "whole"      # whole ones of 16 outputs: test_layer_gpu.py
    assert teams == {1, 2, 3, 4, 8}


def test_limits_have_both_sides(both):
    plan, _ = both
    two = [plan(*case, 0, CUS).two for case in LIMITS]
    assert two[:8] == [1, 0, 1, 0, 0, 0, 1, 0] and all(two[8:])
    own = [[plan(*case, raw, CUS).own_quant for raw in RAW] for case in LIMITS[8:]]
    assert own == [[0, 0, 1], [0, 1, 1], [0, 0, 0], [0, 0, 1], [0, 0, 1], [0, 1, 1]]


def test_launches_fit(both):
    """Blocks of at most 1024 threads and 150 KiB, and grids of fewer than 2^32 threads in a row."""
    plan, _ = both
    for cus in (1, 32, 256):
        for t in (1, 2, 4, 5, 6, 16):
            for e in (1, 2, 16, 64, 256):
                for k in (1, 2, 3, 8, 16):
                    for f in (16, 64, 1024, 1040, 9472, 131072):
                        for kk in (16, 64, 2560, 9472, 131072):
                            for n in (1, 1 << 20, (1 << 25) - 1, 1 << 25):
                                for raw in RAW:
                                    p = plan(t, e, k, f, kk, n, raw, cus)
                                    if not p.two or k > e:
                                        continue
                                    stride = lambda v: -(-v // 256) * 256 + 16  # noqa: E731
                                    use = 0 if p.own_quant else raw
                                    assert t * (stride(kk) + use * kk) <= 150 * 1024 >= k * stride(f)
                                    assert p.gate_waves in (4, 8) and not (p.pairs and (t > 4 or p.gate_waves != 4))
                                    assert p.team >= 1 and 64 * k * p.team <= 1024 and p.down_tiles in (1, 2)
                                    assert -(-n // (16 * p.down_tiles)) * 1024 < 1 << 32
