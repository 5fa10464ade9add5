"""Which kernel a 4-bit product takes, asked on the host."""

import numpy as np
import pytest
import torch

from bitlinear_w1_a8_amd import workloads as wl
from oracle import w4_ref as ref
from tests import w4_cases
from tests.w4_plan import compiled

CUS = 256


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("w4_plan")))


def passes(p, t):
    """Times that a product reads its matrix."""
    return 1 if p.wn else -(-t // p.tokens)


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("n", [16, 1024, 2560, 4096, 8192, 28672, 128256])
@pytest.mark.parametrize("k", [128, 2560, 8192, 9600, 10240, 14336, 28672, 65536, 131072])
def test_no_batch_reads_the_matrix_many_times(plan, n, k, g):
    """A token more never takes the product from several passes over the matrix
    to one: two passes at most, and those only for matrices whose 16-row tiles leave
    CUs idle."""
    for t in range(1, 18):
        p = plan(t, n, k, g, CUS)
        assert passes(p, t) <= (2 if n < 16 * CUS else 1), (t, p)


def test_few_tokens_in_one_pass_stream(plan):
    for t in range(1, 17):
        p = plan(t, 2560, 6912, 64, CUS)
        assert p.wn == 0 and p.tokens == 16
    assert plan(17, 2560, 6912, 64, CUS).wn
    assert plan(1, 1024, 131072, 128, CUS).wn == 0      # the longest row, alone


def test_team_splits_no_further_than_load_groups(plan):
    for t in (1, 2, 16):
        for n in (1, 500, 5000, 20000, 40000):
            for k in (128, 512, 640, 1024, 2560, 8192):
                team = plan(t, n, k, 128, CUS).team
                assert team in (1, 2, 4, 8) and (team == 1 or 4 * (team // 2) < -(-k // 128))


def test_cases_reach_every_variant(plan):
    """Every kernel that the rule can choose has a case in w4_cases, with all
    group sizes, whole and partial tiles, whole and half last blocks, and every
    remainder of the three stages."""
    for (wn, wk, wmf), shapes in w4_cases.TILED.items():
        groups, stages = set(), set()
        for t, n, gk in shapes:
            assert t > 32 * wmf and t % (32 * wmf) and n > 32 * wn and n % (32 * wn)
            for g, k in gk:
                assert plan(t, n, k, g, CUS)[:3] == (wn, wk, wmf)
                groups.add((g, k % 128 != 0))
                stages.add(-(-(-(-k // 128)) // wk) % 3)
        whole = {(128, False)} if wmf == 4 else {(32, False), (64, False), (128, False), (32, True), (64, True)}
        assert groups >= whole, (wn, groups)
        assert stages == {0, 1, 2}, (wn, wk, wmf, stages)
    few = {(t > 1, g, plan(t, n, k, g, CUS).team) for t, n, k, g in w4_cases.FEW}
    assert all(plan(t, n, k, g, CUS).wn == 0 for t, n, k, g in w4_cases.FEW)
    assert few >= {(many, g, team) for many in (False, True) for g in (32, 64, 128) for team in (1, 2, 4, 8)}
    for t, n, k, g in w4_cases.PASSES:
        assert passes(plan(t, n, k, g, CUS), t) == 2
    assert any(t % plan(t, n, k, g, CUS).tokens == 1 for t, n, k, g in w4_cases.PASSES)
    assert {plan(t, n, k, g, CUS)[:3] for t, n, k, g in w4_cases.LONG} == {(1, 8, 1), (2, 4, 1)}


def test_variants_are_all_that_the_rule_gives(plan):
    """The rule over a grid of sizes gives no variant that has no case."""
    seen = {plan(t, n, k, g, CUS)[:3] for t in (1, 2, 9, 16, 17, 40, 64, 100, 300, 700, 2048, 9000)
            for n in (1, 33, 500, 2560, 4096, 6912, 30000, 128256) for k in (128, 2560, 8192, 28672, 131072)
            for g in (32, 64, 128)}
    assert seen == set(w4_cases.TILED) | {(0, 0, 0)}


@pytest.mark.parametrize("with_zeros", [False, True])
@pytest.mark.parametrize("t,n,k,g", [(3, 9, 416, 32), (1, 5, 320, 64), (4, 7, 256, 128)])
def test_reference_is_the_oracles(t, n, k, g, with_zeros):
    rng = np.random.default_rng(k)
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    s = wl.bf16_bits(rng.uniform(0.002, 0.02, (n, k // g)).astype(np.float32))
    z = rng.integers(-8, 8, (n, k // g)).astype(np.int8) if with_zeros else np.zeros((n, k // g), np.int8)
    q = rng.integers(-127, 128, (t, k)).astype(np.int8)
    a = rng.uniform(0, 4, t).astype(np.float32)
    a[0] = 0.0
    want, size = ref.forward(codes, s, z, q, a)
    got, gsize = w4_cases.forward(torch.from_numpy(ref.pack(codes)),
                                  torch.from_numpy(s.view(np.int16)).view(torch.bfloat16),
                                  torch.from_numpy(z) if with_zeros else None, torch.from_numpy(q), torch.from_numpy(a))
    assert np.allclose(got.numpy(), want, rtol=1e-14, atol=0) and np.allclose(gsize.numpy(), size, rtol=1e-14, atol=0)


def test_team_fills_the_device(plan):
    """No team is half as large as it could be with its blocks of eight waves
    still one per CU (two for one token)."""
    for t in (1, 2, 5, 16):
        for n in (16, 2560, 4080, 4096, 4112, 6912, 8192, 8208, 16384, 16400, 32768, 32784):
            for k in (512, 1280, 2560, 8192, 28672):
                p = plan(t, n, k, 128, CUS)
                if p.wn or p.team == 8 or -(-k // 128) <= 4 * p.team:
                    continue
                assert -(-n // 16) * 2 * p.team / 8 > (2 if t == 1 else 1) * CUS, (t, n, k, p)


def test_wide_cases_reach_the_larger_tiles(plan):
    assert [plan(t, n, k, g, CUS)[:3] for t, n, k, g in w4_cases.WIDE] == [(4, 2, 1), (4, 1, 1), (4, 1, 2), (8, 1, 4)]
