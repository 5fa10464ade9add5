"""Which kernel a 4-bit product takes, asked on the host."""

import pytest

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
