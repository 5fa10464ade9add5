"""Sums of the e4m3 product in whole numbers (needs an MI355X): products of codes
that are whole numbers, whose magnitudes add to less than 2^24, so every partial
sum is exact in binary32 in any order, and an output is the sum rounded once to
its type.  Large products that cancel stand next to small ones, where a sum in
fewer bits loses the small ones.  Where the caller allows such a sum, the
tolerance is the one stated for it."""

import numpy as np
import pytest
import torch

from oracle import f8_ref as ref
from tests.f8_cases import SHAPES

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bl(built_lib):
    import bitlinear_w1_a8_amd as bl
    return bl


def _whole(t, n, k):
    """Codes x [T, K] and w [N, K]: -3 .. 3 and -4 .. 4, but two products of 2^14 that cancel in
    every 16 k (64 in long rows).  Also the sum of the products' magnitudes at most."""
    g = torch.Generator(device="cuda").manual_seed(t + 3 * n + 7 * k)
    x = torch.randint(-3, 4, (t, k), generator=g, device="cuda").float()
    w = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float()
    every = 16 if k <= 6912 else 64
    pairs = torch.arange(0, k, every, device="cuda")
    sx, sw = (1.0 - 2 * torch.randint(0, 2, (rows, pairs.numel()), generator=g, device="cuda") for rows in (t, n))
    x[:, pairs], x[:, pairs + 1] = 256 * sx, -256 * sx
    w[:, pairs] = w[:, pairs + 1] = 64 * sw
    return x, w, 2 * pairs.numel() * (1 << 14) + 12 * k


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_whole_numbers(bl, t, n, k):
    x, w, size = _whole(t, n, k)
    assert size < 1 << 24
    blocks = (k + 127) // 128
    args = (w.to(F8), torch.ones((n + 127) // 128, blocks, device="cuda"), x.to(F8),
            torch.ones(blocks, t, device="cuda"))
    want = x.double().cpu() @ w.double().cpu().t()
    y = bl.forward_f8(*args)
    assert torch.equal(y.cpu().double(), want)
    b = bl.forward_f8(*args, dtype=torch.bfloat16)
    assert torch.equal(b.cpu(), want.float().bfloat16())


def _random(t, n, k):
    """All codes that are numbers, scales between 1/2 and 2; on the host."""
    rng = np.random.default_rng(5 * t + 11 * n + k)
    live = np.array([b for b in range(256) if b & 127 != 127], np.uint8)
    blocks = (k + 127) // 128
    return (live[rng.integers(0, 254, (n, k))], rng.uniform(0.5, 2, ((n + 127) // 128, blocks)).astype(np.float32),
            live[rng.integers(0, 254, (t, k))], rng.uniform(0.5, 2, (blocks, t)).astype(np.float32))


def _cuda(w, ws, x, xs):
    return (torch.from_numpy(w).cuda().view(F8), torch.from_numpy(ws).cuda(), torch.from_numpy(x).cuda().view(F8),
            torch.from_numpy(xs).cuda())


def _near(y, want, size, k):
    """7 * 2^-13 of the magnitudes for the cut, 128 * 2^-23 and (blocks + 18) * 2^-24 for the additions in
    binary32, 2^-8 for the output's rounding."""
    sums = 7 * 2.0 ** -13 + 128 * 2.0 ** -23 + ((k + 127) // 128 + 18) * 2.0 ** -24
    assert y.dtype == torch.bfloat16
    assert np.all(np.abs(y.float().cpu().numpy() - want) <= size * sums * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8)


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_bfloat16_is_the_binary32_result_rounded(bl, t, n, k):
    """The same kernels and order for either type of output; up to 16 tokens the caller's leave to
    cut sums changes nothing."""
    args = _cuda(*_random(t, n, k))
    y = bl.forward_f8(*args).bfloat16()
    assert torch.equal(bl.forward_f8(*args, dtype=torch.bfloat16), y)
    if t <= 16:
        assert torch.equal(bl.forward_f8(*args, dtype=torch.bfloat16, sums="cut"), y)


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_cut_sums(bl, t, n, k):
    host = _random(t, n, k)
    args = _cuda(*host)
    want, size = ref.forward_f8(*host)
    y = bl.forward_f8(*args, dtype=torch.bfloat16, sums="cut")
    _near(y, want, size, k)
    assert torch.equal(bl.forward_f8(*args, dtype=torch.bfloat16, sums="cut"), y)


@pytest.mark.parametrize("t,n,k", [(20, 40, 272), (130, 6002, 128), (300, 16504, 128), (1100, 8200, 128), (1030, 8193, 144)])
def test_cut_sums_at_any_element(bl, t, n, k):
    """Outputs aligned to their element only, and nothing around them written."""
    args = _cuda(*_random(t, n, k))
    want = bl.forward_f8(*args, dtype=torch.bfloat16, sums="cut")
    buf = torch.full((t * n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    for at in (1, 3):
        bl.forward_f8(*args, out=buf[at:at + t * n].view(t, n), sums="cut")
        assert torch.equal(buf[at:at + t * n].view(t, n), want)
        assert torch.all(buf[:at] == 7) and torch.all(buf[at + t * n:] == 7)
        buf[:] = 7


def test_linear_and_graph(bl):
    w, ws, _, _ = _cuda(*_random(1, 8200, 400))
    raw = torch.randn(1100, 400, device="cuda")
    xq, xs = bl.quant_act_f8(raw)
    bf16 = dict(dtype=torch.bfloat16)
    want = [bl.forward_f8(w, ws, xq, xs, **bf16), bl.forward_f8(w, ws, xq, xs, sums="cut", **bf16)]
    assert torch.equal(want[0], bl.linear_f8(raw, w, ws, **bf16))
    assert torch.equal(want[1], bl.linear_f8(raw, w, ws, sums="cut", **bf16))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [bl.linear_f8(raw, w, ws, **bf16), bl.linear_f8(raw, w, ws, sums="cut", **bf16)]
    for _ in range(3):
        got[0].zero_(), got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(bl.forward_f8(w, ws, xq, xs, **bf16), want[0])
