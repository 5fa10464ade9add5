"""Every kernel variant of the 4-bit product against the definition in binary64
(needs an MI355X; test_w4_plan shows that the cases reach them).

Bound as in test_w4_gpu: each group's sum is exact, its product with the scale
and the additions round once each (fused), over the K / G groups and at most
36 joins of partial sums, absmax / 127 and the last product once each: within
(K / G + 40) u of the sum of |s * group sum| * m / 127, u = 2^-24."""

import pytest
import torch

from tests import w4_cases

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def bl(built_lib):
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import bitlinear_w1_a8_amd
    bitlinear_w1_a8_amd.load()
    return bitlinear_w1_a8_amd


def inputs(t, n, k, g, with_zeros):
    gen = torch.Generator("cuda").manual_seed(t + n + k + g)
    kp = -(-k // 128) * 128
    packed = torch.randint(0, 256, (n, kp // 2), generator=gen, device="cuda", dtype=torch.uint8)
    packed[0] = 0x88                                          # codes of -8: the largest sums
    for at in range(k, kp):                                   # nibbles past K are 0
        byte, shift = w4_cases.ref.place(at)
        packed[:, byte] &= 15 if shift else 240
    scales = (0.002 + 0.018 * torch.rand(n, k // g, generator=gen, device="cuda")).bfloat16()
    zeros = None
    if with_zeros:
        zeros = torch.randint(-8, 8, (n, k // g), generator=gen, device="cuda", dtype=torch.int8)
        zeros[0] = 7
    xq = (40 * torch.randn(t, k, generator=gen, device="cuda")).round().clamp(-127, 127).to(torch.int8)
    absmax = 0.1 + 4 * torch.rand(t, generator=gen, device="cuda")
    if t > 1:
        xq[1] = 127
    absmax[-1] = 0.0
    return packed, scales, zeros, xq, absmax


@pytest.mark.parametrize("with_zeros", [False, True], ids=["sym", "zp"])
@pytest.mark.parametrize("t,n,k,g", w4_cases.CASES, ids=["T%d_N%d_K%d_g%d" % c for c in w4_cases.CASES])
def test_forward(bl, t, n, k, g, with_zeros):
    packed, scales, zeros, xq, absmax = inputs(t, n, k, g, with_zeros)
    whole = torch.full((t + 2, n), 5.0, device="cuda")        # a row before and one behind the output
    y = bl.forward_w4(packed, scales, xq, absmax, zeros=zeros, out=whole[1:-1])
    assert bool((whole[0] == 5).all()) and bool((whole[-1] == 5).all())
    want, size = w4_cases.forward(packed, scales, zeros, xq, absmax)
    assert bool(((y.double() - want).abs() <= (k // g + 40) * U * size).all())
    assert torch.equal(bl.forward_w4(packed, scales, xq, absmax, zeros=zeros), y)
