"""The whole routed layer at sizes that reach every kernel of its two launches
and both sides of their limits (needs an MI355X), bit for bit with the router, the gated
and the linear calls one after the other; tokens without an expert among them."""

import pytest
import torch

from tests.layer_cases import DOWN, GATE, LIMITS
from tests.test_layer_gpu import BF16, F32, Layer, _check, _tokens, bl  # noqa: F401

pytestmark = pytest.mark.gpu


def _run(bl, t, e, k, f, kk, n):  # noqa: F811
    layer = Layer(bl, e, f, kk, n)
    for logits, x, share in ((F32, BF16, "chosen"), (BF16, F32, "all")):
        x, l = _tokens(t, kk, e, logits, x)
        _check(bl, layer, x, l, k, share)
        if t > 2:
            l[t // 2] = float("-inf")            # a token of no expert, and one of a single one
            l[t - 1, 1:] = float("-inf")
            _check(bl, layer, x, l, k, share)


@pytest.mark.parametrize("t,e,k,f,kk,n", GATE)
def test_gate(bl, t, e, k, f, kk, n):  # noqa: F811
    _run(bl, t, e, k, f, kk, n)


@pytest.mark.parametrize("t,e,k,f,kk,n", DOWN)
def test_down(bl, t, e, k, f, kk, n):  # noqa: F811
    _run(bl, t, e, k, f, kk, n)


@pytest.mark.parametrize("t,e,k,f,kk,n", LIMITS)
def test_limits(bl, t, e, k, f, kk, n):  # noqa: F811
    _run(bl, t, e, k, f, kk, n)


@pytest.mark.parametrize("n", [1025, 1041, 1056])
def test_neighbours_untouched(bl, n):  # noqa: F811
    """32 outputs per block: nothing before, between or behind the outputs is written."""
    layer = Layer(bl, 12, 80, 64, n)
    x, l = _tokens(16, 64, 12)
    buf = torch.full((16 * n + 64,), 7.0, device="cuda")
    y = buf[32:-32].view(16, n)
    assert layer(x, l, 3, out=y) is y
    assert torch.equal(y, layer.calls(x, l, 3))
    assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)
