"""What the routed-expert calls leave allocated (needs an MI355X)."""

import pytest
import torch

from tests.test_experts_gpu import bl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,e,k", [(1, 64, 8), (64, 128, 8), (65, 1024, 1), (4096, 256, 2)])
def test_a_routing_holds_no_scratch(bl, t, e, k):  # noqa: F811
    """The router's outputs keep their own bytes alive and none of the workspace's."""
    logits = torch.randn(t, e, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    r = bl.route_experts(logits, k)
    for v in (r.ids, r.slots, r.pairs, r.offsets):
        assert v.untyped_storage().nbytes() == 4 * (3 * t * k + e + 1)
    assert r.weights.untyped_storage().nbytes() == 4 * t * k


def test_scratch_of_two_calls_at_once(bl):  # noqa: F811
    """Calls on two streams, their scratch handed back while they run."""
    gen = torch.Generator("cuda").manual_seed(2)
    logits = [torch.randn(5000, 200, device="cuda", generator=gen) for _ in range(6)]
    want = [bl.route_experts(x, 4) for x in logits]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, x in enumerate(logits):
        with torch.cuda.stream(side[i % 2]):
            got.append(bl.route_experts(x, 4))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for name in ("ids", "weights", "offsets", "pairs", "slots"):
            assert torch.equal(getattr(a, name), getattr(b, name))
