"""Refusals of the routed-expert binding that are made before any memory is
allocated, on the CPU: the device check is replaced, nothing is launched."""

import pytest
import torch


@pytest.fixture
def experts(built_lib, monkeypatch):
    from bitlinear_w1_a8_amd import experts as mod

    def stop(*args, **kw):
        raise AssertionError("allocated")
    monkeypatch.setattr(mod, "device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(mod.torch, "empty", stop)
    return mod


@pytest.mark.parametrize("k", [0, -1, 33, 1 << 40, 1 << 70])
def test_ranks_out_of_range(experts, k):
    with pytest.raises(ValueError, match="k must be in"):
        experts.route_experts(torch.zeros(3, 64), k)


@pytest.mark.parametrize("k", [2.5, "2", None])
def test_ranks_not_whole(experts, k):
    with pytest.raises(TypeError):
        experts.route_experts(torch.zeros(3, 64), k)
