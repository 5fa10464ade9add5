"""Sizes of the 4-bit binding that are not whole numbers are refused, on the
CPU: the device check is replaced, nothing is launched."""

import pytest
import torch


@pytest.fixture
def w4(built_lib, monkeypatch):
    from bitlinear_w1_a8_amd import w4 as mod

    def stop(*args, **kw):
        raise AssertionError("allocated")
    monkeypatch.setattr(mod, "device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(mod.torch, "empty", stop)
    return mod


@pytest.mark.parametrize("group", [32.5, "64", None])
def test_group_not_whole(w4, group):
    with pytest.raises(TypeError, match="integer"):
        w4.pack_weights_w4(torch.zeros(2, 128), group)


@pytest.mark.parametrize("k", [128.9, "128"])
def test_row_length_not_whole(w4, k):
    with pytest.raises(TypeError, match="integer"):
        w4.unpack_weights_w4(torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.bfloat16), None, k)
