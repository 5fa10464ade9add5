"""Sizes out of range of the whole routed layer are named as such (CPU): by the C ABI also
where no workspace could be had for them, and to the binding's caller."""

import pytest
import torch

from tests.test_abi import BL_ERR_SHAPE
from tests.test_layer_refusals import _call, lib  # noqa: F401

U8 = torch.uint8


@pytest.mark.parametrize("kw,name", [
    (dict(t=0), "T=0"), (dict(t=(1 << 24) + 1), "T=16777217"), (dict(e=1025), "E=1025"), (dict(k=9), "k=9"),
    (dict(kk=131088), "K=131088"), (dict(f=0), "F=0"), (dict(f=131088), "F=131088"), (dict(f=24), "F=24"), (dict(n=0), "N=0"),
    (dict(n=(1 << 26) + 1), "N=67108865"), (dict(t=1 << 22, n=1 << 14), "N=16384")])
def test_c_abi_names_the_size(lib, kw, name):  # noqa: F811
    """The query answers 0 bytes, so there is no workspace (of some sizes no other tensor either)."""
    for pointers in (dict(ws=None, wsb=0), dict(ws=None, wsb=0, x=None, logits=None, y=None, gu=None, dn=None)):
        assert _call(lib, **kw, **pointers) == BL_ERR_SHAPE
        assert name in lib.bitlinear_last_error().decode()


@pytest.mark.parametrize("kw,name", [(dict(t=0), "T=0"), (dict(e=1025), "E=1025"), (dict(k=9), "k=9"), (dict(n=0), "N=0"),
                                     (dict(f=0), "F=0"), (dict(kk=24), "K=24")])
def test_binding_names_the_size(built_lib, monkeypatch, kw, name):
    """The binding with the device's part replaced: the library refuses before any HIP call."""
    from bitlinear_w1_a8_amd import _marshal, binding, experts

    def call(dev, fn, *args):
        binding._check(fn(*args, None))
    monkeypatch.setattr(_marshal, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(experts, "device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(experts, "call", call)
    s = dict(dict(t=3, e=8, k=2, f=32, kk=64, n=24), **kw)
    t, e, k, f, kk, n = (s[i] for i in ("t", "e", "k", "f", "kk", "n"))
    one = torch.ones(e)
    with pytest.raises(binding.BitLinearError, match=name):
        experts.experts_ffn(torch.zeros(t, kk), torch.zeros(t, e), k, torch.zeros(e, 2 * f, kk // 4, dtype=U8), one, one,
                            torch.zeros(e, n, f // 4, dtype=U8), one)
