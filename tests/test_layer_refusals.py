"""Refusals of the whole routed layer (CPU): of the C ABI before any HIP call,
of the binding before any memory is allocated."""

import pytest
import torch

from tests.test_abi import (A16, A_ODD, BL_ERR_ALIGN, BL_ERR_ARG, BL_ERR_DTYPE, BL_ERR_NULL,
                            BL_ERR_SHAPE, BL_ERR_WORKSPACE)

BIG = 1 << 62
F32, BF16, I8, U8 = torch.float32, torch.bfloat16, torch.int8, torch.uint8


@pytest.fixture(scope="module")
def lib(built_lib):
    from bitlinear_w1_a8_amd import experts
    return experts._load()


def _call(lib, logits=A16, ld=0, t=4, e=8, k=2, share=0, x=A16, xd=1, absmax=None, gu=A16, gg=A16, ug=A16,
          f=32, kk=64, dn=A16, dg=A16, n=16, y=A16, ws=A16, wsb=BIG):
    return lib.bitlinear_experts_ffn(logits, ld, t, e, k, share, x, xd, absmax, gu, gg, ug, f, kk, dn, dg, n, y,
                                     ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), BL_ERR_NULL), (dict(x=None), BL_ERR_NULL), (dict(gu=None), BL_ERR_NULL),
    (dict(gg=None), BL_ERR_NULL), (dict(ug=None), BL_ERR_NULL), (dict(dn=None), BL_ERR_NULL),
    (dict(dg=None), BL_ERR_NULL), (dict(y=None), BL_ERR_NULL), (dict(ws=None), BL_ERR_NULL),
    (dict(xd=2), BL_ERR_NULL), (dict(xd=1, absmax=A16), BL_ERR_ARG), (dict(xd=3), BL_ERR_DTYPE),
    (dict(ld=2), BL_ERR_DTYPE), (dict(ld=-1), BL_ERR_DTYPE), (dict(share=2), BL_ERR_ARG),
    (dict(t=0), BL_ERR_SHAPE), (dict(t=(1 << 24) + 1), BL_ERR_SHAPE), (dict(e=0), BL_ERR_SHAPE),
    (dict(e=1025), BL_ERR_SHAPE), (dict(k=0), BL_ERR_SHAPE), (dict(k=9), BL_ERR_SHAPE),
    (dict(e=64, k=33), BL_ERR_SHAPE), (dict(kk=40), BL_ERR_SHAPE), (dict(kk=131088), BL_ERR_SHAPE),
    (dict(f=24), BL_ERR_SHAPE), (dict(f=0), BL_ERR_SHAPE), (dict(f=131088), BL_ERR_SHAPE),
    (dict(e=16, f=131072, kk=131072), BL_ERR_SHAPE), (dict(n=0), BL_ERR_SHAPE), (dict(n=(1 << 26) + 1), BL_ERR_SHAPE),
    (dict(n=(1 << 62) + 1), BL_ERR_SHAPE), (dict(n=1 << 26, f=1024), BL_ERR_SHAPE),
    (dict(t=1 << 22, n=1 << 14), BL_ERR_SHAPE), (dict(x=A16 + 8), BL_ERR_ALIGN), (dict(gu=A16 + 8), BL_ERR_ALIGN),
    (dict(dn=A16 + 8), BL_ERR_ALIGN), (dict(ws=A16 + 8), BL_ERR_ALIGN), (dict(logits=A16 + 2), BL_ERR_ALIGN),
    (dict(ld=1, logits=A_ODD), BL_ERR_ALIGN), (dict(xd=2, absmax=A16 + 2), BL_ERR_ALIGN),
    (dict(gg=A_ODD), BL_ERR_ALIGN), (dict(ug=A16 + 2), BL_ERR_ALIGN), (dict(dg=A16 + 2), BL_ERR_ALIGN),
    (dict(y=A16 + 2), BL_ERR_ALIGN), (dict(wsb=0), BL_ERR_WORKSPACE)])
def test_refusals(lib, kw, code):
    assert _call(lib, **kw) == code
    assert lib.bitlinear_last_error()


def test_workspace(lib):
    f = lib.bitlinear_experts_ffn_workspace_bytes
    need = f(4, 8, 2, 32, 64, 16)
    assert need >= 8 * (4 + 4 + 2 * 32 + 4 * 16) and need % 16 == 0
    assert _call(lib, wsb=need - 1) == BL_ERR_WORKSPACE
    for bad in ((0, 8, 2, 32, 64, 16), (4, 0, 2, 32, 64, 16), (4, 8, 33, 32, 64, 16), (4, 8, 2, 0, 64, 16),
                (4, 8, 2, 32, 0, 16), (4, 8, 2, 32, 64, 0), (1 << 24, 64, 32, 131072, 64, 16)):
        assert f(*bad) == 0


@pytest.fixture
def experts(built_lib, monkeypatch):
    from bitlinear_w1_a8_amd import _marshal, experts as mod

    def stop(*args, **kw):
        raise AssertionError("reached")

    def need_cuda(t, name, dtype=None):
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must have dtype {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    monkeypatch.setattr(_marshal, "_need_cuda", need_cuda)
    monkeypatch.setattr(mod, "device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(mod, "call", stop)
    monkeypatch.setattr(mod.torch, "empty", stop)
    return mod


def _good(x=None):
    e, f, k, n = 8, 32, 64, 24
    return dict(x=torch.zeros(3, k) if x is None else x, logits=torch.zeros(3, e), k=2,
                packed_gu=torch.zeros(e, 2 * f, k // 4, dtype=U8), gamma_gate=torch.ones(e), gamma_up=torch.ones(e),
                packed_down=torch.zeros(e, n, f // 4, dtype=U8), gamma_down=torch.ones(e))


@pytest.mark.parametrize("bad,error", [
    (dict(x=torch.zeros(3, 64).half()), TypeError), (dict(x=torch.zeros(64)), ValueError),
    (dict(x=torch.zeros(3, 64, dtype=I8)), ValueError), (dict(absmax=torch.ones(3)), ValueError),
    (dict(x=torch.zeros(3, 64, dtype=I8), absmax=torch.ones(4)), ValueError),
    (dict(x=torch.zeros(3, 64, dtype=I8), absmax=torch.ones(3).bfloat16()), TypeError),
    (dict(x=torch.zeros(4, 64)), ValueError), (dict(x=torch.zeros(3, 128)), ValueError),
    (dict(x=torch.zeros(64, 3).t()), ValueError), (dict(logits=torch.zeros(3, 8).half()), TypeError),
    (dict(logits=torch.zeros(3, 7)), ValueError), (dict(logits=torch.zeros(24)), ValueError),
    (dict(k=0), ValueError), (dict(k=33), ValueError), (dict(k=2.0), TypeError), (dict(share="some"), ValueError),
    (dict(packed_gu=torch.zeros(8, 64, 15, dtype=U8)), ValueError), (dict(packed_gu=torch.zeros(8, 64, 16)), TypeError),
    (dict(packed_gu=torch.zeros(8, 65, 16, dtype=U8)), ValueError), (dict(packed_gu=torch.zeros(64, 16, dtype=U8)), ValueError),
    (dict(packed_down=torch.zeros(8, 24, 9, dtype=U8)), ValueError), (dict(packed_down=torch.zeros(7, 24, 8, dtype=U8)), ValueError),
    (dict(gamma_gate=torch.ones(7)), ValueError), (dict(gamma_up=torch.ones(8).double()), TypeError),
    (dict(gamma_down=torch.ones(8, 1)), ValueError), (dict(out=torch.zeros(3, 25)), ValueError),
    (dict(out=torch.zeros(3, 24).bfloat16()), TypeError)])
def test_binding(experts, bad, error):
    with pytest.raises(error):
        experts.experts_ffn(**{**_good(), **bad})


def test_binding_lets_good_ones_pass(experts):
    with pytest.raises(AssertionError, match="reached"):
        experts.experts_ffn(**_good())
