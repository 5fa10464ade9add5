"""Refusals of the residual norms and of the 8-bit floating point calls (CPU):
of the C ABI before any HIP call, of the binding before any memory is
allocated.  Every call below fails a check; none reaches a launch."""

import pytest
import torch

from tests.test_abi import (A16, A_ODD, BL_ERR_ALIGN, BL_ERR_ARG, BL_ERR_DTYPE, BL_ERR_NULL,
                            BL_ERR_SHAPE)
from tests.test_experts_abi import functions

F8, F32, BF16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lib(built_lib):
    from bitlinear_w1_a8_amd import f8, norm
    norm._load()
    return f8._load()


def test_headers_bound_and_exported(lib):
    import bitlinear_w1_a8_amd as bl
    from bitlinear_w1_a8_amd import f8, norm
    assert functions("bitlinear_f8.h") == sorted(f8.SIGNATURES)
    assert functions("bitlinear_norm.h") == sorted(norm.SIGNATURES)
    for name in functions("bitlinear_f8.h") + functions("bitlinear_norm.h"):
        assert hasattr(lib, name), name
    for name in ("add_subln_quant_act", "add_subln_quant_act_f8", "quant_act_f8", "pack_weights_f8",
                 "unpack_weights_f8", "forward_f8", "linear_f8"):
        assert callable(getattr(bl, name))


# ------------------------------------------------------------ C ABI

def _norm(lib, x=A16, xd=0, r=A16, rd=1, gain=A16, eps=1e-5, t=4, k=64, total=A16, xq=A16, s=A16, rs=None):
    a = lib.bitlinear_add_subln_quant_act(x, xd, r, rd, gain, eps, t, k, total, xq, s, rs, None)
    if rs is None:
        assert lib.bitlinear_add_subln_quant_act_f8(x, xd, r, rd, gain, eps, t, k, total, xq, s, None) == a
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BL_ERR_NULL), (dict(gain=None), BL_ERR_NULL), (dict(total=None), BL_ERR_NULL),
    (dict(xq=None), BL_ERR_NULL), (dict(s=None), BL_ERR_NULL), (dict(r=None), BL_ERR_ARG),
    (dict(xd=2), BL_ERR_DTYPE), (dict(rd=-1), BL_ERR_DTYPE), (dict(eps=0.0), BL_ERR_ARG),
    (dict(eps=-1.0), BL_ERR_ARG), (dict(eps=float("nan")), BL_ERR_ARG), (dict(eps=float("inf")), BL_ERR_ARG),
    (dict(eps=1e-50), BL_ERR_ARG), (dict(t=0), BL_ERR_SHAPE), (dict(t=(1 << 24) + 1), BL_ERR_SHAPE),
    (dict(k=0), BL_ERR_SHAPE), (dict(k=24), BL_ERR_SHAPE), (dict(k=131088), BL_ERR_SHAPE),
    (dict(x=A16 + 8), BL_ERR_ALIGN), (dict(r=A16 + 8), BL_ERR_ALIGN), (dict(gain=A16 + 4), BL_ERR_ALIGN),
    (dict(total=A16 + 8), BL_ERR_ALIGN), (dict(xq=A16 + 8), BL_ERR_ALIGN), (dict(s=A16 + 2), BL_ERR_ALIGN),
    (dict(rs=A_ODD), BL_ERR_ALIGN)])
def test_norm_refusals(lib, kw, code):
    assert _norm(lib, **kw) == code
    assert lib.bitlinear_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BL_ERR_NULL), (dict(q=None), BL_ERR_NULL), (dict(s=None), BL_ERR_NULL),
    (dict(d=3), BL_ERR_DTYPE), (dict(t=0), BL_ERR_SHAPE), (dict(t=(1 << 24) + 1), BL_ERR_SHAPE),
    (dict(k=8), BL_ERR_SHAPE), (dict(k=131088), BL_ERR_SHAPE), (dict(x=A16 + 4), BL_ERR_ALIGN),
    (dict(q=A16 + 8), BL_ERR_ALIGN), (dict(s=A_ODD), BL_ERR_ALIGN)])
def test_quant_refusals(lib, kw, code):
    def call(x=A16, d=1, t=3, k=48, q=A16, s=A16):
        return lib.bitlinear_quant_act_f8(x, d, t, k, q, s, None)
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), BL_ERR_NULL), (dict(q=None), BL_ERR_NULL), (dict(s=None), BL_ERR_NULL),
    (dict(n=0), BL_ERR_SHAPE), (dict(n=(1 << 26) + 1), BL_ERR_SHAPE), (dict(n=1 << 26, k=8192), BL_ERR_SHAPE),
    (dict(k=0), BL_ERR_SHAPE), (dict(k=40), BL_ERR_SHAPE), (dict(k=131088), BL_ERR_SHAPE),
    (dict(w=A16 + 4), BL_ERR_ALIGN), (dict(q=A16 + 4), BL_ERR_ALIGN), (dict(s=A16 + 1), BL_ERR_ALIGN)])
def test_pack_refusals(lib, kw, code):
    def pack(w=A16, n=16, k=128, q=A16, s=A16):
        return lib.bitlinear_pack_weights_f8(w, n, k, q, s, None)

    def unpack(w=A16, n=16, k=128, q=A16, s=A16):
        return lib.bitlinear_unpack_weights_f8(q, s, n, k, w, None)
    assert pack(**kw) == code and unpack(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), BL_ERR_NULL), (dict(ws=None), BL_ERR_NULL), (dict(x=None), BL_ERR_NULL),
    (dict(xs=None), BL_ERR_NULL), (dict(y=None), BL_ERR_NULL), (dict(yd=2), BL_ERR_DTYPE),
    (dict(t=0), BL_ERR_SHAPE), (dict(t=(1 << 24) + 1), BL_ERR_SHAPE), (dict(t=1 << 24, n=1 << 13), BL_ERR_SHAPE),
    (dict(n=0), BL_ERR_SHAPE), (dict(n=(1 << 62) + 1), BL_ERR_SHAPE), (dict(n=1 << 26, k=8192), BL_ERR_SHAPE),
    (dict(k=100), BL_ERR_SHAPE), (dict(w=A16 + 8), BL_ERR_ALIGN), (dict(x=A16 + 1), BL_ERR_ALIGN),
    (dict(ws=A16 + 2), BL_ERR_ALIGN), (dict(xs=A16 + 2), BL_ERR_ALIGN), (dict(y=A16 + 2), BL_ERR_ALIGN),
    (dict(yd=1, y=A_ODD), BL_ERR_ALIGN)])
def test_forward_refusals(lib, kw, code):
    def call(w=A16, ws=A16, x=A16, xs=A16, t=2, n=16, k=128, y=A16, yd=0):
        return lib.bitlinear_forward_f8(w, ws, x, xs, t, n, k, y, yd, None)
    assert call(**kw) == code

    def linear(w=A16, ws=A16, x=A16, xs=A16, t=2, n=16, k=128, y=A16, yd=0, raw=A16, rd=1):
        return lib.bitlinear_linear_f8(raw, rd, w, ws, t, n, k, x, xs, y, yd, None)
    assert linear(**kw) == code
    assert linear(raw=None) == BL_ERR_NULL and linear(rd=2) == BL_ERR_DTYPE and linear(raw=A16 + 8) == BL_ERR_ALIGN


# ------------------------------------------------------------ binding

def test_cpu_tensors_refused(built_lib):
    import bitlinear_w1_a8_amd as bl
    x = torch.zeros(2, 32)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        bl.add_subln_quant_act(x, x, torch.ones(32))
    with pytest.raises(TypeError, match="x must be a CUDA"):
        bl.quant_act_f8(x)
    with pytest.raises(TypeError, match="w must be a CUDA"):
        bl.pack_weights_f8(x)
    with pytest.raises(TypeError, match="xq must be a CUDA"):
        bl.forward_f8(x.to(F8), torch.ones(1, 1), x.to(F8), torch.ones(1, 2))


@pytest.fixture
def mods(built_lib, monkeypatch):
    """norm and f8 with the device check replaced; allocating or calling fails the test."""
    from bitlinear_w1_a8_amd import _marshal, f8, norm

    def stop(*args, **kw):
        raise AssertionError("reached")
    monkeypatch.setattr(_marshal, "_need_cuda", lambda t, name, dtype=None: (_ for _ in ()).throw(
        TypeError(f"{name} dtype") if dtype is not None and t.dtype != dtype else
        ValueError(f"{name} must be contiguous")) if (dtype is not None and t.dtype != dtype) or
        not t.is_contiguous() else None)
    for m in (f8, norm):
        monkeypatch.setattr(m, "device_of", lambda t, name: t.get_device())
        monkeypatch.setattr(m, "call", stop)
    return norm, f8


def test_norm_binding(mods):
    norm, _ = mods
    x, r, g = torch.zeros(3, 64), torch.zeros(3, 64, dtype=BF16), torch.ones(64)
    for f in (norm.add_subln_quant_act, norm.add_subln_quant_act_f8):
        for bad in ((x.half(), r, g), (x, r.half(), g), (x, r, g.bfloat16()), (x, x.int(), g)):
            with pytest.raises(TypeError):
                f(*bad)
        for bad in ((x[0], r, g), (x, r[:2], g), (x, r, g[:32]), (x, r[:, :32], g), (x, r, torch.ones(1, 64)),
                    (torch.zeros(3, 128)[:, ::2], r, g), (x, torch.zeros(64, 3, dtype=BF16).t(), g)):
            with pytest.raises(ValueError):
                f(*bad)
        with pytest.raises(ValueError, match="out is the sum's place"):
            f(x, None, g, out=x)
        with pytest.raises(TypeError):
            f(x, r, g, out=torch.zeros(3, 64))       # the sum has the residual's type
        with pytest.raises(ValueError):
            f(x, r, g, out=torch.zeros(4, 64, dtype=BF16))


def test_f8_binding(mods):
    _, f8 = mods
    w, ws = torch.zeros(130, 144).to(F8), torch.ones(2, 2)
    x, xs = torch.zeros(5, 144).to(F8), torch.ones(2, 5)
    for bad in ((w.float(), ws, x, xs), (w, ws, x.float(), xs), (w, ws.bfloat16(), x, xs), (w, ws, x, xs.double())):
        with pytest.raises(TypeError):
            f8.forward_f8(*bad)
    for bad in ((w[0], ws, x, xs), (w, ws[:1], x, xs), (w, ws, x[0], xs), (w, ws, x, xs.t().contiguous()),
                (w[:, :128].contiguous(), ws, x, xs), (w, ws, x, xs[:, :4].contiguous()), (w, ws[:, :1], x, xs)):
        with pytest.raises(ValueError):
            f8.forward_f8(*bad)
    with pytest.raises(TypeError):
        f8.forward_f8(w, ws, x, xs, dtype=torch.float16)
    with pytest.raises(TypeError):
        f8.forward_f8(w, ws, x, xs, out=torch.zeros(5, 130, dtype=torch.float16))
    with pytest.raises(ValueError):
        f8.forward_f8(w, ws, x, xs, out=torch.zeros(5, 131))
    raw = torch.zeros(5, 144)
    for bad in ((raw.half(), w, ws), (raw, w.float(), ws), (raw, w, ws.bfloat16())):
        with pytest.raises(TypeError):
            f8.linear_f8(*bad)
    for bad in ((raw[0], w, ws), (raw[:, :128].contiguous(), w, ws), (raw, w, ws[:1]), (raw, w[0], ws),
                (torch.zeros(144, 5).t(), w, ws)):
        with pytest.raises(ValueError):
            f8.linear_f8(*bad)
    with pytest.raises(TypeError):
        f8.linear_f8(raw, w, ws, dtype=torch.float16)
    with pytest.raises(ValueError):
        f8.linear_f8(raw, w, ws, out=torch.zeros(4, 130))
    with pytest.raises(TypeError):
        f8.quant_act_f8(torch.zeros(3, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        f8.quant_act_f8(torch.zeros(64))
    with pytest.raises(TypeError):
        f8.pack_weights_f8(torch.zeros(3, 64, dtype=BF16))
    with pytest.raises(ValueError):
        f8.pack_weights_f8(torch.zeros(64))
    with pytest.raises(ValueError):
        f8.unpack_weights_f8(w, ws[:1])
    with pytest.raises(TypeError):
        f8.unpack_weights_f8(w.float(), ws)
