"""The C ABI of the routed-expert and 4-bit operators without a GPU: exported
symbols, binding signatures, and every refusal, made on the host before any
HIP call.  Every call below fails at least one check; none reaches a launch."""

import os
import re

import pytest

from tests.conftest import ROOT
from tests.test_abi import (A16, A_ODD, BL_ERR_ALIGN, BL_ERR_ARG, BL_ERR_DTYPE, BL_ERR_NULL,
                            BL_ERR_SHAPE, BL_ERR_WORKSPACE)

BIG = 1 << 62


def functions(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bitlinear_\w+)\s*\(", text)))


@pytest.fixture(scope="module")
def lib(built_lib):
    from bitlinear_w1_a8_amd import experts, w4
    experts._load()
    return w4._load()


def test_headers_bound_and_exported(lib):
    from bitlinear_w1_a8_amd import experts, w4
    assert functions("bitlinear_experts.h") == sorted(experts.SIGNATURES)
    assert functions("bitlinear_w4.h") == sorted(w4.SIGNATURES)
    for name in functions("bitlinear_experts.h") + functions("bitlinear_w4.h"):
        assert hasattr(lib, name), name


def test_package_names():
    import bitlinear_w1_a8_amd as bl
    for name in ("Routing", "route_experts", "gated_relu2_experts", "linear_experts",
                 "pack_weights_w4", "unpack_weights_w4", "forward_w4"):
        assert callable(getattr(bl, name))
    with pytest.raises(AttributeError):
        bl.no_such_name


def test_sizes(lib):
    assert lib.bitlinear_route_workspace_bytes(64, 128) == 0
    assert lib.bitlinear_route_workspace_bytes(65, 128) > 0
    assert lib.bitlinear_route_workspace_bytes(0, 128) == 0
    assert lib.bitlinear_experts_workspace_bytes(3, 2, 5) >= 3 * 2 * 5 * 4
    assert lib.bitlinear_w4_row_bytes(128) == 64
    assert lib.bitlinear_w4_row_bytes(160) == 128
    assert lib.bitlinear_w4_row_bytes(0) == 0


def _route(lib, logits=A16, dtype=0, t=4, e=8, k=2, share=0, ids=A16, weights=A16, offsets=A16,
           pairs=A16, slots=A16, ws=A16, wsb=BIG):
    return lib.bitlinear_route_experts(logits, dtype, t, e, k, share, ids, weights, offsets, pairs,
                                       slots, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), BL_ERR_NULL), (dict(ids=None), BL_ERR_NULL), (dict(weights=None), BL_ERR_NULL),
    (dict(offsets=None), BL_ERR_NULL), (dict(pairs=None), BL_ERR_NULL), (dict(slots=None), BL_ERR_NULL),
    (dict(t=65, ws=None), BL_ERR_NULL), (dict(dtype=2), BL_ERR_DTYPE), (dict(dtype=-1), BL_ERR_DTYPE),
    (dict(t=0), BL_ERR_SHAPE), (dict(t=(1 << 24) + 1), BL_ERR_SHAPE), (dict(e=0), BL_ERR_SHAPE),
    (dict(e=1025), BL_ERR_SHAPE), (dict(k=0), BL_ERR_SHAPE), (dict(k=9), BL_ERR_SHAPE),
    (dict(e=64, k=33), BL_ERR_SHAPE), (dict(t=1 << 24, e=64, k=32, k_=0), BL_ERR_ALIGN),
    (dict(share=2), BL_ERR_ARG), (dict(logits=A16 + 2), BL_ERR_ALIGN), (dict(ids=A_ODD), BL_ERR_ALIGN),
    (dict(slots=A16 + 2), BL_ERR_ALIGN), (dict(dtype=1, logits=A_ODD), BL_ERR_ALIGN),
    (dict(t=65, ws=A16 + 2), BL_ERR_ALIGN), (dict(t=65, wsb=7), BL_ERR_WORKSPACE)])
def test_route_refusals(lib, kw, code):
    kw = dict(kw)
    if kw.pop("k_", None) is not None:      # the largest T * k passes the size check
        kw.update(ids=A_ODD)
    assert _route(lib, **kw) == code
    assert lib.bitlinear_last_error()


def _desc(t=4, k=2, e=8, offsets=A16, pairs=A16, slots=A16, weights=A16):
    from bitlinear_w1_a8_amd.experts import _ROUTING
    return _ROUTING.pack(t, k, e, offsets or 0, pairs or 0, slots or 0, weights or 0)


def _gated(lib, desc=None, x=A16, dt=1, packed=A16, g=A16, u=A16, n=16, k=64, h=A16, xq=A16,
           absmax=A16, acc=None):
    d = desc or _desc()
    return lib.bitlinear_gated_relu2_experts(d, x, dt, packed, g, u, n, k, h, xq,
                                             absmax, acc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BL_ERR_NULL), (dict(packed=None), BL_ERR_NULL), (dict(g=None), BL_ERR_NULL),
    (dict(u=None), BL_ERR_NULL), (dict(h=None), BL_ERR_NULL), (dict(xq=None), BL_ERR_NULL),
    (dict(absmax=None), BL_ERR_NULL), (dict(dt=2), BL_ERR_DTYPE), (dict(k=40), BL_ERR_SHAPE),
    (dict(k=0), BL_ERR_SHAPE), (dict(n=0), BL_ERR_SHAPE), (dict(n=(1 << 25) + 1), BL_ERR_SHAPE),
    (dict(n=1 << 25, k=131072), BL_ERR_SHAPE), (dict(n=(1 << 62) + 1), BL_ERR_SHAPE),
    (dict(x=A16 + 8), BL_ERR_ALIGN),
    (dict(packed=A16 + 8), BL_ERR_ALIGN), (dict(xq=A16 + 4), BL_ERR_ALIGN), (dict(h=A_ODD), BL_ERR_ALIGN),
    (dict(acc=A16 + 2), BL_ERR_ALIGN), (dict(absmax=A16 + 1), BL_ERR_ALIGN)])
def test_gated_refusals(lib, kw, code):
    assert _gated(lib, **kw) == code


def test_routing_refusals(lib):
    assert lib.bitlinear_gated_relu2_experts(None, A16, 1, A16, A16, A16, 16, 64, A16, A16, A16, None,
                                             None) == BL_ERR_NULL
    assert _gated(lib, _desc(offsets=None)) == BL_ERR_NULL
    assert _gated(lib, _desc(pairs=None)) == BL_ERR_NULL
    for kw in (dict(t=0), dict(t=(1 << 24) + 1), dict(k=0), dict(k=9), dict(e=0), dict(e=1025)):
        assert _gated(lib, _desc(**kw)) == BL_ERR_SHAPE
    assert _gated(lib, _desc(t=1 << 24, k=32, e=64), n=1 << 12) == BL_ERR_SHAPE   # T k 2N above 2^36
    assert _gated(lib, _desc(offsets=A16 + 2)) == BL_ERR_ALIGN
    assert _linear(lib, _desc(slots=None)) == BL_ERR_NULL
    assert _linear(lib, _desc(weights=None)) == BL_ERR_NULL
    assert _linear(lib, _desc(slots=A_ODD)) == BL_ERR_ALIGN


def _linear(lib, desc=None, x=A16, dt=1, xr=1, packed=A16, g=A16, n=16, k=64, y=A16, yr=0, xq=A16,
            absmax=A16, acc=None, ws=A16, wsb=BIG):
    d = desc or _desc()
    return lib.bitlinear_linear_experts(d, x, dt, xr, packed, g, n, k, y, yr, xq, absmax,
                                        acc, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BL_ERR_NULL), (dict(packed=None), BL_ERR_NULL), (dict(g=None), BL_ERR_NULL),
    (dict(y=None), BL_ERR_NULL), (dict(xq=None), BL_ERR_NULL), (dict(absmax=None), BL_ERR_NULL),
    (dict(ws=None), BL_ERR_NULL), (dict(dt=3), BL_ERR_DTYPE), (dict(xr=2), BL_ERR_ARG),
    (dict(yr=-1), BL_ERR_ARG), (dict(acc=A16), BL_ERR_ARG), (dict(k=17), BL_ERR_SHAPE),
    (dict(n=0), BL_ERR_SHAPE), (dict(n=(1 << 26) + 1), BL_ERR_SHAPE),
    (dict(n=1 << 26, k=131072), BL_ERR_SHAPE), (dict(x=A16 + 2), BL_ERR_ALIGN),
    (dict(packed=A16 + 4), BL_ERR_ALIGN), (dict(y=A16 + 2), BL_ERR_ALIGN), (dict(ws=A16 + 8), BL_ERR_ALIGN),
    (dict(yr=1, acc=A16 + 2), BL_ERR_ALIGN), (dict(wsb=4 * 2 * 16 * 4 - 1), BL_ERR_WORKSPACE)])
def test_linear_refusals(lib, kw, code):
    assert _linear(lib, **kw) == code


def _w4(lib, packed=A16, s=A16, z=None, xq=A16, a=A16, t=2, n=16, k=128, g=64, y=A16):
    return lib.bitlinear_forward_w4(packed, s, z, xq, a, t, n, k, g, y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(packed=None), BL_ERR_NULL), (dict(s=None), BL_ERR_NULL), (dict(xq=None), BL_ERR_NULL),
    (dict(a=None), BL_ERR_NULL), (dict(y=None), BL_ERR_NULL), (dict(g=16), BL_ERR_ARG),
    (dict(g=0), BL_ERR_ARG), (dict(g=256, k=256), BL_ERR_ARG), (dict(k=96), BL_ERR_SHAPE),
    (dict(k=0), BL_ERR_SHAPE), (dict(k=131072 + 64), BL_ERR_SHAPE), (dict(n=0), BL_ERR_SHAPE),
    (dict(n=(1 << 26) + 1), BL_ERR_SHAPE), (dict(n=1 << 26, k=8192), BL_ERR_SHAPE),
    (dict(t=0), BL_ERR_SHAPE), (dict(t=(1 << 24) + 1), BL_ERR_SHAPE),
    (dict(t=1 << 24, n=1 << 13), BL_ERR_SHAPE), (dict(packed=A16 + 8), BL_ERR_ALIGN),
    (dict(xq=A16 + 8), BL_ERR_ALIGN), (dict(s=A_ODD), BL_ERR_ALIGN), (dict(y=A16 + 2), BL_ERR_ALIGN)])
def test_w4_refusals(lib, kw, code):
    assert _w4(lib, **kw) == code


def test_w4_pack_refusals(lib):
    for f in (lambda w=A16, n=16, k=128, g=64, p=A16, s=A16: lib.bitlinear_pack_weights_w4(
                  w, n, k, g, p, s, None, None),
              lambda w=A16, n=16, k=128, g=64, p=A16, s=A16: lib.bitlinear_unpack_weights_w4(
                  p, s, None, n, k, g, w, None)):
        assert f(w=None) == BL_ERR_NULL
        assert f(p=None) == BL_ERR_NULL
        assert f(s=None) == BL_ERR_NULL
        assert f(g=48) == BL_ERR_ARG
        assert f(k=96) == BL_ERR_SHAPE
        assert f(n=0) == BL_ERR_SHAPE
        assert f(n=1 << 26, k=8192) == BL_ERR_SHAPE
        assert f(w=A16 + 4) == BL_ERR_ALIGN
        assert f(p=A16 + 4) == BL_ERR_ALIGN
        assert f(s=A_ODD) == BL_ERR_ALIGN


def test_cpu_tensors_refused(built_lib):
    import torch
    import bitlinear_w1_a8_amd as bl
    with pytest.raises(TypeError):
        bl.route_experts(torch.zeros(3, 4), 2)
    with pytest.raises(TypeError):
        bl.pack_weights_w4(torch.zeros(3, 128))
