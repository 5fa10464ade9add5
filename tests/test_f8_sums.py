"""The choice between full and cut sums of e4m3 products: what is refused (CPU),
by the C ABI before any HIP call and by the binding before memory is allocated."""

import re

import pytest
import torch

from tests.test_abi import A16, A_ODD, BL_ERR_ALIGN, BL_ERR_DTYPE
from tests.test_f8_refusals import lib, mods  # noqa: F401

F8, BF16 = torch.float8_e4m3fn, torch.bfloat16
CUT = 0x100


def test_header_and_binding_agree(built_lib):
    import os

    from bitlinear_w1_a8_amd import f8
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "bitlinear_f8.h")) as h:
        assert int(re.search(r"#define BL_CUT_SUMS (\w+)", h.read()).group(1), 16) == CUT
    assert f8.SUMS == {"full": 0, "cut": CUT}


@pytest.mark.parametrize("kind,code", [(CUT, BL_ERR_DTYPE), (CUT | 2, BL_ERR_DTYPE), (2 * CUT | 1, BL_ERR_DTYPE),
                                       (CUT | 1, BL_ERR_ALIGN)])
def test_c_abi(lib, kind, code):  # noqa: F811
    """Cut sums belong to bfloat16 outputs (whose bad address is the next thing found)."""
    assert lib.bitlinear_forward_f8(A16, A16, A16, A16, 40, 16, 128, A_ODD, kind, None) == code
    assert lib.bitlinear_linear_f8(A16, 0, A16, A16, 40, 16, 128, A16, A16, A_ODD, kind, None) == code


def test_binding(mods, monkeypatch):  # noqa: F811
    _, f8 = mods

    def stop(*args, **kw):
        raise AssertionError("reached")
    w, ws, xs = torch.zeros(130, 144).to(F8), torch.ones(2, 2), torch.ones(2, 5)
    x, raw = torch.zeros(5, 144).to(F8), torch.zeros(5, 144)
    y, b = torch.zeros(5, 130), torch.zeros(5, 130, dtype=BF16)
    monkeypatch.setattr(f8.torch, "empty", stop)
    for call, args in ((f8.forward_f8, (w, ws, x, xs)), (f8.linear_f8, (raw, w, ws))):
        for kw in (dict(sums="cut"), dict(sums="cut", out=y), dict(sums="some"), dict(sums=None, dtype=BF16),
                   dict(sums="f32", out=b)):
            with pytest.raises(ValueError, match="sums"):
                call(*args, **kw)
        for kw in (dict(sums="cut", out=b), dict(sums="cut", dtype=BF16), dict(sums="full", out=y)):
            with pytest.raises(AssertionError, match="reached"):
                call(*args, **kw)
