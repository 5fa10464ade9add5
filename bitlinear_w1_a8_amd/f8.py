"""Linear layers in 8-bit floating point with a scale for each block of 128
(include/bitlinear_f8.h), same names.  Argument marshalling only, as
``binding``."""

import torch

from . import binding
from ._marshal import call, device_of, need
from .binding import BL_BF16, BL_F32, _c_i64, _c_int, _c_vp

# name -> (restype, argtypes), as declared in include/bitlinear_f8.h
SIGNATURES = {
    "bitlinear_quant_act_f8": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "bitlinear_pack_weights_f8": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "bitlinear_unpack_weights_f8": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "bitlinear_forward_f8": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp,
                                      _c_int, _c_vp]),
    "bitlinear_linear_f8": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp,
                                     _c_vp, _c_int, _c_vp]),
}

#: what a product's sums keep: binary32, or (bfloat16 outputs) what e4m3 matrix instructions keep
SUMS = {"full": 0, "cut": 0x100}             # BL_CUT_SUMS
_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}
_F8 = torch.float8_e4m3fn

_lib = None


def _load():
    global _lib
    if _lib is None:
        _lib = binding.declare(SIGNATURES)
    return _lib


def _blocks(n):
    return (n + 127) // 128


def _matrix(dev, w, w_scales):
    """Checks a matrix; returns its shape."""
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    n, k = shape = w.shape
    need(dev, w, "w", _F8, shape)
    need(dev, w_scales, "w_scales", torch.float32, (_blocks(n), _blocks(k)))
    return n, k


def quant_act_f8(x):
    """x [T, K] (float32 or bfloat16) -> (xq float8_e4m3fn [T, K], scales
    float32 [ceil(K / 128), T]), one scale per token and 128 features."""
    lib = _load()
    dev = device_of(x, "x")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    t, k = shape = x.shape
    need(dev, x, "x", x.dtype, shape)
    xq = torch.empty_like(x, dtype=_F8)                 # half the time of torch.empty(shape)
    scales = torch.empty((_blocks(k), t), dtype=torch.float32, device=x.device)
    call(dev, lib.bitlinear_quant_act_f8, x.data_ptr(), dt, t, k, xq.data_ptr(), scales.data_ptr())
    return xq, scales


def pack_weights_f8(w):
    """float32 w [N, K] -> (codes float8_e4m3fn [N, K], scales float32
    [ceil(N / 128), ceil(K / 128)]), one scale per block of 128 x 128."""
    lib = _load()
    dev = device_of(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    n, k = shape = w.shape
    need(dev, w, "w", torch.float32, shape)
    codes = torch.empty_like(w, dtype=_F8)
    scales = torch.empty((_blocks(n), _blocks(k)), dtype=torch.float32, device=w.device)
    call(dev, lib.bitlinear_pack_weights_f8, w.data_ptr(), n, k, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def unpack_weights_f8(w, w_scales):
    """The float32 values [N, K] that a matrix of pack_weights_f8 stands for."""
    lib = _load()
    dev = device_of(w, "w")
    n, k = _matrix(dev, w, w_scales)
    out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    call(dev, lib.bitlinear_unpack_weights_f8, w.data_ptr(), w_scales.data_ptr(), n, k, out.data_ptr())
    return out


def _out(dev, out, shape, dtype, on, sums):
    """The outputs' tensor, and the C ABI's y_dtype."""
    if out is not None:
        device_of(out, "out")
        dtype = out.dtype
    kind = _DTYPES.get(dtype)
    if kind is None:
        raise TypeError(f"{'dtype' if out is None else 'out'} must be float32 or bfloat16, got {dtype}")
    if sums not in SUMS:
        raise ValueError(f"sums must be one of {sorted(SUMS)}, got {sums!r}")
    if sums == "cut" and kind != BL_BF16:
        raise ValueError("cut sums are for bfloat16 outputs")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=on)
    else:
        need(dev, out, "out", dtype, shape)
    return out, kind | SUMS[sums]


def _rows(w, k):
    """Rows of a matrix of k columns."""
    device_of(w, "w")
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError(f"w must be [N, {k}], got {tuple(w.shape)}")
    return w.shape[0]


def forward_f8(w, w_scales, xq, x_scales, dtype=torch.float32, out=None, sums="full"):
    """y [T, N] of ``dtype`` (float32 or bfloat16; ``out`` brings its own) =
    tokens (xq float8_e4m3fn [T, K], x_scales float32 [ceil(K / 128), T], from
    quant_act_f8 or add_subln_quant_act_f8) times a matrix of pack_weights_f8,
    summed in binary32.  ``sums="cut"`` allows bfloat16 outputs to be formed
    faster from sums that lose up to 7 * 2^-13 of their products' magnitudes."""
    lib = _load()
    dev = device_of(xq, "xq")
    if xq.dim() != 2:
        raise ValueError("xq must be [T, K]")
    t, k = shape = xq.shape
    n = _rows(w, k)
    need(dev, xq, "xq", _F8, shape)
    need(dev, w, "w", _F8, (n, k))
    need(dev, w_scales, "w_scales", torch.float32, (_blocks(n), _blocks(k)))
    need(dev, x_scales, "x_scales", torch.float32, (_blocks(k), t))
    out, kind = _out(dev, out, (t, n), dtype, xq.device, sums)
    call(dev, lib.bitlinear_forward_f8, w.data_ptr(), w_scales.data_ptr(), xq.data_ptr(),
         x_scales.data_ptr(), t, n, k, out.data_ptr(), kind)
    return out


def linear_f8(x, w, w_scales, dtype=torch.float32, out=None, sums="full"):
    """quant_act_f8 of x [T, K] (float32 or bfloat16), then forward_f8: y [T, N]."""
    lib = _load()
    dev = device_of(x, "x")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    t, k = shape = x.shape
    n, blocks = _rows(w, k), _blocks(k)
    need(dev, x, "x", x.dtype, shape)
    need(dev, w, "w", _F8, (n, k))
    need(dev, w_scales, "w_scales", torch.float32, (_blocks(n), blocks))
    on = x.device
    out, kind = _out(dev, out, (t, n), dtype, on, sums)
    codes = (t * k + 255) & ~255                # the codes, then their scales, in one piece
    scratch = torch.empty(codes + 4 * blocks * t, dtype=torch.uint8, device=on)
    at = scratch.data_ptr()
    call(dev, lib.bitlinear_linear_f8, x.data_ptr(), dt, w.data_ptr(), w_scales.data_ptr(), t, n, k, at,
         at + codes, out.data_ptr(), kind)
    return out
