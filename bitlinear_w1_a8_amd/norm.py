"""The step between two layers (include/bitlinear_norm.h), same names: the
residual's addition, the sub-layer norm and 8-bit codes of its output.
Argument marshalling only, as ``binding``."""

import ctypes

import torch

from . import binding
from ._marshal import call, device_of, need
from .binding import BL_BF16, BL_F32, _c_i64, _c_int, _c_vp

_NORM = [_c_vp, _c_int, _c_vp, _c_int, _c_vp, ctypes.c_float, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]

# name -> (restype, argtypes), as declared in include/bitlinear_norm.h
SIGNATURES = {
    "bitlinear_add_subln_quant_act": (_c_int, [*_NORM, _c_vp, _c_vp]),
    "bitlinear_add_subln_quant_act_f8": (_c_int, [*_NORM, _c_vp]),
}

_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}

_lib = None


def _load():
    global _lib
    if _lib is None:
        _lib = binding.declare(SIGNATURES)
    return _lib


def _inputs(x, residual, gain, out):
    """Checked; returns (device, shape, x's dtype, the residual's, total)."""
    dev = device_of(x, "x")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    shape = x.shape
    need(dev, x, "x", x.dtype, shape)
    need(dev, gain, "gain", torch.float32, shape[1:])
    if residual is None:
        if out is not None:
            raise ValueError("out is the sum's place: there is none without a residual")
        return dev, shape, dt, BL_F32, None
    device_of(residual, "residual")
    rt = _DTYPES.get(residual.dtype)
    if rt is None:
        raise TypeError(f"residual must be float32 or bfloat16, got {residual.dtype}")
    need(dev, residual, "residual", residual.dtype, shape)
    if out is None:
        out = torch.empty_like(residual)
    else:
        need(dev, out, "out", residual.dtype, shape)
    return dev, shape, dt, rt, out


def add_subln_quant_act(x, residual, gain, eps_n=1e-5, with_rowsum=True, out=None):
    """total = x + residual, its sub-layer norm and step A1's codes, in one
    launch: x [T, K] and residual [T, K] (float32 or bfloat16 each; residual
    None: the norm of x alone), gain float32 [K] -> (xq int8 [T, K], scale
    float32 [T], rowsum int32 [T] or None, total of the residual's dtype or
    None).  ``out`` takes the sum; it may be the residual itself, or x where
    their dtypes are the same."""
    lib = _load()
    dev, shape, dt, rt, total = _inputs(x, residual, gain, out)
    t, k = shape
    on = x.device
    xq = torch.empty_like(x, dtype=torch.int8)          # half the time of torch.empty(shape)
    scale = torch.empty(t, dtype=torch.float32, device=on)
    rowsum = torch.empty(t, dtype=torch.int32, device=on) if with_rowsum else None
    call(dev, lib.bitlinear_add_subln_quant_act, x.data_ptr(), dt,
         None if residual is None else residual.data_ptr(), rt, gain.data_ptr(), float(eps_n), t, k,
         None if total is None else total.data_ptr(), xq.data_ptr(), scale.data_ptr(),
         rowsum.data_ptr() if with_rowsum else None)
    return xq, scale, rowsum, total


def add_subln_quant_act_f8(x, residual, gain, eps_n=1e-5, out=None):
    """As add_subln_quant_act, with e4m3 codes and one scale per 128 features:
    -> (xq float8_e4m3fn [T, K], scales float32 [ceil(K / 128), T], total or
    None), what forward_f8 takes."""
    lib = _load()
    dev, shape, dt, rt, total = _inputs(x, residual, gain, out)
    t, k = shape
    xq = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    scales = torch.empty(((k + 127) // 128, t), dtype=torch.float32, device=x.device)
    call(dev, lib.bitlinear_add_subln_quant_act_f8, x.data_ptr(), dt,
         None if residual is None else residual.data_ptr(), rt, gain.data_ptr(), float(eps_n), t, k,
         None if total is None else total.data_ptr(), xq.data_ptr(), scales.data_ptr())
    return xq, scales, total
