"""Linear layers with 4-bit weights and group scales
(include/bitlinear_w4.h), same names: packing, unpacking, the product with
step A1's int8 tokens.  Argument marshalling only, as ``binding``."""

import operator

import torch

from . import binding
from ._marshal import call, device_of, need
from .binding import _c_i64, _c_int, _c_vp

# name -> (restype, argtypes), as declared in include/bitlinear_w4.h
SIGNATURES = {
    "bitlinear_w4_row_bytes": (_c_i64, [_c_i64]),
    "bitlinear_pack_weights_w4": (_c_int, [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp]),
    "bitlinear_unpack_weights_w4": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp,
                                             _c_vp]),
    "bitlinear_forward_w4": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64,
                                      _c_i64, _c_vp, _c_vp]),
}

_lib = None


def _load():
    global _lib
    if _lib is None:
        _lib = binding.declare(SIGNATURES)
    return _lib


def _matrix(dev, packed, scales, zeros, k):
    """Checks a packed matrix of rows of k weights; returns (rows, group)."""
    if packed.dim() != 2 or scales.dim() != 2:
        raise ValueError("packed must be [N, row bytes] and scales [N, K/G]")
    n, groups = shape = scales.shape
    if groups < 1 or k % groups:
        raise ValueError(f"scales of {groups} groups do not cut rows of {k} weights evenly")
    need(dev, scales, "scales", torch.bfloat16, shape)
    need(dev, packed, "packed", torch.uint8, (n, (k + 127) // 128 * 64))
    if zeros is not None:
        need(dev, zeros, "zeros", torch.int8, shape)
    return n, k // groups


def pack_weights_w4(w, group=128, with_zeros=False):
    """float32 w [N, K] -> (packed uint8 [N, 64 * ceil(K / 128)], scales
    bfloat16 [N, K / group], zeros int8 [N, K / group] or None); group 32, 64
    or 128."""
    lib = _load()
    dev = device_of(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    n, k = shape = w.shape
    need(dev, w, "w", torch.float32, shape)
    group, on = operator.index(group), w.device
    if group not in (32, 64, 128) or k % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide K={k}, got {group}")
    packed = torch.empty((n, (k + 127) // 128 * 64), dtype=torch.uint8, device=on)
    scales = torch.empty((n, k // group), dtype=torch.bfloat16, device=on)
    zeros = torch.empty((n, k // group), dtype=torch.int8, device=on) if with_zeros else None
    call(dev, lib.bitlinear_pack_weights_w4, w.data_ptr(), n, k, group, packed.data_ptr(),
         scales.data_ptr(), zeros.data_ptr() if with_zeros else None)
    return packed, scales, zeros


def unpack_weights_w4(packed, scales, zeros, k):
    """The float32 values [N, k] that a packed matrix stands for."""
    lib = _load()
    k, dev = operator.index(k), device_of(packed, "packed")
    n, group = _matrix(dev, packed, scales, zeros, k)
    w = torch.empty((n, k), dtype=torch.float32, device=packed.device)
    call(dev, lib.bitlinear_unpack_weights_w4, packed.data_ptr(), scales.data_ptr(),
         None if zeros is None else zeros.data_ptr(), n, k, group, w.data_ptr())
    return w


def forward_w4(packed, scales, xq, absmax, zeros=None, out=None):
    """y float32 [T, N] = tokens of step A1 (xq int8 [T, K], absmax float32
    [T], from quant_act or subln_quant_act) times a 4-bit matrix."""
    lib = _load()
    dev = device_of(xq, "xq")
    if xq.dim() != 2:
        raise ValueError("xq must be [T, K]")
    t, k = shape = xq.shape
    need(dev, xq, "xq", torch.int8, shape)
    n, group = _matrix(dev, packed, scales, zeros, k)
    need(dev, absmax, "absmax", torch.float32, (t,))
    if out is None:
        out = torch.empty((t, n), dtype=torch.float32, device=xq.device)
    else:
        need(dev, out, "out", torch.float32, (t, n))
    call(dev, lib.bitlinear_forward_w4, packed.data_ptr(), scales.data_ptr(),
         None if zeros is None else zeros.data_ptr(), xq.data_ptr(), absmax.data_ptr(), t, n, k,
         group, out.data_ptr())
    return out
