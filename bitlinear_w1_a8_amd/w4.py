"""Linear layers with 4-bit weights and group scales
(include/bitlinear_w4.h), same names: packing, unpacking, the product with
step A1's int8 tokens.  Argument marshalling only, as ``binding``."""

import torch

from . import binding
from .binding import (_c_i64, _c_int, _c_vp, _check, _need_cuda, _need_shape, _ptr, _same_device,
                      _stream)

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


def _matrix(packed, scales, zeros, k):
    """Checks a packed matrix of rows of k weights; returns (rows, group)."""
    _need_cuda(packed, "packed", torch.uint8)
    _need_cuda(scales, "scales", torch.bfloat16)
    if packed.dim() != 2 or scales.dim() != 2 or scales.shape[0] != packed.shape[0]:
        raise ValueError("packed must be [N, row bytes] and scales [N, K/G]")
    n, groups = scales.shape
    if groups < 1 or k % groups:
        raise ValueError(f"scales of {groups} groups do not cut rows of {k} weights evenly")
    _need_shape(packed, "packed", (n, (k + 127) // 128 * 64))
    if zeros is not None:
        _need_cuda(zeros, "zeros", torch.int8)
        _need_shape(zeros, "zeros", (n, groups))
    return n, k // groups


def pack_weights_w4(w, group=128, with_zeros=False):
    """float32 w [N, K] -> (packed uint8 [N, 64 * ceil(K / 128)], scales
    bfloat16 [N, K / group], zeros int8 [N, K / group] or None); group 32, 64
    or 128."""
    lib = _load()
    _need_cuda(w, "w", torch.float32)
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    n, k = w.shape
    group, dev = int(group), w.device
    if group not in (32, 64, 128) or k % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide K={k}, got {group}")
    packed = torch.empty((n, (k + 127) // 128 * 64), dtype=torch.uint8, device=dev)
    scales = torch.empty((n, k // group), dtype=torch.bfloat16, device=dev)
    zeros = torch.empty((n, k // group), dtype=torch.int8, device=dev) if with_zeros else None
    with binding.on_device(dev):
        _check(lib.bitlinear_pack_weights_w4(_ptr(w), n, k, group, _ptr(packed), _ptr(scales),
                                             _ptr(zeros), _stream(dev)))
    return packed, scales, zeros


def unpack_weights_w4(packed, scales, zeros, k):
    """The float32 values [N, k] that a packed matrix stands for."""
    lib = _load()
    k = int(k)
    n, group = _matrix(packed, scales, zeros, k)
    _same_device("unpack_weights_w4", packed, scales, zeros)
    dev = packed.device
    w = torch.empty((n, k), dtype=torch.float32, device=dev)
    with binding.on_device(dev):
        _check(lib.bitlinear_unpack_weights_w4(_ptr(packed), _ptr(scales), _ptr(zeros), n, k, group,
                                               _ptr(w), _stream(dev)))
    return w


def forward_w4(packed, scales, xq, absmax, zeros=None, out=None):
    """y float32 [T, N] = tokens of step A1 (xq int8 [T, K], absmax float32
    [T], from quant_act or subln_quant_act) times a 4-bit matrix."""
    lib = _load()
    _need_cuda(xq, "xq", torch.int8)
    _need_cuda(absmax, "absmax", torch.float32)
    if xq.dim() != 2:
        raise ValueError("xq must be [T, K]")
    t, k = xq.shape
    n, group = _matrix(packed, scales, zeros, k)
    _need_shape(absmax, "absmax", (t,))
    dev = xq.device
    if out is None:
        y = torch.empty((t, n), dtype=torch.float32, device=dev)
    else:
        _need_cuda(out, "out", torch.float32)
        _need_shape(out, "out", (t, n))
        y = out
    _same_device("forward_w4", packed, scales, zeros, xq, absmax, y)
    with binding.on_device(dev):
        _check(lib.bitlinear_forward_w4(_ptr(packed), _ptr(scales), _ptr(zeros), _ptr(xq),
                                        _ptr(absmax), t, n, k, group, _ptr(y), _stream(dev)))
    return y
