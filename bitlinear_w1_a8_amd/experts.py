"""Routed experts (include/bitlinear_experts.h), same names: the router, the
experts' gated feed-forward half and their linear layers.

Argument marshalling only, as ``binding``: tensors are allocated with torch on
the caller's device and every step runs in the library's HIP kernels on the
current stream of that device.
"""

import ctypes

import torch

from . import binding
from .binding import (BL_BF16, BL_F32, _c_i64, _c_int, _c_sz, _c_vp, _check, _need_cuda, _need_shape,
                      _ptr, _same_device, _stream)

#: most experts and most experts per token that the library takes
MAX_EXPERTS, MAX_TOP_K = 1024, 32
#: what a token's weights add up to (bl_share)
SHARES = {"chosen": 0, "all": 1}
_TOKENS, _SLOTS = 0, 1                       # bl_rows
_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}


class BlRouting(ctypes.Structure):
    """struct bl_routing of include/bitlinear_experts.h."""
    _fields_ = [("T", _c_i64), ("k", _c_i64), ("E", _c_i64), ("offsets", _c_vp), ("pairs", _c_vp),
                ("slots", _c_vp), ("weights", _c_vp)]


_ROUTING = ctypes.POINTER(BlRouting)

# name -> (restype, argtypes), as declared in include/bitlinear_experts.h
SIGNATURES = {
    "bitlinear_route_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "bitlinear_route_experts": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_vp,
                                         _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "bitlinear_gated_relu2_experts": (_c_int, [_ROUTING, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_i64,
                                               _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "bitlinear_experts_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "bitlinear_linear_experts": (_c_int, [_ROUTING, _c_vp, _c_int, _c_int, _c_vp, _c_vp, _c_i64,
                                          _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz,
                                          _c_vp]),
}

_lib = None


def _load():
    global _lib
    if _lib is None:
        _lib = binding.declare(SIGNATURES)
    return _lib


class Routing:
    """Where a batch of tokens goes: what route_experts returns and the
    experts' products take.  T tokens, k experts each, P = T * k pairs:

    ids      int32 [T, k]    experts of each token by falling logit, -1 for none
    weights  float32 [T, k]  their weights, 0 for none
    offsets  int32 [E + 1]   first slot of each expert, then the slots in use
    pairs    int32 [P]       pair (token * k + rank) of each slot, -1 in empty ones
    slots    int32 [T, k]    slot of each pair, -1 for none
    """

    __slots__ = ("ids", "weights", "offsets", "pairs", "slots")

    def __init__(self, ids, weights, offsets, pairs, slots):
        self.ids, self.weights, self.offsets, self.pairs, self.slots = ids, weights, offsets, pairs, slots

    def _struct(self, name, x):
        """Checked against the shapes that the library reads, and as its struct."""
        if self.slots.dim() != 2:
            raise ValueError("routing.slots must be [T, k]")
        t, k = self.slots.shape
        e = self.offsets.numel() - 1
        for field in ("offsets", "pairs", "slots"):
            _need_cuda(getattr(self, field), f"routing.{field}", torch.int32)
        _need_cuda(self.weights, "routing.weights", torch.float32)
        _need_shape(self.offsets, "routing.offsets", (e + 1,))
        _need_shape(self.pairs, "routing.pairs", (t * k,))
        _need_shape(self.weights, "routing.weights", (t, k))
        _same_device(name, x, self.offsets, self.pairs, self.slots, self.weights)
        return t, k, e, BlRouting(t, k, e, self.offsets.data_ptr(), self.pairs.data_ptr(),
                                  self.slots.data_ptr(), self.weights.data_ptr())


def route_experts(logits, k, share="chosen"):
    """The router: logits [T, E] (float32 or bfloat16) -> Routing over each
    token's k largest logits (ties to the lower expert; -inf and NaN never
    taken).  share: "chosen" (softmax over the chosen logits) or "all"."""
    lib = _load()
    _need_cuda(logits, "logits")
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if share not in SHARES:
        raise ValueError(f"share must be one of {sorted(SHARES)}, got {share!r}")
    t, e = logits.shape
    k, dev = int(k), logits.device
    if k < 1:
        raise ValueError(f"k must be at least 1, got {k}")
    ids = torch.empty((t, k), dtype=torch.int32, device=dev)
    weights = torch.empty((t, k), dtype=torch.float32, device=dev)
    offsets = torch.empty(e + 1, dtype=torch.int32, device=dev)
    pairs = torch.empty(t * k, dtype=torch.int32, device=dev)
    slots = torch.empty((t, k), dtype=torch.int32, device=dev)
    wsb = lib.bitlinear_route_workspace_bytes(t, e)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    with binding.on_device(dev):
        _check(lib.bitlinear_route_experts(_ptr(logits), dt, t, e, k, SHARES[share], _ptr(ids),
                                           _ptr(weights), _ptr(offsets), _ptr(pairs), _ptr(slots),
                                           _ptr(ws), wsb, _stream(dev)))
    return Routing(ids, weights, offsets, pairs, slots)


def _rows(x, name, rows, what):
    _need_cuda(x, name)
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"{name} must have one row per {what}: [{rows}, K], got {tuple(x.shape)}")
    return dt


def _out(out, name, shape, dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need_cuda(out, name, dtype)
    _need_shape(out, name, shape)
    return out


def gated_relu2_experts(x, packed_gu, gamma_gate, gamma_up, routing, want_acc=False, out=None):
    """Gate and up projections of the routed tokens with the squared-ReLU gate.

    x [T, K] (float32 or bfloat16); packed_gu uint8 [E, 2N, K/4], each
    expert's rows from interleave_rows; gamma_gate, gamma_up float32 [E].
    Returns (h bfloat16 [T * k, N] by slot, xq, absmax, acc int32 [T * k, 2N]
    or None).  Rows of empty slots are not written: undefined, or with `out`
    as they were."""
    lib = _load()
    t, k, e, desc = routing._struct("gated_relu2_experts", x)
    dt = _rows(x, "x", t, "token")
    kk = x.shape[1]
    _need_cuda(packed_gu, "packed_gu", torch.uint8)
    _need_cuda(gamma_gate, "gamma_gate", torch.float32)
    _need_cuda(gamma_up, "gamma_up", torch.float32)
    if packed_gu.dim() != 3 or packed_gu.shape[1] % 2:
        raise ValueError("packed_gu must be [E, 2N, K/4]")
    n = packed_gu.shape[1] // 2
    _need_shape(packed_gu, "packed_gu", (e, 2 * n, kk // 4))
    _need_shape(gamma_gate, "gamma_gate", (e,))
    _need_shape(gamma_up, "gamma_up", (e,))
    dev = x.device
    h = _out(out, "out", (t * k, n), torch.bfloat16, dev)
    _same_device("gated_relu2_experts", x, packed_gu, gamma_gate, gamma_up, h)
    xq = torch.empty((t, kk), dtype=torch.int8, device=dev)
    absmax = torch.empty(t, dtype=torch.float32, device=dev)
    acc = torch.empty((t * k, 2 * n), dtype=torch.int32, device=dev) if want_acc else None
    with binding.on_device(dev):
        _check(lib.bitlinear_gated_relu2_experts(ctypes.byref(desc), _ptr(x), dt, _ptr(packed_gu),
                                                 _ptr(gamma_gate), _ptr(gamma_up), n, kk, _ptr(h),
                                                 _ptr(xq), _ptr(absmax), _ptr(acc), _stream(dev)))
    return h, xq, absmax, acc


def linear_experts(x, packed, gamma, routing, combine=True, x_rows="slots", want_acc=False, out=None):
    """One BitLinear per expert over the routed rows.

    x (float32 or bfloat16): one row per slot, [T * k, K] (x_rows "slots", as
    gated_relu2_experts writes them), or one per token, [T, K] ("tokens");
    packed uint8 [E, N, K/4], gamma float32 [E].  Returns y float32: with
    `combine` the weighted sum over each token's experts, [T, N]; without, one
    row per slot, [T * k, N], rows of empty slots not written (undefined, or
    with `out` as they were), and (y, acc int32) if want_acc."""
    lib = _load()
    t, k, e, desc = routing._struct("linear_experts", x)
    if x_rows not in ("slots", "tokens"):
        raise ValueError(f"x_rows must be 'slots' or 'tokens', got {x_rows!r}")
    if combine and want_acc:
        raise ValueError("want_acc: the sums are per slot (combine=False only)")
    by_slot = x_rows == "slots"
    rows = t * k if by_slot else t
    dt = _rows(x, "x", rows, "slot" if by_slot else "token")
    kk = x.shape[1]
    _need_cuda(packed, "packed", torch.uint8)
    _need_cuda(gamma, "gamma", torch.float32)
    if packed.dim() != 3:
        raise ValueError("packed must be [E, N, K/4]")
    n = packed.shape[1]
    _need_shape(packed, "packed", (e, n, kk // 4))
    _need_shape(gamma, "gamma", (e,))
    dev = x.device
    y = _out(out, "out", (t if combine else t * k, n), torch.float32, dev)
    _same_device("linear_experts", x, packed, gamma, y)
    xq = torch.empty((rows, kk), dtype=torch.int8, device=dev)
    absmax = torch.empty(rows, dtype=torch.float32, device=dev)
    acc = torch.empty((t * k, n), dtype=torch.int32, device=dev) if want_acc else None
    wsb = lib.bitlinear_experts_workspace_bytes(t, k, n) if combine else 0
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if combine else None
    with binding.on_device(dev):
        _check(lib.bitlinear_linear_experts(ctypes.byref(desc), _ptr(x), dt,
                                            _SLOTS if by_slot else _TOKENS, _ptr(packed),
                                            _ptr(gamma), n, kk, _ptr(y),
                                            _TOKENS if combine else _SLOTS, _ptr(xq),
                                            _ptr(absmax), _ptr(acc), _ptr(ws), wsb, _stream(dev)))
    return (y, acc) if want_acc else y
