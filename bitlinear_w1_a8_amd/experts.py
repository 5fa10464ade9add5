"""Routed experts (include/bitlinear_experts.h), same names: the router, the
experts' gated feed-forward half, their linear layers, and all three as one
layer.

Argument marshalling only, as ``binding``: tensors are allocated with torch on
the caller's device and every step runs in the library's HIP kernels on the
current stream of that device.
"""

import functools
import operator
import struct

import torch

from . import binding
from ._marshal import call, device_of, need
from .binding import BL_BF16, BL_F32, _c_i64, _c_int, _c_sz, _c_vp

#: most experts and most experts per token that the library takes
MAX_EXPERTS, MAX_TOP_K = 1024, 32
#: what a token's weights add up to (bl_share)
SHARES = {"chosen": 0, "all": 1}
_TOKENS, _SLOTS = 0, 1                       # bl_rows
_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}
_CODES = 2                                   # BL_CODES


#: struct bl_routing: T, k, E, then the pointers offsets, pairs, slots, weights
_ROUTING = struct.Struct("=7q")

# name -> (restype, argtypes), as declared in include/bitlinear_experts.h
SIGNATURES = {
    "bitlinear_route_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "bitlinear_route_experts": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_vp,
                                         _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "bitlinear_gated_relu2_experts": (_c_int, [_c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_i64,
                                               _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "bitlinear_experts_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "bitlinear_linear_experts": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp, _c_vp, _c_i64,
                                          _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz,
                                          _c_vp]),
    "bitlinear_experts_ffn_workspace_bytes": (_c_sz, [_c_i64] * 6),
    "bitlinear_experts_ffn": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_int,
                                       _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp,
                                       _c_i64, _c_vp, _c_vp, _c_sz, _c_vp]),
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

    def _struct(self, dev):
        """Checked against the shapes that the library reads, and as its struct."""
        slots, offsets = self.slots, self.offsets
        if slots.dim() != 2:
            raise ValueError("routing.slots must be [T, k]")
        shape = slots.shape
        t, k = shape
        e = offsets.numel() - 1
        need(dev, slots, "routing.slots", torch.int32, shape)
        need(dev, offsets, "routing.offsets", torch.int32, (e + 1,))
        need(dev, self.pairs, "routing.pairs", torch.int32, (t * k,))
        need(dev, self.weights, "routing.weights", torch.float32, shape)
        return t, k, e, _ROUTING.pack(t, k, e, offsets.data_ptr(), self.pairs.data_ptr(),
                                      slots.data_ptr(), self.weights.data_ptr())


def route_experts(logits, k, share="chosen"):
    """The router: logits [T, E] (float32 or bfloat16) -> Routing over each
    token's k largest logits (ties to the lower expert; -inf and NaN never
    taken).  share: "chosen" (softmax over the chosen logits) or "all".  The
    int32 arrays are views of one allocation."""
    lib = _load()
    dev = device_of(logits, "logits")
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if share not in SHARES:
        raise ValueError(f"share must be one of {sorted(SHARES)}, got {share!r}")
    t, e = shape = logits.shape
    need(dev, logits, "logits", logits.dtype, shape)
    k = operator.index(k)
    if not 1 <= k <= MAX_TOP_K:              # before anything of that size is allocated
        raise ValueError(f"k must be in [1, {MAX_TOP_K}], got {k}")
    on, p = logits.device, t * k
    wsb = lib.bitlinear_route_workspace_bytes(t, e)
    weights = torch.empty((t, k), dtype=torch.float32, device=on)
    # the int32 arrays in one piece: 0.9 us less on the host than one by one.  The
    # scratch is not part of it: it goes back to the allocator, however long they are kept
    ids, slots, pairs, offsets = torch.empty(
        3 * p + e + 1, dtype=torch.int32, device=on).split_with_sizes((p, p, p, e + 1))
    ids, slots = ids.view(t, k), slots.view(t, k)
    ws = torch.empty(wsb, dtype=torch.uint8, device=on) if wsb else None
    call(dev, lib.bitlinear_route_experts, logits.data_ptr(), dt, t, e, k, SHARES[share],
         ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), pairs.data_ptr(),
         slots.data_ptr(), ws.data_ptr() if wsb else None, wsb)
    return Routing(ids, weights, offsets, pairs, slots)


def _rows(dev, x, rows, what):
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"x must have one row per {what}: [{rows}, K], got {tuple(x.shape)}")
    need(dev, x, "x", x.dtype, x.shape)
    return dt, x.shape[1]


def _out(dev, out, shape, dtype, on):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=on)
    need(dev, out, "out", dtype, shape)
    return out


def _up(n):
    return (n + 255) & ~255


def gated_relu2_experts(x, packed_gu, gamma_gate, gamma_up, routing, want_codes=False,
                        want_acc=False, out=None):
    """Gate and up projections of the routed tokens with the squared-ReLU gate.

    x [T, K] (float32 or bfloat16); packed_gu uint8 [E, 2N, K/4], each
    expert's rows from interleave_rows; gamma_gate, gamma_up float32 [E].
    Returns (h bfloat16 [T * k, N] by slot, xq int8 [T, K] and absmax float32
    [T] of the tokens with an expert or None without `want_codes`, acc int32
    [T * k, 2N] or None without `want_acc`).  Rows of empty slots are not
    written: undefined, or with `out` as they were."""
    lib = _load()
    dev = device_of(x, "x")
    t, k, e, desc = routing._struct(dev)
    dt, kk = _rows(dev, x, t, "token")
    if packed_gu.dim() != 3 or packed_gu.shape[1] % 2:
        raise ValueError("packed_gu must be [E, 2N, K/4]")
    n = packed_gu.shape[1] // 2
    need(dev, packed_gu, "packed_gu", torch.uint8, (e, 2 * n, kk // 4))
    need(dev, gamma_gate, "gamma_gate", torch.float32, (e,))
    need(dev, gamma_up, "gamma_up", torch.float32, (e,))
    on = x.device
    h = _out(dev, out, (t * k, n), torch.bfloat16, on)
    if want_codes:
        xq = torch.empty((t, kk), dtype=torch.int8, device=on)
        absmax = torch.empty(t, dtype=torch.float32, device=on)
        codes = xq.data_ptr(), absmax.data_ptr()
    else:                       # scratch, in one piece
        xq = absmax = None
        scratch = torch.empty(_up(t * kk) + 4 * t, dtype=torch.uint8, device=on)
        at = scratch.data_ptr()
        codes = at, at + _up(t * kk)
    acc = torch.empty((t * k, 2 * n), dtype=torch.int32, device=on) if want_acc else None
    call(dev, lib.bitlinear_gated_relu2_experts, desc, x.data_ptr(), dt, packed_gu.data_ptr(),
         gamma_gate.data_ptr(), gamma_up.data_ptr(), n, kk, h.data_ptr(), *codes,
         acc.data_ptr() if want_acc else None)
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
    dev = device_of(x, "x")
    t, k, e, desc = routing._struct(dev)
    if x_rows not in ("slots", "tokens"):
        raise ValueError(f"x_rows must be 'slots' or 'tokens', got {x_rows!r}")
    if combine and want_acc:
        raise ValueError("want_acc: the sums are per slot (combine=False only)")
    by_slot = x_rows == "slots"
    rows = t * k if by_slot else t
    dt, kk = _rows(dev, x, rows, "slot" if by_slot else "token")
    if packed.dim() != 3:
        raise ValueError("packed must be [E, N, K/4]")
    n = packed.shape[1]
    need(dev, packed, "packed", torch.uint8, (e, n, kk // 4))
    need(dev, gamma, "gamma", torch.float32, (e,))
    on = x.device
    y = _out(dev, out, (t if combine else t * k, n), torch.float32, on)
    acc = torch.empty((t * k, n), dtype=torch.int32, device=on) if want_acc else None
    # the int8 rows, their absmax and the slots' rows, in one piece
    wsb = lib.bitlinear_experts_workspace_bytes(t, k, n) if combine else 0
    a, b = _up(rows * kk), _up(4 * rows)
    scratch = torch.empty(a + b + wsb, dtype=torch.uint8, device=on)
    at = scratch.data_ptr()
    call(dev, lib.bitlinear_linear_experts, desc, x.data_ptr(), dt, _SLOTS if by_slot else _TOKENS,
         packed.data_ptr(), gamma.data_ptr(), n, kk, y.data_ptr(), _TOKENS if combine else _SLOTS,
         at, at + a, acc.data_ptr() if want_acc else None, at + a + b if combine else None, wsb)
    return (y, acc) if want_acc else y


@functools.lru_cache(maxsize=256)
def _ffn_workspace(*sizes):
    """The library's answer, which depends on these sizes alone."""
    return _load().bitlinear_experts_ffn_workspace_bytes(*sizes)


def experts_ffn(x, logits, k, packed_gu, gamma_gate, gamma_up, packed_down, gamma_down, absmax=None,
                share="chosen", out=None):
    """A whole routed layer, the same bits as route_experts, gated_relu2_experts
    and linear_experts one after the other; for up to 16 tokens in two launches
    (three where more than a few are not quantised yet), if k <= 16, E <= 256,
    N < 2^25, and T int8 rows of K and k of F fit 150 KiB each.

    x [T, K]: float32 or bfloat16, or int8 codes with their ``absmax`` float32
    [T] (quant_act, subln_quant_act, add_subln_quant_act); logits [T, E] (float32
    or bfloat16); packed_gu uint8 [E, 2F, K/4], each expert's rows from
    interleave_rows; packed_down uint8 [E, N, F/4]; the gammas float32 [E].
    Returns y float32 [T, N]."""
    lib = _load()
    dev = device_of(x, "x")
    if x.dtype is torch.int8:
        if absmax is None:
            raise ValueError("int8 codes need their absmax")
        dt = _CODES
    else:
        dt = _DTYPES.get(x.dtype)
        if dt is None:
            raise TypeError(f"x must be float32, bfloat16 or int8 codes, got {x.dtype}")
        if absmax is not None:
            raise ValueError("absmax belongs to int8 codes")
    device_of(logits, "logits")
    lt = _DTYPES.get(logits.dtype)
    if lt is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if x.dim() != 2 or logits.dim() != 2 or packed_gu.dim() != 3 or packed_down.dim() != 3:
        raise ValueError("x must be [T, K], logits [T, E], packed_gu [E, 2F, K/4], packed_down [E, N, F/4]")
    if share not in SHARES:
        raise ValueError(f"share must be one of {sorted(SHARES)}, got {share!r}")
    t, kk = shape = x.shape
    e = logits.shape[1]
    f, n = packed_gu.shape[1] // 2, packed_down.shape[1]
    k = operator.index(k)
    if not 1 <= k <= MAX_TOP_K:
        raise ValueError(f"k must be in [1, {MAX_TOP_K}], got {k}")
    need(dev, x, "x", x.dtype, shape)
    need(dev, logits, "logits", logits.dtype, (t, e))
    need(dev, packed_gu, "packed_gu", torch.uint8, (e, 2 * f, kk // 4))
    need(dev, packed_down, "packed_down", torch.uint8, (e, n, f // 4))
    need(dev, gamma_gate, "gamma_gate", torch.float32, (e,))
    need(dev, gamma_up, "gamma_up", torch.float32, (e,))
    need(dev, gamma_down, "gamma_down", torch.float32, (e,))
    if absmax is not None:
        need(dev, absmax, "absmax", torch.float32, (t,))
    on = x.device
    y = _out(dev, out, (t, n), torch.float32, on)
    wsb = _ffn_workspace(t, e, k, f, kk, n)
    ws = torch.empty(wsb, dtype=torch.uint8, device=on)
    call(dev, lib.bitlinear_experts_ffn, logits.data_ptr(), lt, t, e, k, SHARES[share], x.data_ptr(),
         dt, None if absmax is None else absmax.data_ptr(), packed_gu.data_ptr(),
         gamma_gate.data_ptr(), gamma_up.data_ptr(), f, kk, packed_down.data_ptr(),
         gamma_down.data_ptr(), n, y.data_ptr(), ws.data_ptr(), wsb)
    return y
