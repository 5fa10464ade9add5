"""CPU oracle of the 4-bit weights with group scales (W4A8).

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see the package docstring).

No page gives a 4-bit format; the reading is the library's own.  Quantisation
in binary32, one rounding per operation, the scale rounded to bfloat16 before
the codes are chosen:

    without zero points:  s = bf16(max |w| / 7),  t = clip(rint(w / s), -8, 7), z = 0
    with zero points:     lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15),
                          z = clip(rint(-lo / s), 0, 15) - 8,
                          t = clip(rint(w / s) + z, -8, 7)
    s = 0:                t = z = 0

A weight stands for (t - z) * s.  Storage: rows of 64 * ceil(K / 128) bytes;
in a block of 128, weight k sits in 16-byte chunk (k / 8) % 4, word k / 32,
byte k % 4, low nibble where k % 8 < 4, as two's complement.
"""

import numpy as np

from .bitlinear_ref import EPS_A, _check_finite
from .ffn_ref import bf16_rne


def _widen(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)


def quantize(w, group, with_zeros):
    """(t int8 [N, K], scale bfloat16 bits [N, K/G], z int8 [N, K/G])."""
    w = np.asarray(w, np.float32)
    _check_finite(w, "w")
    n, k = w.shape
    v = w.reshape(n, k // group, group)
    if with_zeros:
        lo = np.minimum(v.min(2), np.float32(0))
        hi = np.maximum(v.max(2), np.float32(0))
        bits = bf16_rne((hi - lo) / np.float32(15))
    else:
        bits = bf16_rne(np.abs(v).max(2) / np.float32(7))
    s = _widen(bits)
    d = np.where(s > 0, s, np.float32(1))
    if with_zeros:
        z = np.clip(np.rint(-lo / d), 0, 15) - 8
        z = np.where(s > 0, z, 0)
    else:
        z = np.zeros_like(s)
    t = np.clip(np.rint(v / d[:, :, None]) + z[:, :, None], -8, 7)
    t = np.where(s[:, :, None] > 0, t, 0)
    return t.reshape(n, k).astype(np.int8), bits, z.astype(np.int8)


def place(k):
    """(byte of the row, shift) of weight k."""
    return k // 128 * 64 + k // 8 % 4 * 16 + k % 128 // 32 * 4 + k % 4, 4 * (k % 8 // 4)


def pack(t):
    n, k = t.shape
    out = np.zeros((n, (k + 127) // 128 * 64), np.uint8)
    for i in range(k):
        byte, shift = place(i)
        out[:, byte] |= ((t[:, i].astype(np.uint8) & 15) << shift).astype(np.uint8)
    return out


def unpack(packed, k):
    byte, shift = place(np.arange(k))
    c = (packed[:, byte] >> shift) & 15
    return np.where(c > 7, c.astype(np.int16) - 16, c).astype(np.int8)


def values(t, bits, z):
    """(t - z) * s in binary64, [N, K]."""
    n, k = t.shape
    g = k // bits.shape[1]
    s = np.repeat(_widen(bits).astype(np.float64), g, axis=1)
    return (t.astype(np.float64) - np.repeat(z.astype(np.float64), g, axis=1)) * s


def forward(t, bits, z, q, absmax):
    """(y binary64 [T, N], sum over groups of |s * group sum| * m / 127)."""
    n, k = t.shape
    g = k // bits.shape[1]
    s = _widen(bits).astype(np.float64)
    d = (t.astype(np.int64) - np.repeat(z.astype(np.int64), g, axis=1)).astype(np.float64)
    q = np.asarray(q, np.float64)
    m = np.maximum(np.asarray(absmax, np.float32), EPS_A).astype(np.float64)[:, None] / 127.0
    y, size = np.zeros((q.shape[0], n)), np.zeros((q.shape[0], n))
    for i in range(k // g):
        part = (q[:, i * g:(i + 1) * g] @ d[:, i * g:(i + 1) * g].T) * s[:, i]   # integers below 2^53
        y += part
        size += np.abs(part)
    return y * m, size * m
