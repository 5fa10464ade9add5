"""CPU oracle of the 8-bit floating point format with a scale for each block
of 128, and of the residual's addition in front of the norms.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see the package docstring).

No page gives an 8-bit floating point format; the reading is the library's own.
Codes are e4m3 (sign, 4 exponent bits of bias 7, 3 significand bits, subnormals,
0x7f and 0xff not numbers, largest value 448).  A group with m = max |v| is held
as code = e4m3(RN32(v * RN32(448 / m'))), scale = RN32(m' / 448), with
m' = max(m, 2^-100).
"""

import numpy as np

from .bitlinear_ref import quant_act, widen_bf16
from .ffn_ref import bf16_rne
from .subln_ref import EPS_N, normalise

FLOOR = np.float32(2.0 ** -100)
TOP = np.float32(448)
BLOCK = 128


def e4m3_values():
    """The value of every code byte (NaN for the two that are not numbers)."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(float) - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7, -v, v)


def e4m3(v):
    """Code bytes of values of magnitude up to about 448: nearest, ties to the even
    code (neighbouring codes of one sign are neighbouring numbers)."""
    v = np.asarray(v, np.float64)
    grid = e4m3_values()[:127]                      # rising
    m = np.abs(v)
    assert np.all(m < 464)                          # 448 (1 + a rounding) is 448
    hi = np.clip(np.searchsorted(grid, m), 1, 126)  # grid[hi - 1] < m <= grid[hi], or m = 0
    down, up = m - grid[hi - 1], grid[hi] - m
    c = np.where(down < up, hi - 1, np.where(up < down, hi, np.where(hi % 2 == 0, hi, hi - 1)))
    return (c + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _codes(v, m):
    """Codes and scale of binary32 values with group maxima m."""
    m = np.maximum(np.asarray(m, np.float32), FLOOR)
    return e4m3(v * (TOP / m)), m / TOP


def _as_f32(x):
    x = np.asarray(x)
    return widen_bf16(x) if x.dtype == np.uint16 else np.asarray(x, np.float32)


def quant_act_f8(x):
    """(codes uint8 [T, K], scales float32 [groups, T])."""
    x = _as_f32(x)
    t, k = x.shape
    q = np.empty((t, k), np.uint8)
    s = np.empty(((k + BLOCK - 1) // BLOCK, t), np.float32)
    for g in range(s.shape[0]):
        v = x[:, g * BLOCK:(g + 1) * BLOCK]
        c, sc = _codes(v, np.abs(v).max(1, keepdims=True))
        q[:, g * BLOCK:(g + 1) * BLOCK], s[g] = c, sc[:, 0]
    return q, s


def pack_weights_f8(w):
    """(codes uint8 [N, K], scales float32 [row blocks, column blocks])."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    q = np.empty((n, k), np.uint8)
    s = np.empty(((n + BLOCK - 1) // BLOCK, (k + BLOCK - 1) // BLOCK), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK)
            q[at], s[i, j] = _codes(w[at], np.abs(w[at]).max())
    return q, s


def weights(codes, scales):
    """The values that a matrix stands for, binary64 (not rounded)."""
    n, k = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0)[:n], BLOCK, 1)[:, :k]
    return e4m3_values()[codes] * s


def tokens(codes, scales):
    """The values that tokens stand for, binary64."""
    return e4m3_values()[codes] * np.repeat(scales.T.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]


def forward_f8(codes, w_scales, xq, x_scales):
    """(y binary64 [T, N], the sums of the products' magnitudes)."""
    w, x = weights(codes, w_scales), tokens(xq, x_scales)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def add(x, residual):
    """total as the residual is held: float32, or bfloat16 bit patterns."""
    total = _as_f32(x) + _as_f32(residual)          # one binary32 addition
    return bf16_rne(total) if np.asarray(residual).dtype == np.uint16 else total


def add_subln_quant_act(x, residual, gain, eps_n=EPS_N):
    """(total, codes int8, absmax, rowsum)."""
    total = x if residual is None else add(x, residual)
    xh, _ = normalise(total, gain, eps_n)
    return total, *quant_act(xh)


def add_subln_quant_act_f8(x, residual, gain, eps_n=EPS_N):
    """(total, codes uint8, scales [groups, T])."""
    total = x if residual is None else add(x, residual)
    xh, _ = normalise(total, gain, eps_n)
    return total, *quant_act_f8(xh)
