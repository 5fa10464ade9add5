"""4-bit products that reach every kernel variant of csrc/w4_plan.h on 256 CUs,
and the result from the definition in binary64, on whatever device the inputs are."""

import torch

from oracle import w4_ref as ref

# variant (wn, wk, wmf) -> (T, N) with whole and partial tiles both ways, and
# (G, K): one to five steps of 128 k per group of waves, a half last block or a
# whole one, groups of waves with fewer steps than the others or none
TILED = {
    (1, 8, 1): [(50, 1000, [(32, 1120), (32, 2176), (64, 320), (64, 2560), (128, 1280), (128, 3200)])],
    (2, 4, 1): [(70, 4000, [(32, 416), (32, 1184), (32, 1280), (64, 640), (64, 960), (128, 1280), (128, 384)])],
    (4, 2, 1): [(130, 4100, [(32, 416), (32, 640), (64, 320), (64, 256), (128, 384), (128, 768)])],
    (8, 1, 4): [(1300, 4200, [(128, 384), (128, 640), (128, 128), (128, 512)])],
    (4, 1, 2): [(1100, 2500, [(32, 416), (32, 640), (64, 320), (64, 256), (128, 384), (128, 128)])],
    (4, 1, 1): [(500, 2100, [(32, 416), (32, 640), (64, 320), (64, 256), (128, 384), (128, 128)])],
}

# few tokens: (T, N, K, G); teams of 1, 2, 4 and 8 waves for one token and for
# several, every group size
TEAMS = [(t, n, k, g) for t, shapes in (
    (1, [(40000, 512), (20000, 672), (10000, 1344), (300, 2656)]),
    (7, [(17000, 512), (10000, 672), (5000, 1344), (300, 2656)]))
    for n, k in shapes for g in (32, 64, 128) for k in (k // g * g,)]
# several tiles and several load groups per wave: one wave a team, and teams that
# come round again with one long token per block
ROUNDS = [(t, 70000, k, g) for t in (1, 7) for g, k in ((32, 672), (64, 704), (128, 640))]
ROUNDS += [(1, 8200, 65536, 128), (1, 8200, 65568, 32)]
# two passes over the matrix, the second with several tokens or with one
PASSES = [(16, 300, 14336, 32), (11, 300, 14336, 64), (16, 300, 14400, 64), (13, 260, 14336, 128), (2, 40, 131072, 128)]
# up to 16 tokens on the tiled kernel: longer rows than LDS has room for
LONG = [(12, 5000, 14336, 64), (16, 9000, 12288, 128), (16, 4100, 9632, 32), (3, 33, 131072, 128)]
# the same over so many rows that larger tiles take them, with one partial row block
WIDE = [(16, 20000, 12288, 64), (16, 35000, 9856, 32), (16, 41000, 9728, 64), (16, 41000, 9728, 128)]

FEW = TEAMS + ROUNDS + PASSES
CASES = [(t, n, k, g) for shapes in TILED.values() for t, n, gk in shapes for g, k in gk] + FEW + LONG + WIDE


def forward(packed, scales, zeros, xq, absmax):
    """(y, sum over groups of |s * group sum| * m / 127), both binary64 [T, N]."""
    on, (t, k), (n, groups) = xq.device, xq.shape, scales.shape
    g = k // groups
    byte, shift = (v.to(on) for v in ref.place(torch.arange(k)))
    y = torch.zeros(t, n, dtype=torch.float64, device=on)
    size = torch.zeros_like(y)
    q = xq.double()
    step = max(1, (1 << 27) // k)
    for r in range(0, n, step):
        c = (packed[r:r + step, byte].int() >> shift) & 15
        d = (c - 16 * (c > 7)).double()
        if zeros is not None:
            d -= zeros[r:r + step].double().repeat_interleave(g, 1)
        s = scales[r:r + step].double()
        for i in range(groups):
            at = slice(i * g, (i + 1) * g)
            part = (q[:, at] @ d[:, at].t()) * s[:, i]       # whole numbers below 2^53, then one product
            y[:, r:r + step] += part
            size[:, r:r + step] += part.abs()
    m = absmax.clamp_min(torch.tensor(1e-5, device=on)).double()[:, None] / 127
    return y * m, size * m
