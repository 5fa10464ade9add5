"""CPU oracle of the routed-expert layers.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see the package docstring).

"BitNet解读" (future work) names 1-bit mixtures of experts and gives no
method.  Reading (stated): a token's experts are its k largest router logits,
ties to the lower expert, masked (-inf) and NaN entries never taken; their
weights are the softmax over the chosen logits or over all usable ones; every
expert is a BitLinear with a matrix and gamma of its own; a token's output is
the weighted sum of its experts' outputs.
"""

import math

import numpy as np

from .bitlinear_ref import contract, rescale
from .ffn_ref import gated_relu2


def route(logits, k, share="chosen"):
    """(ids [T, k], weights binary64 [T, k], offsets [E + 1], pairs [T * k],
    slots [T, k]), entry by entry from the definition."""
    logits = np.asarray(logits, np.float32)
    t_n, e_n = logits.shape
    ids = np.full((t_n, k), -1, np.int32)
    weights = np.zeros((t_n, k))
    for t in range(t_n):
        usable = [e for e in range(e_n) if logits[t, e] > -np.inf]
        order = sorted(usable, key=lambda e: (-float(logits[t, e]), e))
        chosen = order[:k]
        if not chosen:
            continue
        top = float(logits[t, chosen[0]])
        u = {e: 1.0 if float(logits[t, e]) == top else math.exp(float(logits[t, e]) - top)
             for e in usable}
        total = math.fsum(u[e] for e in (chosen if share == "chosen" else usable))
        for j, e in enumerate(chosen):
            ids[t, j] = e
            weights[t, j] = u[e] / total
    offsets = np.zeros(e_n + 1, np.int32)
    pairs = np.full(t_n * k, -1, np.int32)
    slots = np.full((t_n, k), -1, np.int32)
    place = 0
    flat = ids.reshape(-1)
    for e in range(e_n):
        offsets[e] = place
        for pair in np.nonzero(flat == e)[0]:
            pairs[place] = pair
            slots.reshape(-1)[pair] = place
            place += 1
    offsets[e_n] = place
    return ids, weights, offsets, pairs, slots


def _by_expert(offsets, fn):
    for e in range(len(offsets) - 1):
        p = np.arange(offsets[e], offsets[e + 1])
        if len(p):
            fn(e, p)


def linear_slots(q, absmax, tern, gammas, offsets, rows):
    """(y binary64 [P, N], acc int32 [P, N]) of the slots in use; rows[p] is
    the row of q of slot p.  Other rows are zero."""
    y = np.zeros((len(rows), tern.shape[1]))
    acc = np.zeros((len(rows), tern.shape[1]), np.int32)

    def one(e, p):
        acc[p] = contract(q[rows[p]], tern[e])
        y[p] = rescale(acc[p], gammas[e], absmax[rows[p]])
    _by_expert(offsets, one)
    return y, acc


def gated_slots(q, absmax, tern_gate, tern_up, gamma_gate, gamma_up, offsets, rows):
    """(h bfloat16 bits [P, N], acc int32 [P, 2N] interleaved) of the slots in use."""
    n = tern_gate.shape[1]
    h = np.zeros((len(rows), n), np.uint16)
    acc = np.zeros((len(rows), 2 * n), np.int32)

    def one(e, p):
        r = rows[p]
        acc[p, 0::2], acc[p, 1::2] = contract(q[r], tern_gate[e]), contract(q[r], tern_up[e])
        h[p] = gated_relu2(acc[p, 0::2], acc[p, 1::2], gamma_gate[e], gamma_up[e], absmax[r])
    _by_expert(offsets, one)
    return h, acc


def combine(y, slots, weights):
    """(sum_j w * y_slot, sum_j |w * y_slot|) per token, pairs without a slot left out."""
    t_n, k = slots.shape
    out, size = np.zeros((t_n, y.shape[1])), np.zeros((t_n, y.shape[1]))
    for t in range(t_n):
        for j in range(k):
            if slots[t, j] >= 0:
                part = float(weights[t, j]) * y[slots[t, j]]
                out[t] += part
                size[t] += np.abs(part)
    return out, size
