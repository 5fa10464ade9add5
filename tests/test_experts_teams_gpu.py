"""The one-launch weighted sum with every way it shares a row between waves
(needs an MI355X).

A token's k slots have a team of min(16 / k, chunks of 256 in K / 4) waves
each; a wave quantises its chunks into LDS and reads them back across its
lanes.  Teams of one to sixteen waves, runs of one chunk to more than the
four that a wave holds in registers, runs that the last wave has fewer of or
none, rows that end inside a chunk.  Bounds as in test_experts_gpu."""

import numpy as np
import pytest

import oracle
from oracle import experts_ref as ref
from tests.test_experts_gpu import U, activations, bl, dev, host, routing, weights  # noqa: F401

pytestmark = pytest.mark.gpu

# (T, E, k, N, K, dtype): all within 32 pairs
CASES = [(1, 3, 1, 40, 16384, "bf16"), (2, 3, 1, 33, 32768, "bf16"), (1, 2, 1, 17, 20496, "f32"),
         (3, 4, 2, 50, 10240, "f32"), (2, 5, 3, 48, 5136, "bf16"), (3, 6, 4, 31, 4096, "bf16"),
         (2, 6, 5, 20, 4112, "f32"), (4, 8, 8, 64, 2304, "bf16"), (2, 16, 9, 18, 8192, "bf16"),
         (2, 16, 16, 35, 8192, "f32"), (1, 16, 16, 16, 80, "bf16"), (32, 2, 1, 24, 1296, "bf16")]


@pytest.mark.parametrize("t,e,k,n,kk,dtype", CASES,
                         ids=[f"T{c[0]}_E{c[1]}_k{c[2]}_N{c[3]}_K{c[4]}_{c[5]}" for c in CASES])
def test_weighted_sum_of_every_team(bl, t, e, k, n, kk, dtype):  # noqa: F811
    rng = np.random.default_rng(t + n)
    r, off, pairs, slots, w = routing(bl, t, e, k, 41 * t + e)
    tern, packed, gam = weights(rng, e, n, kk)
    for x_rows in ("slots", "tokens"):
        xin, xref = activations(t * k if x_rows == "slots" else t, kk, 9 + t, dtype)
        q, a, _ = oracle.quant_act(xref)
        at = np.arange(t * k) if x_rows == "slots" else np.maximum(pairs, 0) // k
        y_ref, _ = ref.linear_slots(q, a, tern, gam, off, at)
        both, size = ref.combine(y_ref, slots, w)
        got = host(bl.linear_experts(xin, packed, dev(gam), r, x_rows=x_rows)).astype(np.float64)
        assert np.all(np.abs(got - both) <= (k + 5) * U * size)
