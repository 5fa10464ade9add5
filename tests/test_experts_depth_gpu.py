"""The decode kernel of the routed rows at every load depth (needs an MI355X;
test_experts_depth shows that the rows reach them): sums and gated outputs bit
for bit, rows within the bounds of test_experts_gpu."""

import numpy as np
import pytest
import torch

import oracle
from oracle import experts_ref as ref
from tests.test_experts_depth import ROWS
from tests.test_experts_gpu import U, activations, bits, bl, dev, host, routing, weights  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,dtype", [(3, "bf16"), (3, "f32"), (11, "bf16")], ids=["T3_bf16", "T3_f32", "T11"])
@pytest.mark.parametrize("kk", ROWS)
def test_rows(bl, kk, t, dtype):  # noqa: F811
    e, k, n = 6, 2, 37
    rng = np.random.default_rng(kk + t)
    r, off, pairs, _, _ = routing(bl, t, e, k, kk, "masked" if t > 4 else "normal")
    used = off[-1]
    tern, packed, gam = weights(rng, e, n, kk)
    xin, xref = activations(t, kk, 3 + t, dtype)
    q, a, _ = oracle.quant_act(xref)
    at = np.maximum(pairs, 0) // k
    y_ref, acc_ref = ref.linear_slots(q, a, tern, gam, off, at)
    y, acc = bl.linear_experts(xin, packed, dev(gam), r, combine=False, x_rows="tokens", want_acc=True)
    assert np.array_equal(host(acc)[:used], acc_ref[:used])
    assert np.all(np.abs(host(y).astype(np.float64) - y_ref)[:used] <= 4 * U * np.abs(y_ref)[:used])
    up, packed_up, gam_up = weights(rng, e, n, kk)
    both = torch.stack([bl.interleave_rows(packed[i], packed_up[i]) for i in range(e)])
    h, _, _, acc = bl.gated_relu2_experts(xin, both, dev(gam), dev(gam_up), r, want_acc=True)
    h_ref, acc_ref = ref.gated_slots(q, a, tern, up, gam, gam_up, off, at)
    assert np.array_equal(host(acc)[:used], acc_ref[:used])
    assert np.array_equal(bits(h)[:used], h_ref[:used])
