"""Pins of the routed-expert and 4-bit oracles (CPU): worked examples by hand,
invariants, and a second route to each result."""

import numpy as np
import pytest

from oracle import experts_ref, w4_ref
from oracle.bitlinear_ref import contract, rescale

NINF = -np.inf


def test_route_by_hand():
    # token 0: ties at 2.0 between experts 1 and 3; token 1: one usable; token 2: none
    logits = np.array([[0.0, 2.0, -1.0, 2.0], [NINF, NINF, 5.0, np.nan], [NINF] * 4], np.float32)
    ids, w, off, pairs, slots = experts_ref.route(logits, 2)
    assert ids.tolist() == [[1, 3], [2, -1], [-1, -1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]
    assert off.tolist() == [0, 0, 1, 2, 3]
    assert pairs.tolist() == [0, 2, 1, -1, -1, -1]
    assert slots.tolist() == [[0, 2], [1, -1], [-1, -1]]
    _, w, *_ = experts_ref.route(logits[:1], 1, "all")
    assert w[0, 0] == pytest.approx(1 / (2 + np.exp(-2) + np.exp(-3)), rel=1e-14)


def test_route_zero_signs_and_lowest_values():
    low = np.finfo(np.float32).min
    ids, w, *_ = experts_ref.route(np.array([[-0.0, 0.0, -1.0], [low, low, low]], np.float32), 2)
    assert ids.tolist() == [[0, 1], [0, 1]]
    assert w.tolist() == [[0.5, 0.5], [0.5, 0.5]]


@pytest.mark.parametrize("share", ["chosen", "all"])
def test_route_against_sorting(share):
    rng = np.random.default_rng(5)
    logits = rng.normal(0, 1, (40, 9)).round(1).astype(np.float32)      # with ties
    logits[rng.random((40, 9)) < 0.3] = NINF
    ids, w, off, pairs, slots = experts_ref.route(logits, 4, share)
    order = np.argsort(-logits, axis=1, kind="stable")[:, :4]
    keep = np.take_along_axis(logits, order, 1) > NINF
    assert np.array_equal(ids, np.where(keep, order, -1))
    flat = ids.reshape(-1)
    want = np.argsort(np.where(flat < 0, 99, flat), kind="stable")[: int((flat >= 0).sum())]
    assert np.array_equal(pairs[: off[-1]], want)
    assert np.all(pairs[off[-1]:] == -1)
    assert np.array_equal(np.diff(off), np.bincount(flat[flat >= 0], minlength=9))
    used = slots.reshape(-1) >= 0
    assert np.array_equal(pairs[slots.reshape(-1)[used]], np.nonzero(used)[0])
    total = w.sum(1)[keep.any(1)]
    assert np.all(total <= 1 + 1e-12) and (share == "all" or np.allclose(total, 1))


def test_slots_against_one_expert_per_row():
    rng = np.random.default_rng(6)
    q = rng.integers(-127, 128, (6, 32)).astype(np.int8)
    a = rng.uniform(0.5, 2, 6).astype(np.float32)
    tern = rng.integers(-1, 2, (3, 5, 32)).astype(np.int8)
    gam = rng.uniform(0.01, 0.02, 3).astype(np.float32)
    offsets, rows = np.array([0, 4, 4, 6]), np.array([5, 0, 2, 2, 1, 5])
    y, acc = experts_ref.linear_slots(q, a, tern, gam, offsets, rows)
    for p, e in enumerate([0, 0, 0, 0, 2, 2]):
        r = rows[p:p + 1]
        assert np.array_equal(acc[p:p + 1], contract(q[r], tern[e]))
        assert np.array_equal(y[p:p + 1], rescale(acc[p:p + 1], gam[e], a[r]))
    out, size = experts_ref.combine(y, np.array([[0, -1], [5, 2]]), np.array([[2.0, 9.0], [1.0, -1.0]]))
    assert np.allclose(out, [2 * y[0], y[5] - y[2]]) and np.all(size >= np.abs(out))


def test_w4_by_hand():
    w = np.zeros((1, 32), np.float32)
    w[0, :4] = [7.0, -3.5, 0.5, -7.0]            # s = 1: ties to even
    t, bits, z = w4_ref.quantize(w, 32, False)
    assert bits[0, 0] == 0x3F80 and t[0, :4].tolist() == [7, -4, 0, -7] and z[0, 0] == 0
    w[0, :4] = [10.0, -5.0, 1.5, 0.0]            # lo -5, hi 10: s = 1, z = 5 - 8
    t, bits, z = w4_ref.quantize(w, 32, True)
    assert bits[0, 0] == 0x3F80 and z[0, 0] == -3 and t[0, :4].tolist() == [7, -8, -1, -3]
    assert w4_ref.values(t, bits, z)[0, :4].tolist() == [10.0, -5.0, 2.0, 0.0]
    t, bits, z = w4_ref.quantize(np.zeros((1, 32), np.float32), 32, True)
    assert not t.any() and not bits.any() and not z.any()


def test_w4_layout_by_hand():
    t = np.zeros((1, 160), np.int8)
    t[0, 0], t[0, 4], t[0, 8], t[0, 33], t[0, 131] = 1, -1, 2, 3, -8
    p = w4_ref.pack(t)
    assert p.shape == (1, 128)
    assert p[0, 0] == 0xF1 and p[0, 16] == 0x02 and p[0, 5] == 0x03 and p[0, 64 + 3] == 0x08
    assert np.count_nonzero(p) == 4
    assert np.array_equal(w4_ref.unpack(p, 160), t)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("with_zeros", [False, True])
def test_w4_error_and_forward(group, with_zeros):
    rng = np.random.default_rng(7)
    w = (rng.normal(0, 0.02, (9, 384)) + (0.01 if with_zeros else 0)).astype(np.float32)
    t, bits, z = w4_ref.quantize(w, group, with_zeros)
    assert np.array_equal(w4_ref.unpack(w4_ref.pack(t), 384), t)
    v = w4_ref.values(t, bits, z)
    s = np.repeat(w4_ref._widen(bits).astype(np.float64), group, axis=1)
    # half a step, and what the scale's rounding (2^-8) clips off 15 steps
    # (with zero points the rounded z moves the range by up to half a step more)
    assert np.all(np.abs(v - w) <= s * (0.5 + 15 / 256 + (0.5 if with_zeros else 0)))
    q = rng.integers(-127, 128, (4, 384)).astype(np.int8)
    a = np.array([0.0, 1.0, 2.0, 1e-7], np.float32)
    y, size = w4_ref.forward(t, bits, z, q, a)
    m = np.maximum(a, np.float32(1e-5)).astype(np.float64)[:, None] / 127
    assert np.allclose(y, (q.astype(np.float64) @ v.T) * m, rtol=1e-12, atol=1e-15)
    assert np.all(size >= np.abs(y) * (1 - 1e-12))
