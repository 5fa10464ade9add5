"""Pins of the e4m3 oracle (CPU)."""

import numpy as np
import pytest
import torch

from oracle import f8_ref as ref


def test_code_values():
    v = ref.e4m3_values()
    assert v[0x7e] == 448 and v[0xfe] == -448 and v[0x38] == 1 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff])
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)


def test_rounding_ties_and_signs():
    # halfway cases go to the even code; 17 lies between 16 (0x58, even) and 18 (0x59)
    for value, code in ((17, 0x58), (19, 0x5a), (-17, 0xd8), (1.0625, 0x38), (1.1875, 0x3a),
                        (2.0 ** -10, 0), (3 * 2.0 ** -10, 2), (2.0 ** -10 * 1.01, 1), (448, 0x7e), (-0.0, 0x80)):
        assert ref.e4m3(np.array([value]))[0] == code, value


def test_rounding_against_torch():
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(0, 0.02, 20000),
                        (ref.e4m3_values()[:126] + ref.e4m3_values()[1:127]) / 2]).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3(x), t)


def test_groups():
    x = np.zeros((2, 144), np.float32)
    x[0, 5], x[0, 6], x[1, 130] = -896.0, 2.0, 2.0 ** -110
    q, s = ref.quant_act_f8(x)
    assert s.shape == (2, 2) and s[0, 0] == 2.0
    assert q[0, 5] == 0xfe and q[0, 6] == 0x38
    assert s[0, 1] == s[1, 1] == np.float32(2.0 ** -100) / np.float32(448)     # the floor
    assert ref.e4m3_values()[q[1, 130]] == 448 * 2.0 ** -10 // 2.0 ** -9 * 2.0 ** -9    # 224 steps of 2^-9
    w = np.zeros((130, 16), np.float32)
    w[0, 0], w[129, 3] = 448, 1
    q, s = ref.pack_weights_f8(w)
    assert s.shape == (2, 1) and s[0, 0] == 1 and s[1, 0] == np.float32(1) / np.float32(448)
    assert q[0, 0] == q[129, 3] == 0x7e


def test_quantisation_error():
    """A value is off by half a step: 2^-4 of itself, or half the spacing of the
    subnormals (2^-10 of a scale), with two binary32 roundings on the way."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((20, 400)).astype(np.float32)
    q, s = ref.quant_act_f8(x)
    scale = np.repeat(s.T.astype(np.float64), 128, 1)[:, :400]
    off = np.abs(ref.tokens(q, s) - x)
    assert np.all(off <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -18) + np.abs(x) * 2.0 ** -22)


def test_product_small():
    w = np.array([[448, 224], [-448, 0]], np.float32).repeat(64, 1)
    codes, ws = ref.pack_weights_f8(w)
    xq, xs = ref.quant_act_f8(np.full((1, 128), 0.5, np.float32))
    y, size = ref.forward_f8(codes, ws, xq, xs)
    assert y[0] == pytest.approx([64 * 336.0, -64 * 224.0], rel=1e-7)
    assert size[0] == pytest.approx([64 * 336.0, 64 * 224.0], rel=1e-7)


def test_sum_is_rounded_to_the_residual():
    x = np.array([[1.0, 2.0 ** -30, 1.0]], np.float32)
    r32 = np.array([[2.0 ** -24, 1.0, 2.0 ** -9]], np.float32)
    assert np.array_equal(ref.add(x, r32), np.array([[1.0, 1.0, 1 + 2.0 ** -9]], np.float32))
    bits = np.array([[0x3f80, 0x3f80, 0x3b80]], np.uint16)       # 1, 1, 2^-8
    assert np.array_equal(ref.add(x, bits), np.array([[0x4000, 0x3f80, 0x3f80]], np.uint16))
