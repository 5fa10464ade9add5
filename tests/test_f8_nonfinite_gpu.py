"""NaN and infinities in the norms, the e4m3 codes and their products (needs an
MI355X): they stay in their token, matrix row or group, and there they are seen."""

import pytest
import torch

pytestmark = pytest.mark.gpu

F8, BF16 = torch.float8_e4m3fn, torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def bl(built_lib):
    import bitlinear_w1_a8_amd as bl
    return bl


def _bytes(q):
    return q.view(torch.uint8)


def _nan(q):
    return (_bytes(q) & 127) == 127


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 130, 399])
def test_quant_act(bl, dtype, value, at):
    x = torch.randn(6, 400, generator=torch.Generator().manual_seed(at)).to(dtype).cuda()
    q0, s0 = bl.quant_act_f8(x)
    x[3, at] = value
    q, s = bl.quant_act_f8(x)
    assert bool(_nan(q)[3, at])
    group = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    group[3, at // 128] = True
    keep = ~group.repeat_interleave(128, 1)[:, :400]
    assert torch.equal(_bytes(q)[keep], _bytes(q0)[keep]) and torch.equal(s.t()[~group], s0.t()[~group])


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [(0, 0), (140, 200), (299, 271)])
def test_pack(bl, value, at):
    w = torch.randn(300, 272, generator=torch.Generator().manual_seed(at[0])).cuda()
    q0, s0 = bl.pack_weights_f8(w)
    w[at] = value
    q, s = bl.pack_weights_f8(w)
    assert bool(_nan(q)[at])
    block = torch.zeros(3, 3, dtype=torch.bool, device="cuda")
    block[at[0] // 128, at[1] // 128] = True
    keep = ~block.repeat_interleave(128, 0).repeat_interleave(128, 1)[:300, :272]
    assert torch.equal(_bytes(q)[keep], _bytes(q0)[keep]) and torch.equal(s[~block], s0[~block])
    assert bool(torch.isnan(bl.unpack_weights_f8(q, s)[at]))


@pytest.mark.parametrize("k", [272, 2560, 40000])
@pytest.mark.parametrize("xd,rd", [(torch.float32, BF16), (BF16, torch.float32), (torch.float32, None)])
@pytest.mark.parametrize("value", [NAN, INF, -INF, 3e38, "sum"])
def test_norm(bl, k, xd, rd, value):
    """A row whose mean square is no binary32 number (3e38 has a square of 9e76) has
    no norm: every e4m3 code of it is NaN.  The other rows are as without it, in either form."""
    g = torch.Generator().manual_seed(k)
    x, r = torch.randn(5, k, generator=g).to(xd).cuda(), None if rd is None else torch.randn(5, k, generator=g).to(rd).cuda()
    gain = (1 + 0.1 * torch.randn(k, generator=g)).cuda()
    want8, want = bl.add_subln_quant_act_f8(x, r, gain), bl.add_subln_quant_act(x, r, gain)
    if value == "sum" and r is not None:
        x[2, k - 3], r[2, k - 3] = 3e38, 3e38            # finite both
    else:
        x[2, k - 3] = 3e38 if value == "sum" else value
    got8, got = bl.add_subln_quant_act_f8(x, r, gain), bl.add_subln_quant_act(x, r, gain)
    rest = [0, 1, 3, 4]
    assert torch.all(_nan(got8[0])[2])
    assert torch.equal(_bytes(got8[0])[rest], _bytes(want8[0])[rest]) and torch.equal(got8[1][:, rest], want8[1][:, rest])
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got[:3], want[:3]))
    if r is not None:
        plain = (x.float() + r.float()).to(rd)
        for total in (got8[2], got[3]):
            assert torch.equal(total.isnan(), plain.isnan())
            assert torch.equal(total.nan_to_num(nan=5.0), plain.nan_to_num(nan=5.0))


@pytest.mark.parametrize("value", [NAN, INF])
def test_norm_gain(bl, value):
    """A feature whose gain is not finite: its own group."""
    x, gain = torch.randn(4, 400, device="cuda"), torch.ones(400, device="cuda")
    want = bl.add_subln_quant_act_f8(x, None, gain)
    gain[140] = value
    got = bl.add_subln_quant_act_f8(x, None, gain)
    assert torch.all(_nan(got[0])[:, 140])
    keep = [i for i in range(400) if i // 128 != 1]
    assert torch.equal(_bytes(got[0])[:, keep], _bytes(want[0])[:, keep]) and torch.equal(got[1][[0, 2, 3]], want[1][[0, 2, 3]])


@pytest.mark.parametrize("t,n,k", [
    (5, 300, 272), (20, 100, 400), (28, 4100, 272), (40, 1100, 384), (400, 1000, 128), (300, 1201, 400), (130, 6001, 272),
    (200, 9001, 272), (257, 17000, 528), (1030, 8193, 144), (1025, 8448, 256)])
@pytest.mark.parametrize("kw", [dict(), dict(dtype=BF16), dict(dtype=BF16, sums="cut")])
def test_product(bl, t, n, k, kw):
    g = torch.Generator(device="cuda").manual_seed(t)
    w = torch.randint(-9, 10, (n, k), generator=g, device="cuda").float().to(F8)
    x = torch.randint(-9, 10, (t, k), generator=g, device="cuda").float().to(F8)
    ws, xs = torch.ones((n + 127) // 128, (k + 127) // 128, device="cuda"), torch.ones((k + 127) // 128, t, device="cuda")
    want = bl.forward_f8(w, ws, x, xs, **kw)
    assert torch.all(torch.isfinite(want))
    rows, tokens = [0, n // 2, n - 1], [t // 3, t - 1]
    for i, row in enumerate(rows):
        _bytes(w)[row, (0, k // 2, k - 1)[i]] = (0x7f, 0xff, 0x7f)[i]
    for i, token in enumerate(tokens):
        _bytes(x)[token, (k - 1, 5)[i]] = (0xff, 0x7f)[i]
    y = bl.forward_f8(w, ws, x, xs, **kw)
    bad = torch.zeros(t, n, dtype=torch.bool, device="cuda")
    bad[tokens], bad[:, rows] = True, True
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("t", [1, 3, 6, 16, 20])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_layer_keeps_tokens_apart(bl, t, dtype):
    from tests.test_layer_gpu import Layer, _tokens
    layer = Layer(bl, 64, 608, 272, 50)
    x, logits = _tokens(t + 2, 272, 64, x=dtype)
    want = layer(x, logits, 4)
    x[1, 7], x[0, 0] = NAN, INF
    got = layer(x, logits, 4)
    assert torch.equal(got[2:], want[2:])
