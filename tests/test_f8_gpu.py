"""The 8-bit floating point format and product (needs an MI355X): codes and
scales bit for bit with the oracle; products against binary64.

Tolerance of a binary32 output: the products of two codes
are exact in binary32; the sum over a block of 128 is formed in the matrix unit,
where each of 128 additions may lose up to a unit in the last place (2^-23) of a
sum no larger than the sum of magnitudes A; then one rounding of the scales'
product, one per multiply-add over the blocks and up to 16 where waves or parts
of K meet, 2^-24 each.  So |y - y64| <= A (128 * 2^-23 + (blocks + 18) * 2^-24).

A bfloat16 output: the e4m3 matrix instructions may cut each of the seven
smaller products of eight at 2^-13 of the largest, 7 * 2^-13 of A at most, and the
result is rounded once (2^-8 of it)."""

import numpy as np
import pytest
import torch

from oracle import f8_ref as ref
from tests.f8_cases import SHAPES

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bl(built_lib):
    import bitlinear_w1_a8_amd as bl
    return bl


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _tolerance(k):
    return 128 * 2.0 ** -23 + ((k + 127) // 128 + 18) * 2.0 ** -24


def _check_bf16(y, want, size, k):
    assert y.dtype == torch.bfloat16
    assert np.all(np.abs(y.float().cpu().numpy() - want)
                  <= size * (7 * 2.0 ** -13 + _tolerance(k)) * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8)


# ------------------------------------------------------------ quantisation

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,k", [(1, 16), (1, 128), (3, 144), (5, 2576), (17, 6912), (2, 131072), (1000, 48)])
def test_quant_act(bl, t, k, dtype):
    x = torch.randn(t, k, generator=torch.Generator().manual_seed(k))
    x[:, ::61] *= 50
    x = x.to(dtype)
    q, s = bl.quant_act_f8(x.cuda())
    host = x.view(torch.uint16).numpy() if dtype == torch.bfloat16 else x.numpy()
    qr, sr = ref.quant_act_f8(host)
    assert np.array_equal(_bytes(q), qr) and np.array_equal(s.cpu().numpy(), sr)


def test_quant_act_special(bl):
    rows = np.zeros((8, 272), np.float32)
    rows[1] = -0.0
    rows[2, ::3] = 1e38
    rows[3, 1], rows[3, 200] = 2.0 ** -101, 1e-45
    rows[4] = np.linspace(-448, 448, 272)             # many ties after the scale of 1
    rows[5, :126] = (ref.e4m3_values()[:126] + ref.e4m3_values()[1:127]) / 2
    rows[5, 127] = 448                                # scale 1: every halfway case
    rows[6] = 3.4e38
    rows[7, 271] = -2.0 ** -149
    q, s = bl.quant_act_f8(torch.from_numpy(rows).cuda())
    qr, sr = ref.quant_act_f8(rows)
    assert np.array_equal(_bytes(q), qr) and np.array_equal(s.cpu().numpy(), sr)


@pytest.mark.parametrize("n,k", [(1, 16), (127, 112), (128, 128), (129, 144), (300, 2512), (5, 131072), (2000, 64)])
def test_pack_and_unpack(bl, n, k):
    w = 0.02 * torch.randn(n, k, generator=torch.Generator().manual_seed(n + k))
    w[: n // 2, : k // 4] = 0
    w[-1, -1] = 2.0 ** -120
    q, s = bl.pack_weights_f8(w.cuda())
    qr, sr = ref.pack_weights_f8(w.numpy())
    assert np.array_equal(_bytes(q), qr) and np.array_equal(s.cpu().numpy(), sr)
    v = bl.unpack_weights_f8(q, s).cpu().numpy()
    assert np.array_equal(v, ref.weights(qr, sr).astype(np.float32))


# ------------------------------------------------------------ products

def _operands(t, n, k, seed=0):
    rng = np.random.default_rng(7 * t + 3 * n + k + seed)
    # all codes that are numbers, subnormals and both zeros among them
    live = np.array([b for b in range(256) if b & 127 != 127], np.uint8)
    w, x = live[rng.integers(0, 254, (n, k))], live[rng.integers(0, 254, (t, k))]
    ws = rng.uniform(0.5, 2, ((n + 127) // 128, (k + 127) // 128)).astype(np.float32)
    xs = rng.uniform(0.5, 2, ((k + 127) // 128, t)).astype(np.float32)
    return w, ws, x, xs


def _cuda(w, ws, x, xs):
    return (torch.from_numpy(w).cuda().view(F8), torch.from_numpy(ws).cuda(),
            torch.from_numpy(x).cuda().view(F8), torch.from_numpy(xs).cuda())


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_product(bl, t, n, k):
    host = _operands(t, n, k)
    w, ws, x, xs = _cuda(*host)
    y = bl.forward_f8(w, ws, x, xs)
    assert y.dtype == torch.float32 and y.shape == (t, n)
    want, size = ref.forward_f8(*host)
    assert np.all(np.abs(y.cpu().numpy() - want) <= size * _tolerance(k))
    b = bl.forward_f8(w, ws, x, xs, dtype=torch.bfloat16)
    _check_bf16(b, want, size, k)
    # the same bits every time
    assert torch.equal(bl.forward_f8(w, ws, x, xs), y)
    assert torch.equal(bl.forward_f8(w, ws, x, xs, dtype=torch.bfloat16), b)


@pytest.mark.parametrize("t", [1, 16, 40, 200])
def test_ordinary_magnitudes(bl, t):
    """Quantised Gaussian data: against the product of what the codes stand for,
    and within the quantisation's error of the product of the data."""
    g = torch.Generator().manual_seed(t)
    x, w = torch.randn(t, 1040, generator=g), 0.02 * torch.randn(260, 1040, generator=g)
    codes, ws = bl.pack_weights_f8(w.cuda())
    xq, xs = bl.quant_act_f8(x.cuda())
    y = bl.forward_f8(codes, ws, xq, xs)
    want, size = ref.forward_f8(_bytes(codes), ws.cpu().numpy(), _bytes(xq), xs.cpu().numpy())
    assert np.all(np.abs(y.cpu().numpy() - want) <= size * _tolerance(1040))
    assert torch.equal(bl.linear_f8(x.cuda(), codes, ws), y)
    plain = x.double() @ w.double().t()
    # each factor is off by at most 2^-4 of itself (or a subnormal's step, which this covers):
    # 1/8 of the sum of magnitudes in the worst case; independent errors make it far smaller
    assert float((y.cpu().double() - plain).norm() / plain.norm()) < 0.125


@pytest.mark.parametrize("t", [1, 20, 64, 100])
def test_scales_of_zero_blocks(bl, t):
    """Blocks of zeros (the floor's scale) add nothing, and the scales of one
    token, group or block reach no other."""
    w, ws, x, xs = _operands(t, 300, 640)
    w[128:256] = 0
    x[:, 128:256] = 0
    xs[1], ws[1] = 2.0 ** -100 / 448, 2.0 ** -100 / 448
    xs[2, 0], ws[0, 3] = 1e20, 1e-20
    y = bl.forward_f8(*_cuda(w, ws, x, xs)).cpu().numpy()
    want, size = ref.forward_f8(w, ws, x, xs)
    assert np.all(y[:, 128:256] == 0)
    assert np.all(np.abs(y - want) <= size * _tolerance(640))


@pytest.mark.parametrize("t,n,k", [(1, 100, 144), (20, 37, 272), (100, 130, 144), (300, 257, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_neighbours_untouched(bl, t, n, k, dtype):
    host = _operands(t, n, k)
    w, ws, x, xs = _cuda(*host)
    buf = torch.full((t + 2, n), 7.0, dtype=dtype, device="cuda")
    bl.forward_f8(w, ws, x, xs, out=buf[1:-1])
    assert torch.all(buf[0] == 7) and torch.all(buf[-1] == 7)
    assert torch.equal(buf[1:-1], bl.forward_f8(w, ws, x, xs, dtype=dtype))


@pytest.mark.parametrize("t,n,k", [(1, 100, 144), (20, 40, 272), (130, 6002, 128), (300, 16504, 128), (1100, 8200, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_output_at_any_element(bl, t, n, k, dtype):
    """y is aligned to its element only, and nothing around it is written."""
    w, ws, x, xs = _cuda(*_operands(t, n, k))
    buf = torch.full((t * n + 16,), 7.0, dtype=dtype, device="cuda")
    for at in (1, 3):
        y = buf[at:at + t * n].view(t, n)
        bl.forward_f8(w, ws, x, xs, out=y)
        assert torch.equal(y, bl.forward_f8(w, ws, x, xs, dtype=dtype))
        assert torch.all(buf[:at] == 7) and torch.all(buf[at + t * n:] == 7)
        buf[:] = 7


def test_infinite_token_scale_stays_in_its_row(bl):
    w, ws, x, xs = _operands(70, 130, 256)
    xs[:, 3] = np.inf
    y = bl.forward_f8(*_cuda(w, ws, x, xs)).cpu().numpy()
    rest = np.arange(70) != 3
    assert np.all(np.isfinite(y[rest])) and not np.any(np.isfinite(y[3]))


def test_graph_and_streams(bl):
    for t in (2, 300):
        w, ws, x, xs = _cuda(*_operands(t, 257, 528))
        want = bl.forward_f8(w, ws, x, xs)
        raw = torch.randn(t, 528, device="cuda")
        linear = bl.linear_f8(raw, w, ws)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append((bl.forward_f8(w, ws, x, xs), bl.linear_f8(raw, w, ws)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, want) and torch.equal(b, linear) for a, b in got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, z = bl.forward_f8(w, ws, x, xs), bl.linear_f8(raw, w, ws)
        for i in range(3):
            y.zero_(), z.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(z, linear)
            assert torch.equal(bl.forward_f8(w, ws, x, xs), want)


# ------------------------------------------------------------ large offsets

@pytest.mark.parametrize("t", [1, 70])
def test_matrix_past_32_bits(bl, t):
    """A matrix of more than 2^32 bytes: rows of one code each, so that y is the
    row's code times the token's sum."""
    n, k = (1 << 22) + 130, 1040
    w = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    w[:] = 0x38                                       # 1
    w[-130:] = 0xc0                                   # -2
    ws = torch.ones((n + 127) // 128, 9, device="cuda")
    x = torch.zeros(t, k, device="cuda")
    x[:, ::5] = 3
    xq, xs = x.to(F8), torch.ones(9, t, device="cuda")
    y = bl.forward_f8(w.view(F8), ws, xq, xs, dtype=torch.bfloat16)
    assert torch.all(y[:, :-130] == 624) and torch.all(y[:, -130:] == -1248)


@pytest.mark.parametrize("t,n", [(48, 1 << 26), (1 << 20, 4099)])
def test_outputs_past_32_bits(bl, t, n):
    k = 16
    w = torch.full((n, k), 0x38, dtype=torch.uint8, device="cuda")
    w[-3:] = 0x40
    ws = torch.ones((n + 127) // 128, 1, device="cuda")
    xq = torch.ones(t, k, device="cuda").to(F8)
    xs = torch.ones(1, t, device="cuda")
    xs[0, -2:] = 0.5
    y = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    bl.forward_f8(w.view(F8), ws, xq, xs, out=y)
    for rows, scale in ((slice(0, t - 2), 1.0), (slice(t - 2, t), 0.5)):
        part = y[rows]
        assert torch.all(part[:, :-3] == 16 * scale) and torch.all(part[:, -3:] == 32 * scale)


def test_pack_past_32_bits(bl):
    n, k = (1 << 20) + 128, 4112
    w = torch.zeros(n, k, device="cuda")
    w[-1, -1] = 2.0
    w[-128, 0] = 448.0
    q, s = bl.pack_weights_f8(w)
    assert int(q.view(torch.uint8)[-1, -1]) == 0x7e and float(s[-1, -1]) == np.float32(2) / np.float32(448)
    assert int(q.view(torch.uint8)[-128, 0]) == 0x7e and float(s[-1, 0]) == 1.0
    del w
    v = bl.unpack_weights_f8(q, s)
    assert float(v[-128, 0]) == 448.0 and float(v[-1, -1]) == 2.0 and float(v[-1, 0]) == 0.0
