"""The residual's addition with the sub-layer norm and 8-bit codes (needs an
MI355X).  Sums, codes, scales and row sums are compared bit for bit: with the
oracle, and with the addition followed by subln_quant_act."""

import numpy as np
import pytest
import torch

from oracle import f8_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def bl(built_lib):
    import bitlinear_w1_a8_amd as bl
    return bl


def _host(t):
    """As the oracle takes it: float32, or bfloat16 bit patterns."""
    return t.cpu().view(torch.uint16).numpy() if t.dtype == BF16 else t.cpu().numpy()


def _inputs(t, k, xd, rd, seed=0):
    g = torch.Generator().manual_seed(1000 * t + k + seed)
    x = torch.randn(t, k, generator=g)
    r = 3 * torch.randn(t, k, generator=g)
    r[:, ::97] *= 30
    gain = 1 + 0.3 * torch.randn(k, generator=g)
    return (x.to(xd).cuda(), None if rd is None else r.to(rd).cuda(), gain.cuda())


def _check(bl, x, r, gain, oracle_rows=None):
    xq, scale, rowsum, total = bl.add_subln_quant_act(x, r, gain)
    fq, fs, ftotal = bl.add_subln_quant_act_f8(x, r, gain)
    if r is None:
        assert total is None and ftotal is None
        plain = x
    else:
        plain = (x.float() + r.float()).to(r.dtype)
        assert torch.equal(total.view(torch.uint8), plain.view(torch.uint8))
        assert torch.equal(ftotal.view(torch.uint8), plain.view(torch.uint8))
    q2, s2, sum2 = bl.subln_quant_act(plain, gain)
    assert torch.equal(xq, q2) and torch.equal(scale, s2) and torch.equal(rowsum, sum2)
    rows = slice(None) if oracle_rows is None else oracle_rows
    x, r = x[rows], None if r is None else r[rows]
    _, q, s, n = ref.add_subln_quant_act(_host(x), None if r is None else _host(r), gain.cpu().numpy())
    assert np.array_equal(xq[rows].cpu().numpy(), q)
    assert np.array_equal(scale[rows].cpu().numpy(), s) and np.array_equal(rowsum[rows].cpu().numpy(), n)
    _, q, s = ref.add_subln_quant_act_f8(_host(x), None if r is None else _host(r), gain.cpu().numpy())
    assert np.array_equal(fq[rows].view(torch.uint8).cpu().numpy(), q)
    assert np.array_equal(fs[:, rows].cpu().numpy(), s)


@pytest.mark.parametrize("xd", [F32, BF16])
@pytest.mark.parametrize("rd", [None, F32, BF16])
@pytest.mark.parametrize("t,k", [(1, 16), (1, 2560), (3, 112), (5, 144), (2, 1024), (7, 2576), (33, 6912), (2, 28672)])
def test_against_oracle(bl, t, k, xd, rd):
    _check(bl, *_inputs(t, k, xd, rd))


@pytest.mark.parametrize("k", [16384 + 16, 32768 + 16, 65536, 131072])
@pytest.mark.parametrize("xd,rd", [(F32, BF16), (BF16, F32), (F32, None)])
def test_long_rows(bl, k, xd, rd):
    _check(bl, *_inputs(2, k, xd, rd))


@pytest.mark.parametrize("xd,rd", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_many_rows(bl, xd, rd):
    _check(bl, *_inputs(3000, 640, xd, rd), oracle_rows=slice(0, 3000, 271))


def _special_rows():
    """Rows whose mean square lies on or next to a border between two binary32
    numbers, and rows of unusual spread."""
    k = 16
    rows = []

    def row(*values):
        v = np.zeros(k, np.float32)
        v[:len(values)] = values
        rows.append(v)
    row()                                            # zeros
    row(1, 2.0 ** -12)                               # (1 + 2^-24) / 16: a tie, to even
    row(1, 2.0 ** -12, 2.0 ** -60)                   # just past the tie: up
    row(1, 2.0 ** -12, 2.0 ** -40, 2.0 ** -70)
    row(1, np.float32(2.0 ** -12) * np.float32(1 - 2.0 ** -24))   # just before it
    row(np.float32(np.sqrt(1 + 2.0 ** -23)), 2.0 ** -12)
    row(1 + 2.0 ** -23, 2.0 ** -12, 2.0 ** -35)
    row(2.0 ** 60, 2.0 ** 48, 2.0 ** -60)            # the same tie, far apart
    row(2.0 ** -70, 2.0 ** -74)
    row(1e-45, 3e-42, 1e-39)                         # subnormals
    row(*[(-1.0) ** i * 2.0 ** -i for i in range(16)])
    row(*[1e18 * (1 + i) for i in range(16)])
    return np.stack(rows)


def test_borders(bl):
    x = torch.from_numpy(_special_rows()).cuda()
    gain = torch.ones(16, device="cuda")
    _check(bl, x, None, gain)
    _check(bl, x, torch.zeros_like(x), gain)
    _check(bl, torch.zeros_like(x), x, gain)
    # the same rows with zeros between them, in a longer row whose length is a power of two
    wide = torch.zeros(x.shape[0], 8192, device="cuda")
    wide[:, ::512] = x
    _check(bl, wide, None, torch.ones(8192, device="cuda"))


@pytest.mark.parametrize("value", [0.0, 1.0, -3.0, 1e-30, 2.0 ** -101])
def test_constant_rows(bl, value):
    x = torch.full((3, 272), value, device="cuda")
    _check(bl, x, torch.zeros_like(x), torch.full((272,), 0.5, device="cuda"))


def test_zero_gain_groups(bl):
    x, r, gain = _inputs(4, 400, F32, BF16)
    gain[128:256] = 0                                # a group of zeros: the floor's scale
    _check(bl, x, r, gain)


@pytest.mark.parametrize("xd,rd", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("k", [272, 2560, 40000])
def test_in_place(bl, xd, rd, k):
    x, r, gain = _inputs(5, k, xd, rd)
    want = bl.add_subln_quant_act(x, r, gain)
    into = r.clone()
    got = bl.add_subln_quant_act(x, into, gain, out=into)
    assert got[3] is into
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    want = bl.add_subln_quant_act_f8(x, r, gain)
    into = r.clone()
    got = bl.add_subln_quant_act_f8(x, into, gain, out=into)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    if xd is rd:                                     # the sum may also take x's place
        into = x.clone()
        got = bl.add_subln_quant_act_f8(into, r, gain, out=into)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))


def test_without_rowsum_and_other_epsilon(bl):
    x, r, gain = _inputs(6, 1040, F32, F32)
    xq, scale, rowsum, total = bl.add_subln_quant_act(x, r, gain, eps_n=0.5, with_rowsum=False)
    assert rowsum is None
    q2, s2, _ = bl.subln_quant_act(total, gain, eps_n=0.5)
    assert torch.equal(xq, q2) and torch.equal(scale, s2)


def test_neighbours_untouched(bl):
    """Outputs end where they should: rows before and after in the same buffer stay."""
    x, r, gain = _inputs(3, 144, F32, BF16)
    buf = torch.full((5, 144), 7.0, dtype=BF16, device="cuda")
    bl.add_subln_quant_act_f8(x, r, gain, out=buf[1:4])
    assert torch.all(buf[0] == 7) and torch.all(buf[4] == 7)
    assert torch.equal(buf[1:4], (x + r.float()).bfloat16())


def test_graph_and_streams(bl):
    x, r, gain = _inputs(40, 2560, F32, BF16)
    out = torch.empty_like(r)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            bl.add_subln_quant_act(x, r, gain, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xq, scale, rowsum, total = bl.add_subln_quant_act(x, r, gain, out=out)
        fq, fs, _ = bl.add_subln_quant_act_f8(x, r, gain)
    for i in range(4):
        x.copy_(torch.randn(40, 2560, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        a, b = bl.add_subln_quant_act(x, r, gain), bl.add_subln_quant_act_f8(x, r, gain)
        torch.cuda.synchronize()
        for got, want in zip((xq, scale, rowsum, total, fq.view(torch.uint8), fs),
                             (*a, b[0].view(torch.uint8), b[1])):
            assert torch.equal(got, want)


def test_more_rows_than_one_launch(bl):
    """2^21 + 3 rows: the second launch's rows, and its scales' places."""
    t, k = (1 << 21) + 3, 16
    x = torch.randn(t, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    gain = torch.ones(k, device="cuda")
    xq, scale, rowsum, total = bl.add_subln_quant_act(x, x, gain)
    fq, fs, _ = bl.add_subln_quant_act_f8(x, x, gain)
    tail = slice(t - 300, t)
    xs = x[tail].contiguous()
    a, b = bl.add_subln_quant_act(xs, xs, gain), bl.add_subln_quant_act_f8(xs, xs, gain)
    for got, want in zip((xq, scale, rowsum, total), a):
        assert torch.equal(got[tail], want)
    assert torch.equal(fq.view(torch.uint8)[tail], b[0].view(torch.uint8)) and torch.equal(fs[:, tail], b[1])


def test_feeds_the_products(bl):
    """What the norm gives goes on: to the ternary, the 4-bit and the e4m3 product."""
    x, r, gain = _inputs(9, 512, F32, BF16)
    w = 0.02 * torch.randn(200, 512, generator=torch.Generator().manual_seed(5)).cuda()
    xq, scale, rowsum, total = bl.add_subln_quant_act(x, r, gain)
    packed, gamma = bl.pack_weights(w)
    q2, s2, sum2 = bl.subln_quant_act(total, gain)
    assert torch.equal(bl.forward(packed, gamma, xq, scale, 200, rowsum=rowsum),
                       bl.forward(packed, gamma, q2, s2, 200, rowsum=sum2))
    p4, sc4, _ = bl.pack_weights_w4(w)
    assert torch.equal(bl.forward_w4(p4, sc4, xq, scale), bl.forward_w4(p4, sc4, q2, s2))
    fq, fs, _ = bl.add_subln_quant_act_f8(x, r, gain)
    codes, ws = bl.pack_weights_f8(w)
    y, size = ref.forward_f8(codes.view(torch.uint8).cpu().numpy(), ws.cpu().numpy(),
                             fq.view(torch.uint8).cpu().numpy(), fs.cpu().numpy())
    got = bl.forward_f8(codes, ws, fq, fs).cpu().numpy()
    assert np.all(np.abs(got - y) <= size * 2.0 ** -15)
