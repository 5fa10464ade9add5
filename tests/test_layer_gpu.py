"""The whole routed layer (needs an MI355X), bit for bit with the router, the
gated and the linear calls one after the other, which have oracle tests of
their own; and a few cases straight against the oracle."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

F32, BF16, I8 = torch.float32, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def bl(built_lib):
    import bitlinear_w1_a8_amd as bl
    return bl


class Layer:
    def __init__(self, bl, e, f, k, n, seed=0):
        self.bl, self.e = bl, e
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * e + f + k + n)

        def ternary(*shape):
            c = torch.randint(0, 3, (4, *shape[:-1], shape[-1] // 4), generator=g, device="cuda", dtype=torch.uint8)
            return c[0] | (c[1] << 2) | (c[2] << 4) | (c[3] << 6)
        self.gu, self.dn = ternary(e, 2 * f, k), ternary(e, n, f)
        self.gg, self.ug, self.dg = (0.01 + 0.02 * torch.rand(e, generator=g, device="cuda") for _ in range(3))

    def __call__(self, x, logits, k, **kw):
        return self.bl.experts_ffn(x, logits, k, self.gu, self.gg, self.ug, self.dn, self.dg, **kw)

    def calls(self, x, logits, k, share="chosen"):
        r = self.bl.route_experts(logits, k, share=share)
        h = self.bl.gated_relu2_experts(x, self.gu, self.gg, self.ug, r)[0]
        return self.bl.linear_experts(h, self.dn, self.dg, r)


def _tokens(t, k, e, logits=F32, x=F32, seed=0):
    g = torch.Generator().manual_seed(100 * t + k + e + seed)
    return (torch.randn(t, k, generator=g).to(x).cuda(),
            (2 * torch.randn(t, e, generator=g)).to(logits).cuda())


def _check(bl, layer, x, logits, k, share="chosen"):
    want = layer.calls(x, logits, k, share)
    got = layer(x, logits, k, share=share)
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    xq, absmax, _ = bl.quant_act(x)
    got = layer(xq, logits, k, absmax=absmax, share=share)
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))


SHAPES = [  # T, E, k, F, K, N
    (1, 1, 1, 16, 16, 1), (1, 8, 2, 64, 64, 64), (1, 64, 8, 1024, 2560, 2560), (2, 4, 4, 48, 112, 33),
    (3, 64, 6, 1008, 2576, 100), (4, 128, 8, 256, 512, 130), (5, 7, 3, 80, 144, 257), (8, 16, 16, 128, 256, 64),
    (9, 65, 5, 272, 400, 48), (15, 256, 16, 64, 128, 80), (16, 64, 8, 512, 1024, 512), (16, 2, 2, 32, 48, 17),
    (16, 129, 1, 336, 1040, 20), (6, 200, 9, 2064, 320, 40), (2, 8, 4, 4096, 7168, 72), (16, 5, 5, 96, 8192, 24),
    (1, 3, 2, 28672, 64, 31), (13, 33, 7, 112, 1536, 96)]


@pytest.mark.parametrize("share", ["chosen", "all"])
@pytest.mark.parametrize("t,e,k,f,kk,n", SHAPES)
def test_equals_the_three_calls(bl, t, e, k, f, kk, n, share):
    layer = Layer(bl, e, f, kk, n)
    for logits, x in ((F32, BF16), (BF16, F32)):
        _check(bl, layer, *_tokens(t, kk, e, logits, x), k, share)


@pytest.mark.parametrize("t,e,k,f,kk,n", [
    (17, 64, 8, 128, 256, 64), (64, 16, 4, 64, 144, 48), (130, 8, 2, 256, 512, 96), (2, 300, 4, 64, 128, 64),
    (3, 1024, 32, 16, 64, 16), (5, 40, 17, 32, 64, 32), (16, 4, 2, 64, 16384, 32), (1, 2, 2, 131072, 16, 16)])
def test_past_the_two_launches(bl, t, e, k, f, kk, n):
    layer = Layer(bl, e, f, kk, n)
    for logits, x in ((F32, BF16), (BF16, F32)):
        _check(bl, layer, *_tokens(t, kk, e, logits, x), k)


@pytest.mark.parametrize("t", [1, 4, 11, 16, 20])
def test_masks_and_ties(bl, t):
    e, k = 48, 6
    layer = Layer(bl, e, 96, 272, 50)
    x, logits = _tokens(t, 272, e)
    logits = logits.round()                          # many equal ones
    logits[:, ::5] = float("-inf")
    logits[0, 3:] = float("-inf")                    # a token of three experts
    logits[t // 2] = float("-inf")                   # and one of none
    logits[t - 1, 7] = float("nan")
    logits[t - 1, 8] = float("inf")
    if t > 3:
        logits[2] = 0.0
        logits[2, ::2] = -0.0                        # equal to +0
        logits[3] = -3.4028234663852886e38           # the lowest value is a logit like any other
    for share in ("chosen", "all"):
        want = layer.calls(x, logits, k, share)
        got = layer(x, logits, k, share=share)
        assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    none = ~(logits > float("-inf")).any(1)          # rows without a usable logit
    assert (t == 4 or t > 1 and none.any()) and torch.all(got[none] == 0) or t == 1


@pytest.mark.parametrize("t,e,k", [(1, 64, 8), (2, 64, 16), (3, 64, 6), (4, 64, 8), (4, 100, 12), (1, 128, 1),
                                   (4, 129, 16), (3, 192, 5), (4, 256, 16), (1, 255, 16), (2, 256, 3)])
def test_few_tokens_of_many_experts(bl, t, e, k):
    """Ties across a wave's 64 logits, experts that several tokens take at different
    ranks, tokens with fewer usable logits than k or none."""
    layer = Layer(bl, e, 1040, 272, 50)
    x, logits = _tokens(t, 272, e)
    same = logits[:1].expand(t, e).contiguous()
    few = torch.full_like(logits, float("-inf"))
    few[0, e - 1] = few[t // 2, e // 2] = float("inf")
    few[t - 1, 3 % e] = -3.4028234663852886e38
    mixed = logits.clone()
    mixed[t - 1] = float("nan")
    shifted = torch.stack([logits[0].roll(i) + 0.01 * i for i in range(t)])
    for l in (logits.round(), torch.zeros_like(logits), same, few, mixed, shifted, -logits.abs().round()):
        _check(bl, layer, x, l, k)
        _check(bl, layer, x, l.bfloat16(), k, "all")


def test_everything_masked_and_one_expert_takes_all(bl):
    layer = Layer(bl, 32, 64, 128, 40)
    x, logits = _tokens(16, 128, 32)
    out = torch.full((16, 40), 7.0, device="cuda")
    assert layer(x, torch.full_like(logits, float("-inf")), 4, out=out) is out
    assert torch.all(out == 0)
    logits[:, 9] = 50
    logits[:, 21] = 40
    _check(bl, layer, x, logits, 2)
    _check(bl, layer, x, logits.bfloat16(), 1)


def test_rows_of_zeros(bl):
    layer = Layer(bl, 8, 64, 128, 40)
    x, logits = _tokens(6, 128, 8)
    x[2] = 0
    x[4] = 1e-7
    _check(bl, layer, x, logits, 3)


@pytest.mark.parametrize("t,e,k,f,kk,n", [(1, 8, 3, 48, 144, 37), (5, 16, 4, 80, 272, 40), (16, 12, 2, 128, 64, 21)])
def test_against_the_oracle(bl, t, e, k, f, kk, n):
    """The sums and codes are exact and the binary32 steps counted: the weight is
    off by the exponential's 2 units in the last place, k + 1 additions and a
    division, each output by its scale's three roundings, the product and k
    additions: (k + 12) 2^-23 of the sum of magnitudes covers them."""
    layer = Layer(bl, e, f, kk, n)
    x, logits = _tokens(t, kk, e)
    got = layer(x, logits, k).cpu().numpy()
    l = logits.double().cpu().numpy()

    def matrix(packed, width):
        at = np.arange(width)
        return ((packed[:, at // 16 * 4 + at % 4].astype(np.int64) >> (2 * (at % 16 // 4))) & 3) - 1
    gu, dn = layer.gu.cpu().numpy(), layer.dn.cpu().numpy()
    gg, ug, dg = (v.cpu().numpy() for v in (layer.gg, layer.ug, layer.dg))
    xq, a, _ = oracle.quant_act(x.cpu().numpy())
    for i in range(t):
        ids = np.argsort(-l[i], kind="stable")[:k]
        w = np.exp(l[i][ids] - l[i].max())
        w /= w.sum()
        y, size = np.zeros(n), np.zeros(n)
        for j, ex in enumerate(ids):
            acc = matrix(gu[ex], kk) @ xq[i].astype(np.int64)
            gate, up = (oracle.a3_f32(acc[None, s::2], g[ex], a[i:i + 1])[0] for s, g in ((0, gg), (1, ug)))
            r = np.maximum(gate, np.float32(0))
            h = oracle.bf16_rne((r * r) * up)
            hq, ha, _ = oracle.quant_act(h[None])
            part = (matrix(dn[ex], f) @ hq[0].astype(np.int64)) * float(dg[ex]) * max(float(ha[0]), 1e-5) / 127
            y += w[j] * part
            size += np.abs(w[j] * part)
        assert np.all(np.abs(got[i] - y) <= size * (k + 12) * 2.0 ** -23)


def test_norm_into_layer(bl):
    """As a decoder runs them: the norm's codes into the layer, its output into the next norm."""
    layer = Layer(bl, 32, 256, 512, 512)
    x, logits = _tokens(7, 512, 32)
    residual, gain = x.bfloat16(), torch.ones(512, device="cuda")
    xq, scale, _, total = bl.add_subln_quant_act(x, residual, gain)
    y = layer(xq, logits, 4, absmax=scale)
    plain = (x + residual.float()).bfloat16()
    q2, s2, _ = bl.subln_quant_act(plain, gain)
    assert torch.equal(y, layer(q2, logits, 4, absmax=s2))
    after = (y + plain.float()).bfloat16()
    fq, fs, total2 = bl.add_subln_quant_act_f8(y, total, gain, out=total)
    assert total2 is total and torch.equal(total, after)
    want = bl.add_subln_quant_act_f8(after, None, gain)
    assert torch.equal(fq.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(fs, want[1])


def test_graph_and_streams(bl):
    for t, x_dtype in ((1, BF16), (6, F32), (16, I8)):
        layer = Layer(bl, 40, 128, 272, 64)
        x, logits = _tokens(t, 272, 40)
        absmax = None
        if x_dtype is I8:
            x, absmax, _ = bl.quant_act(x)
        else:
            x = x.to(x_dtype)
        want = layer(x, logits, 4, absmax=absmax)
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got += [layer(x, logits, 4, absmax=absmax) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(x, logits, 4, absmax=absmax)
        for i in range(4):
            logits.copy_(torch.randn(t, 40, generator=torch.Generator().manual_seed(i)))
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, layer(x, logits, 4, absmax=absmax))
            torch.cuda.synchronize()


def test_matrices_past_32_bits(bl):
    """Experts whose packed matrices together pass 2^32 bytes: the last one's."""
    e, f, kk, n = 130, 8192, 8192, 16
    gu = torch.full((e, 2 * f, kk // 4), 0x55, dtype=torch.uint8, device="cuda")     # zeros
    gu[-1] = 0xAA                                                                    # ones
    dn = torch.full((e, n, f // 4), 0xAA, dtype=torch.uint8, device="cuda")
    one = torch.ones(e, device="cuda")
    x = torch.zeros(2, kk, device="cuda")
    x[:, :127] = 1
    logits = torch.zeros(2, e, device="cuda")
    logits[0, -1] = 9
    logits[1, 0] = 9
    y = bl.experts_ffn(x, logits, 1, gu, one, one, dn, one)
    h = torch.tensor(127.0 ** 3).bfloat16().float()
    assert torch.all(y[1] == 0)
    assert torch.all((y[0] - 8192 * h.cuda()).abs() <= 8192 * h.cuda() * 2.0 ** -22)
