"""The 4-bit operators against their oracle (needs an MI355X).

Codes, scales and zero points are compared bit for bit; unpacked values are
exact.  y: each of the K / G groups' sums is exact, its product with the scale
and the additions (fused, at most one rounding each, over the groups and the
partial sums' joins), absmax / 127 and the last product round once each:
within (K / G + 40) u of the sum of |s * group sum| * m / 127, u = 2^-24, for
at most 36 joins."""

import numpy as np
import pytest
import torch

import oracle
from bitlinear_w1_a8_amd import workloads as wl
from oracle import w4_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def bl(built_lib):
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import bitlinear_w1_a8_amd
    bitlinear_w1_a8_amd.load()
    return bitlinear_w1_a8_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def bits(t):
    torch.cuda.synchronize()
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def latent(n, k, kind, seed):
    rng = np.random.default_rng(seed)
    w = rng.normal(0, 0.02, (n, k))
    if kind == "shifted":
        w += 0.05
    elif kind == "negative":
        w = -np.abs(w)
    elif kind == "ties":            # scales of 1, quotients that end in .5
        w = rng.integers(-14, 15, (n, k)) / 2
        w[:, ::32] = 7.0
    elif kind == "tiny":            # scales below and around bfloat16's smallest
        w = rng.normal(0, 1, (n, k)) * 10.0 ** rng.uniform(-44, -38, (n, 1))
    elif kind == "huge":
        w = rng.normal(0, 1, (n, k)) * 4e37
    elif kind == "zeros":
        w[:, : k // 2] = 0
        w[0] = 0
    elif kind == "outliers":
        w[rng.random((n, k)) < 0.01] *= 300
    return w.astype(np.float32)


PACK = [(1, 32, 32), (3, 64, 64), (5, 128, 128), (7, 96, 32), (33, 320, 64), (20, 2560, 128), (300, 416, 32),
        (64, 1088, 64), (9, 6912, 128)]


@pytest.mark.parametrize("kind", ["normal", "shifted", "negative", "ties", "tiny", "huge", "zeros", "outliers"])
@pytest.mark.parametrize("with_zeros", [False, True], ids=["sym", "zp"])
@pytest.mark.parametrize("n,k,g", PACK, ids=[f"N{n}_K{k}_g{g}" for n, k, g in PACK])
def test_pack_and_unpack(bl, n, k, g, with_zeros, kind):
    w = latent(n, k, kind, n * 7 + k)
    t, s, z = ref.quantize(w, g, with_zeros)
    packed, scales, zeros = bl.pack_weights_w4(dev(w), g, with_zeros)
    assert np.array_equal(bits(scales), s)
    if with_zeros:
        assert np.array_equal(host(zeros), z)
    else:
        assert zeros is None
    assert np.array_equal(host(packed), ref.pack(t))
    v = host(bl.unpack_weights_w4(packed, scales, zeros, k))
    with np.errstate(under="ignore"):
        assert np.array_equal(v, ref.values(t, s, z).astype(np.float32))


def tokens(t, k, seed):
    rng = np.random.default_rng(seed)
    q = np.clip(np.rint(rng.normal(0, 40, (t, k))), -127, 127).astype(np.int8)
    if t > 1:
        q[1] = 127
    if t > 2:
        q[2] = 0
    a = rng.uniform(0.1, 4, t).astype(np.float32)
    a[-1] = 0.0
    return q, a


# (T, N, K, G): one token and few, past one, two and four tiles of 16 tokens,
# many; rows that end inside a block of 128; N from one row to thousands
FORWARD = [(1, 1, 32, 32), (1, 17, 64, 64), (1, 16, 128, 128), (1, 100, 160, 32), (1, 640, 2560, 128),
           (1, 2560, 6912, 64), (1, 5000, 1024, 128), (2, 33, 320, 64), (3, 130, 416, 32), (4, 257, 2560, 32),
           (5, 70, 8192, 128), (7, 2560, 1728, 32), (8, 48, 192, 64), (15, 31, 512, 128), (16, 64, 640, 64),
           (17, 50, 1088, 64), (31, 200, 384, 32), (33, 129, 1280, 128), (48, 100, 96, 32), (64, 300, 2560, 128),
           (65, 77, 320, 64), (100, 513, 640, 128), (127, 250, 1024, 32), (128, 256, 256, 64), (129, 260, 192, 64),
           (200, 1000, 512, 128), (300, 128, 2560, 64), (513, 400, 416, 32), (1000, 700, 384, 128),
           (2, 20000, 256, 128), (1, 3, 131072, 128), (70, 20, 32768, 64)]


@pytest.mark.parametrize("with_zeros", [False, True], ids=["sym", "zp"])
@pytest.mark.parametrize("t,n,k,g", FORWARD, ids=[f"T{c[0]}_N{c[1]}_K{c[2]}_g{c[3]}" for c in FORWARD])
def test_forward(bl, t, n, k, g, with_zeros):
    rng = np.random.default_rng(n + k)
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    codes[0] = -8                                        # the largest sums
    s = wl.bf16_bits(rng.uniform(0.002, 0.02, (n, k // g)).astype(np.float32))
    z = rng.integers(-8, 8, (n, k // g)).astype(np.int8) if with_zeros else np.zeros((n, k // g), np.int8)
    if with_zeros:
        z[0] = 7
    q, a = tokens(t, k, t + k)
    want, size = ref.forward(codes, s, z, q, a)
    args = (dev(ref.pack(codes)), dev_bf16(s), dev(q), dev(a))
    zt = dev(z) if with_zeros else None
    y = bl.forward_w4(*args, zeros=zt)
    assert np.all(np.abs(host(y).astype(np.float64) - want) <= (k // g + 40) * U * size)
    out = torch.full((t, n), 5.0, device="cuda")
    assert bl.forward_w4(*args, zeros=zt, out=out) is out
    assert torch.equal(out, y)


def test_tokens_of_a_batch_do_not_meet(bl):
    """A token's row does not depend on the others' values, within one shape."""
    k, n = 512, 300
    w = dev(latent(n, k, "normal", 5))
    packed, scales, zeros = bl.pack_weights_w4(w, 64, True)
    for t in (3, 40, 150):
        q, a = tokens(t, k, 1)
        y = bl.forward_w4(packed, scales, dev(q), dev(a), zeros=zeros)
        q2, a2 = tokens(t, k, 2)
        q2[0], a2[0] = q[0], a[0]
        a2[1:] = np.inf
        y2 = bl.forward_w4(packed, scales, dev(q2), dev(a2), zeros=zeros)
        assert torch.equal(y[0], y2[0])


@pytest.mark.parametrize("t", [1, 9, 140])
def test_head_after_subln(bl, t):
    """A vocabulary projection as it is used: SubLN + A1, then 4-bit rows; the
    result against the unpacked matrix on A1's codes; on a side stream and in
    graph replays too."""
    k, n, g = 640, 1003, 128
    gain = dev(np.random.default_rng(2).uniform(0.5, 1.5, k).astype(np.float32))
    w = dev(latent(n, k, "normal", 3))
    packed, scales, zeros = bl.pack_weights_w4(w, g)
    xs = [dev_bf16(wl.bf16_bits(wl.activations_student_t(t, k, 4, 40 + i))) for i in range(3)]

    def head(x):
        xq, scale, _ = bl.subln_quant_act(x, gain, with_rowsum=False)
        return bl.forward_w4(packed, scales, xq, scale, zeros=zeros), xq, scale

    v = host(bl.unpack_weights_w4(packed, scales, zeros, k)).astype(np.float64)
    eager = []
    for x in xs:
        y, xq, scale = head(x)
        m = np.maximum(host(scale), np.float32(1e-5)).astype(np.float64)[:, None] / 127
        want = host(xq).astype(np.float64) @ v.T * m
        size = np.abs(host(xq).astype(np.float64)) @ np.abs(v).T * m
        assert np.all(np.abs(host(y) - want) <= (k // g + 40) * U * size)
        eager.append(y.clone())
    with torch.cuda.stream(torch.cuda.Stream()):
        y = head(xs[1])[0]
    torch.cuda.synchronize()
    assert torch.equal(y, eager[1])
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = head(x)[0]
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])
        assert torch.equal(head(xs[i])[0], eager[i])


@pytest.mark.parametrize("t", [1, 20, 80])
def test_matrix_past_32_bits(bl, t):
    """2^20 + 5 rows of 8192 weights: bytes from 2^32 on, y up to 84 M entries."""
    n, k, g = (1 << 20) + 5, 8192, 128
    packed = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((n, k // g), 0.5, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(9)
    codes = rng.integers(-8, 8, (37, k)).astype(np.int8)
    packed[-37:] = dev(ref.pack(codes))
    q, a = tokens(t, k, 3)
    y = bl.forward_w4(packed, scales, dev(q), dev(a))
    s = wl.bf16_bits(np.full((37, k // g), 0.5, np.float32))
    want, size = ref.forward(codes, s, np.zeros((37, k // g), np.int8), q, a)
    assert np.all(np.abs(host(y[:, -37:]).astype(np.float64) - want) <= (k // g + 40) * U * size)
    assert not bool(y[:, :-37].any())
    del packed, scales, y
    torch.cuda.empty_cache()


def test_binding_refuses(bl):
    from bitlinear_w1_a8_amd import BitLinearError
    w = torch.zeros(4, 256, device="cuda")
    packed, scales, zeros = bl.pack_weights_w4(w, 64, True)
    xq = torch.zeros(2, 256, dtype=torch.int8, device="cuda")
    a = torch.ones(2, device="cuda")
    bl.forward_w4(packed, scales, xq, a, zeros=zeros)
    bad = [lambda: bl.pack_weights_w4(w, 48), lambda: bl.pack_weights_w4(w.double(), 64),
           lambda: bl.pack_weights_w4(w[:, :96].contiguous(), 64), lambda: bl.pack_weights_w4(w.t(), 64),
           lambda: bl.pack_weights_w4(w[0], 64),
           lambda: bl.forward_w4(packed[:3].contiguous(), scales, xq, a),
           lambda: bl.forward_w4(packed[:, :64].contiguous(), scales, xq, a),
           lambda: bl.forward_w4(packed, scales[:, :3].contiguous(), xq, a),
           lambda: bl.forward_w4(packed, scales.half(), xq, a),
           lambda: bl.forward_w4(packed, scales, xq, a[:1].contiguous()),
           lambda: bl.forward_w4(packed, scales, xq, a, zeros=zeros[:, :2].contiguous()),
           lambda: bl.forward_w4(packed, scales, xq[:, :128].contiguous(), a),
           lambda: bl.forward_w4(packed, scales, xq, a, out=torch.zeros(2, 5, device="cuda")),
           lambda: bl.unpack_weights_w4(packed, scales, zeros, 128)]
    for f in bad:
        with pytest.raises((TypeError, ValueError, BitLinearError)):
            f()
    # two groups of 128 for a matrix packed with four of 64: another meaning, same extents
    assert bl.unpack_weights_w4(packed, scales[:, :2].contiguous(), None, 256).shape == (4, 256)
    with pytest.raises(BitLinearError):      # one group of 256: no such group size
        bl.unpack_weights_w4(packed, scales[:, :1].contiguous(), None, 256)
