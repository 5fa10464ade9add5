"""The routed-expert operators against their oracle (needs an MI355X).

Whole numbers (experts, slots, int32 sums, int8 codes) and bfloat16 outputs
are compared bit for bit, binary32 outputs within bounds counted from their
roundings, u = 2^-24 each:
  weights   exp of a difference D <= d rounded once (d u relative) by a device
            exp within 1 ulp (2 u), on both sides of a quotient whose sum has
            at most E terms ((E - 1) u), and the quotient (u): within
            (2 d + E + 6) u of the binary64 value
  slot rows (gamma m) / 127 times the sum: three roundings, 4 u with the
            second-order terms
  combined  sum of k products, each of a row within 4 u, added by k fused
            operations: (k + 5) u of sum |w y|
"""

import numpy as np
import pytest
import torch

import oracle
from bitlinear_w1_a8_amd import workloads as wl
from oracle import experts_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NINF = -np.inf


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


# ------------------------------------------------------------------ router

def scores(t, e, seed, kind):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (t, e)) + rng.normal(0, 0.7, e)
    if kind == "ties":
        x = x.round(1)
    elif kind == "equal":
        x[:] = -0.25
    elif kind == "wide":
        x *= 60
    elif kind == "lowest":
        x[rng.random((t, e)) < 0.8] = np.finfo(np.float32).min
    x = x.astype(np.float32)
    if kind == "infinite":
        x[rng.random((t, e)) < 1.5 / e] = np.inf
        x[:, 0] = NINF
    if kind == "masked":
        x[rng.random((t, e)) < 0.5] = NINF
        x[rng.random(t) < 0.3] = NINF
        x[rng.random((t, e)) < 0.1] = np.nan
    elif kind == "empty":
        x[:] = NINF
    elif kind == "zeros":
        x = np.where(rng.random((t, e)) < 0.5, np.float32(0.0), np.float32(-0.0))
    return x


def check_routing(bl, x, xt, k, share):
    ids, w, off, pairs, slots = ref.route(x, k, share)
    r = bl.route_experts(xt, k, share)
    assert np.array_equal(host(r.ids), ids)
    assert np.array_equal(host(r.offsets), off)
    assert np.array_equal(host(r.pairs), pairs)
    assert np.array_equal(host(r.slots), slots)
    with np.errstate(invalid="ignore"):
        usable = np.where(x > NINF, x, np.nan).astype(np.float64)
    got = host(r.weights).astype(np.float64)
    d = np.nan_to_num(np.nanmax(usable, 1, initial=NINF, where=~np.isnan(usable))
                      - np.nanmin(usable, 1, initial=np.inf, where=~np.isnan(usable)), nan=0, neginf=0)
    d = np.minimum(d, 110)[:, None]          # farther terms are 0 in binary32
    # a term that leaves binary32's normal range is off by up to 2^-126 of a sum of at least 1
    assert np.all(np.abs(got - w) <= (2 * d + x.shape[1] + 6) * U * w + 2.0 ** -126)
    again = bl.route_experts(xt, k, share)
    assert torch.equal(again.weights, r.weights) and torch.equal(again.pairs, r.pairs)
    return r


ROUTES = [(1, 1, 1, "normal"), (1, 64, 8, "normal"), (1, 1024, 32, "normal"), (2, 5, 5, "ties"),
          (3, 64, 8, "empty"), (7, 33, 4, "masked"), (63, 65, 6, "ties"), (64, 128, 8, "equal"),
          (65, 128, 8, "masked"), (64, 3, 3, "zeros"), (200, 256, 8, "lowest"), (129, 257, 2, "wide"),
          (1000, 60, 6, "normal"), (4161, 16, 1, "ties"), (300, 8, 8, "masked"), (70, 1000, 9, "ties"),
          (100, 64, 32, "masked"), (128, 7, 2, "empty"), (5, 40, 6, "infinite"), (90, 700, 12, "infinite"),
          (2100, 300, 5, "masked")]


@pytest.mark.parametrize("share", ["chosen", "all"])
@pytest.mark.parametrize("t,e,k,kind", ROUTES, ids=[f"T{t}_E{e}_k{k}_{s}" for t, e, k, s in ROUTES])
def test_route(bl, t, e, k, kind, share):
    x = scores(t, e, t * 1000 + e, kind)
    check_routing(bl, x, dev(x), k, share)


@pytest.mark.parametrize("t,e,k", [(5, 64, 8), (131, 40, 3)])
def test_route_bf16(bl, t, e, k):
    b = wl.bf16_bits(scores(t, e, 17, "masked"))
    x = oracle.widen_bf16(b)
    check_routing(bl, x, dev_bf16(b), k, "all")


def test_route_many_blocks(bl):
    """70000 tokens (1094 blocks: several rounds of the starts' scan), against sorting."""
    x = scores(70000, 12, 3, "ties")
    r = bl.route_experts(dev(x), 3)
    order = np.argsort(-x, axis=1, kind="stable")[:, :3].astype(np.int32)
    assert np.array_equal(host(r.ids), order)
    want = np.argsort(order.reshape(-1), kind="stable")
    assert np.array_equal(host(r.pairs), want)
    assert np.array_equal(np.diff(host(r.offsets)), np.bincount(order.reshape(-1), minlength=12))
    slots = np.empty(210000, np.int64)
    slots[want] = np.arange(210000)
    assert np.array_equal(host(r.slots).reshape(-1), slots)


def test_route_logits_past_32_bits(bl):
    """2^22 + 5 tokens of 1024 experts: logits past element 2^32."""
    t, e = (1 << 22) + 5, 1024
    x = torch.empty(t, e, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(1))
    r = bl.route_experts(x, 2)
    at = torch.cat([torch.arange(50), torch.arange(t - 50, t), torch.arange(0, t, 99991)]).cuda()
    some = bits(x[at]).astype(np.uint32) << 16
    ids, *_ = ref.route(some.view(np.float32), 2)
    assert np.array_equal(host(r.ids[at]), ids)
    flat = r.ids.flatten().long()
    assert int(flat.min()) >= 0 and int(flat.max()) < e
    count = torch.bincount(flat, minlength=e)
    assert torch.equal(r.offsets[1:].long(), count.cumsum(0)) and int(r.offsets[0]) == 0
    # slots and pairs undo each other; along the slots experts, then pairs, grow
    pairs = r.pairs.long()
    assert torch.equal(r.slots.flatten().long()[pairs], torch.arange(2 * t, device="cuda"))
    order = flat[pairs] * (2 * t) + pairs
    assert bool((order[1:] > order[:-1]).all())
    del x, r, flat, pairs, order
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ products

def weights(rng, e, n, k):
    t = rng.integers(-1, 2, (e, n, k)).astype(np.int8)
    packed = np.stack([oracle.pack_ternary(t[i]) for i in range(e)])
    return t, dev(packed), rng.uniform(0.008, 0.024, e).astype(np.float32)


def routing(bl, t, e, k, seed, kind="normal"):
    x = scores(t, e, seed, kind)
    r = bl.route_experts(dev(x), k)
    return r, *[host(a) for a in (r.offsets, r.pairs, r.slots, r.weights)]


def activations(t, k, seed, dtype):
    x = wl.activations_student_t(t, k, 4, seed)
    if t > 2:
        x[1] = 0.0
    if dtype == "bf16":
        b = wl.bf16_bits(x)
        return dev_bf16(b), b
    return dev(x), x


# (T, E, k, N, K, dtype, routing): one token and few (rows per expert in the
# single digits), rows of odd lengths (K of 16, 64, 128, 192 and 16 n), N not a
# multiple of any tile, one expert with everything, experts without rows,
# batches whose experts have from tens to hundreds of rows
GATED = [(1, 8, 2, 40, 256, "bf16", "normal"), (1, 64, 8, 1024, 2560, "bf16", "normal"),
         (1, 4, 4, 7, 16, "f32", "normal"), (2, 16, 3, 33, 48, "f32", "normal"),
         (4, 64, 8, 100, 1024, "bf16", "masked"), (3, 9, 2, 65, 320, "f32", "normal"),
         (33, 64, 6, 250, 512, "bf16", "masked"), (17, 4, 2, 129, 1040, "bf16", "normal"),
         (40, 3, 1, 64, 192, "f32", "equal"), (90, 8, 2, 300, 640, "bf16", "masked"),
         (300, 5, 2, 77, 256, "f32", "normal"), (257, 16, 4, 130, 1088, "bf16", "masked"),
         (700, 4, 3, 520, 384, "bf16", "normal"), (1200, 2, 1, 33, 128, "f32", "normal"),
         (64, 16, 2, 96, 4096, "bf16", "empty"), (1000, 64, 8, 200, 448, "bf16", "ties"),
         # long rows (fewer of them in LDS at a time), many rows of odd lengths,
         # more experts than lanes
         (40, 4, 2, 33, 16400, "bf16", "normal"), (3, 3, 2, 9, 131072, "bf16", "normal"),
         (20, 2, 1, 17, 40000, "f32", "normal"), (400, 3, 2, 70, 272, "bf16", "masked"),
         (2, 4, 2, 20, 8208, "f32", "normal"), (50, 200, 3, 40, 256, "bf16", "masked"),
         (300, 1000, 4, 24, 128, "bf16", "ties"), (4, 1024, 8, 16, 80, "f32", "normal"),
         (600, 520, 8, 20, 208, "bf16", "normal"), (600, 520, 8, 24, 256, "bf16", "masked")]


@pytest.mark.parametrize("t,e,k,n,kk,dtype,kind", GATED,
                         ids=[f"T{c[0]}_E{c[1]}_k{c[2]}_N{c[3]}_K{c[4]}_{c[5]}_{c[6]}" for c in GATED])
def test_gated_experts(bl, t, e, k, n, kk, dtype, kind):
    rng = np.random.default_rng(t + n)
    r, off, pairs, _, _ = routing(bl, t, e, k, 31 * t + e, kind)
    tg, pg, gg = weights(rng, e, n, kk)
    tu, pu, gu = weights(rng, e, n, kk)
    both = torch.stack([bl.interleave_rows(pg[i], pu[i]) for i in range(e)])
    xin, xref = activations(t, kk, 5 + t, dtype)
    q, a, _ = oracle.quant_act(xref)
    out = torch.full((t * k, n), 7.0, dtype=torch.bfloat16, device="cuda")
    h, xq, absmax, acc = bl.gated_relu2_experts(xin, both, dev(gg), dev(gu), r, want_codes=True, want_acc=True,
                                               out=out)
    assert h is out
    given = (host(r.ids) >= 0).any(1)                # tokens with an expert
    assert np.array_equal(host(xq)[given], q[given]) and np.array_equal(host(absmax)[given], a[given])
    used = off[-1]
    h_ref, acc_ref = ref.gated_slots(q, a, tg, tu, gg, gu, off, np.maximum(pairs, 0) // k)
    assert np.array_equal(host(acc)[:used], acc_ref[:used])
    assert np.array_equal(bits(h)[:used], h_ref[:used])
    assert np.all(bits(h)[used:] == 0x40E0)                     # empty slots as they were
    h2 = bl.gated_relu2_experts(xin, both, dev(gg), dev(gu), r)[0]   # without the sums
    assert np.array_equal(bits(h2)[:used], h_ref[:used])


LINEAR = [(1, 8, 2, 40, 256, "bf16", "normal"), (1, 64, 8, 2560, 1024, "bf16", "normal"),
          (1, 5, 5, 9, 16, "f32", "normal"), (2, 16, 3, 34, 48, "f32", "masked"),
          (4, 64, 8, 200, 1728, "bf16", "normal"), (3, 9, 2, 130, 320, "f32", "masked"),
          (5, 12, 12, 67, 640, "bf16", "normal"), (8, 40, 32, 50, 128, "bf16", "masked"),
          (33, 64, 6, 500, 512, "bf16", "masked"), (17, 4, 2, 258, 1040, "bf16", "normal"),
          (40, 3, 1, 128, 192, "f32", "equal"), (90, 8, 2, 601, 640, "bf16", "masked"),
          (300, 5, 2, 154, 256, "f32", "normal"), (257, 16, 4, 260, 1088, "bf16", "masked"),
          (700, 4, 3, 1040, 384, "bf16", "normal"), (1200, 2, 1, 66, 128, "f32", "normal"),
          (64, 16, 2, 192, 4096, "bf16", "empty"), (1000, 64, 8, 400, 448, "bf16", "ties"),
          (2, 6, 2, 96, 6912, "bf16", "normal"),
          (40, 4, 2, 33, 16400, "bf16", "normal"), (2, 3, 1, 9, 131072, "bf16", "normal"),
          (1, 4, 4, 18, 36880, "f32", "normal"), (400, 3, 2, 70, 272, "bf16", "masked"),
          (50, 200, 3, 40, 256, "bf16", "masked"), (300, 1000, 4, 24, 128, "bf16", "ties"),
          (4, 1024, 8, 17, 80, "f32", "normal"), (6, 64, 17, 30, 96, "bf16", "normal"),
          (600, 520, 8, 24, 208, "bf16", "masked"), (600, 520, 8, 20, 256, "bf16", "normal")]


@pytest.mark.parametrize("x_rows", ["slots", "tokens"])
@pytest.mark.parametrize("t,e,k,n,kk,dtype,kind", LINEAR,
                         ids=[f"T{c[0]}_E{c[1]}_k{c[2]}_N{c[3]}_K{c[4]}_{c[5]}_{c[6]}" for c in LINEAR])
def test_linear_experts(bl, t, e, k, n, kk, dtype, kind, x_rows):
    rng = np.random.default_rng(t + n)
    r, off, pairs, slots, w = routing(bl, t, e, k, 37 * t + e, kind)
    tern, packed, gam = weights(rng, e, n, kk)
    rows = t * k if x_rows == "slots" else t
    xin, xref = activations(rows, kk, 9 + t, dtype)
    used = off[-1]
    if x_rows == "slots" and used < rows:
        xin[used:] = float("nan")                    # rows that nothing may read a result from
        xref = xref.copy()
        xref[used:] = 0
    q, a, _ = oracle.quant_act(xref)
    at = np.arange(t * k) if x_rows == "slots" else np.maximum(pairs, 0) // k
    y_ref, acc_ref = ref.linear_slots(q, a, tern, gam, off, at)
    out = torch.full((t * k, n), -3.0, device="cuda")
    y, acc = bl.linear_experts(xin, packed, dev(gam), r, combine=False, x_rows=x_rows, want_acc=True, out=out)
    assert y is out
    assert np.array_equal(host(acc)[:used], acc_ref[:used])
    got = host(y).astype(np.float64)
    assert np.all(np.abs(got - y_ref)[:used] <= 4 * U * np.abs(y_ref)[:used])
    assert np.all(got[used:] == -3.0)
    both, size = ref.combine(y_ref, slots, w)
    got = host(bl.linear_experts(xin, packed, dev(gam), r, x_rows=x_rows)).astype(np.float64)
    assert np.all(np.abs(got - both) <= (k + 5) * U * size)
    assert np.all(got[(slots < 0).all(1)] == 0.0)     # tokens routed nowhere


def test_linear_experts_repeats_bits(bl):
    r, *_ = routing(bl, 500, 16, 4, 71, "masked")
    rng = np.random.default_rng(1)
    _, packed, gam = weights(rng, 16, 300, 512)
    xin, _ = activations(2000, 512, 2, "bf16")
    first = bl.linear_experts(xin, packed, dev(gam), r)
    for _ in range(3):
        assert torch.equal(bl.linear_experts(xin, packed, dev(gam), r), first)


def test_same_expert_twice(bl):
    """A routing not made by the router: both ranks of a token on one expert."""
    t, k, e, n, kk = 6, 2, 3, 50, 256
    rng = np.random.default_rng(8)
    tern, packed, gam = weights(rng, e, n, kk)
    xin, xref = activations(t, kk, 3, "bf16")
    q, a, _ = oracle.quant_act(xref)
    off = np.array([0, 0, 12, 12], np.int32)
    pairs, slots = np.arange(12, dtype=np.int32), np.arange(12, dtype=np.int32).reshape(t, k)
    w = rng.uniform(0.1, 1, (t, k)).astype(np.float32)
    r = bl.Routing(None, dev(w), dev(off), dev(pairs), dev(slots))
    y_ref, _ = ref.linear_slots(q, a, tern, gam, off, pairs // k)
    both, size = ref.combine(y_ref, slots, w)
    got = host(bl.linear_experts(xin, packed, dev(gam), r, x_rows="tokens")).astype(np.float64)
    assert np.all(np.abs(got - both) <= (k + 5) * U * size)


# ------------------------------------------------------------------ as they are used

class Layer:
    """A routed feed-forward layer: SubLN + A1 stay with the caller, router
    logits come in, gate / up, down, weighted sum."""

    def __init__(self, bl, e, d, f, seed):
        rng = np.random.default_rng(seed)
        self.bl = bl
        gate, up, down = (rng.normal(0, 0.02, (e, a, b)).astype(np.float32) for a, b in ((f, d), (f, d), (d, f)))
        pk = lambda w: [bl.pack_weights(dev(x)) for x in w]  # noqa: E731
        g, u, dn = pk(gate), pk(up), pk(down)
        self.gu = torch.stack([bl.interleave_rows(a[0], b[0]) for a, b in zip(g, u)])
        self.gg, self.ug = torch.cat([a[1] for a in g]), torch.cat([a[1] for a in u])
        self.dn, self.dg = torch.stack([a[0] for a in dn]), torch.cat([a[1] for a in dn])
        self.each = (g, u, dn)

    def __call__(self, x, logits, k):
        r = self.bl.route_experts(logits, k)
        h = self.bl.gated_relu2_experts(x, self.gu, self.gg, self.ug, r)[0]
        return self.bl.linear_experts(h, self.dn, self.dg, r), r


@pytest.mark.parametrize("t", [1, 3, 20, 200])
def test_layer_equals_one_expert_at_a_time(bl, t):
    """route -> gated -> down against the framework's single-matrix calls on
    each (token, expert): the same bfloat16 hidden rows, the same sums."""
    e, d, f, k = 6, 512, 320, 2
    layer = Layer(bl, e, d, f, 4)
    x, _ = activations(t, d, 5, "bf16")
    logits = dev(scores(t, e, 6, "normal"))
    y, r = layer(x, logits, k)
    ids, w = host(r.ids), host(r.weights)
    size, want = np.zeros((t, d)), np.zeros((t, d))
    for i in range(min(t, 40)):
        for j in range(k):
            ex = ids[i, j]
            g, u, dn = (m[ex] for m in layer.each)
            hh = bl.gated_relu2(x[i:i + 1].contiguous(), bl.interleave_rows(g[0], u[0]), g[1], u[1])[0]
            one = host(bl.bitlinear(hh, dn[0], dn[1], d)).astype(np.float64)[0] * float(w[i, j])
            want[i] += one
            size[i] += np.abs(one)
    got = host(y).astype(np.float64)
    assert np.all(np.abs(got - want)[:40] <= (k + 9) * U * size[:40])


@pytest.mark.parametrize("t", [1, 2, 37, 300])
def test_layer_on_a_side_stream_and_in_a_graph(bl, t):
    e, d, f, k = 8, 256, 192, 3
    layer = Layer(bl, e, d, f, 14)
    xs = [activations(t, d, 20 + i, "bf16")[0] for i in range(4)]
    ls = [dev(scores(t, e, 30 + i, "masked" if t > 2 else "normal")) for i in range(4)]
    eager = [layer(x, l, k)[0].clone() for x, l in zip(xs, ls)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(4):                       # two streams at once
        with torch.cuda.stream(side[i % 2]):
            got.append(layer(xs[i], ls[i], k)[0])
    torch.cuda.synchronize()
    for a, b in zip(got, eager):
        assert torch.equal(a, b)
    x, l = xs[0].clone(), ls[0].clone()
    layer(x, l, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, l, k)[0]
    for i in (1, 2, 3, 0, 1):                # replays, eager work between them
        x.copy_(xs[i])
        l.copy_(ls[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])
        assert torch.equal(layer(xs[i], ls[i], k)[0], eager[i])


# ------------------------------------------------------------------ sizes past 32 bits

def test_expert_matrices_past_32_bits(bl):
    """1024 experts of 8.4 MB: matrices from byte 2^33 on."""
    e, n, kk, t = 1024, 1 << 17, 256, 2
    rng = np.random.default_rng(3)
    packed = torch.full((e, n, kk // 4), 0x55, dtype=torch.uint8, device="cuda")      # t = 0
    tern = rng.integers(-1, 2, (n, kk)).astype(np.int8)
    packed[e - 1] = dev(oracle.pack_ternary(tern))
    gam = np.full(e, 0.01, np.float32)
    x, xref = activations(t, kk, 4, "bf16")
    q, a, _ = oracle.quant_act(xref)
    off = np.full(e + 1, 0, np.int32)
    off[e] = t                                               # both tokens on the last expert
    pairs = np.arange(t, dtype=np.int32)
    r = bl.Routing(None, torch.ones(t, 1, device="cuda"), dev(off), dev(pairs), dev(pairs.reshape(t, 1)))
    y, acc = bl.linear_experts(x, packed, dev(gam), r, combine=False, x_rows="tokens", want_acc=True)
    assert np.array_equal(host(acc), oracle.contract(q, tern))
    y2 = bl.linear_experts(x, packed, dev(gam), r, x_rows="tokens")
    assert torch.equal(y2, y)
    del packed
    torch.cuda.empty_cache()


@pytest.mark.parametrize("combine", [False, True])
def test_rows_past_32_bits(bl, combine):
    """2^19 + 3 tokens with 4112 outputs: y from element 2^31 on."""
    t, e, n, kk = (1 << 19) + 3, 4, 4112, 64
    rng = np.random.default_rng(4)
    tern, packed, gam = weights(rng, e, n, kk)
    x = torch.randint(-127, 128, (t, kk), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).float()
    x[:, 0] = 127.0                                          # absmax 127: the codes are x itself
    logits = torch.randn(t, e, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    r = bl.route_experts(logits, 1)
    y = bl.linear_experts(x, packed, dev(gam), r, combine=combine, x_rows="tokens")
    ids = logits.argmax(1)
    where = torch.cat([torch.arange(40), torch.arange(t - 40, t), torch.arange(0, t, 9973)]).cuda()
    rows = where if combine else r.slots[where, 0].long()
    got = y[rows].cpu().double().numpy()
    xs, es = x[where].cpu().double().numpy(), ids[where].cpu().numpy()
    want = np.einsum("tk,tnk->tn", xs, tern[es].astype(np.float64)) * gam[es].astype(np.float64)[:, None]
    # absmax / 127 = 1 here; the weight of a single expert is exactly 1
    assert np.all(np.abs(got - want) <= 6 * U * np.abs(want))
    del y
    torch.cuda.empty_cache()


def test_more_rows_than_a_launch_takes(bl):
    """2^26 + 9 slots of K = 16, one row of x each: more than 2^32 threads of step A1."""
    t, k, e, kk = (1 << 26) // 8 + 1, 8, 8, 16
    p = t * k
    tern, packed, gam = weights(np.random.default_rng(5), e, 4, kk)
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(p, kk, device="cuda", generator=gen, dtype=torch.bfloat16)
    r = bl.route_experts(torch.randn(t, e, device="cuda", generator=gen), k)   # every expert: t slots each
    y = bl.linear_experts(x, packed, dev(gam), r, combine=False)
    for i in (0, 3, e - 1):
        at = slice(i * t, (i + 1) * t)
        rows = torch.cat([torch.arange(70), torch.arange(t - 70, t), torch.arange(0, t, 99991)]).cuda()
        q, a = bl.quant_act(x[at][rows].contiguous())[:2]
        want = bl.forward(packed[i].contiguous(), dev(gam[i:i + 1]), q, a, 4)
        assert torch.equal(y[at][rows], want[0] if isinstance(want, tuple) else want)
    del x, y, r
    torch.cuda.empty_cache()


def test_as_many_outputs_as_there_may_be(bl):
    """2^26 outputs of one token with 16 experts: more blocks than the kernel of
    few tokens may launch."""
    n, k, kk = 1 << 26, 16, 16
    gen = torch.Generator("cuda").manual_seed(4)
    packed = torch.full((k, n, kk // 4), 0x55, dtype=torch.uint8, device="cuda")         # t = 0
    rng = np.random.default_rng(6)
    tern, small, gam = weights(rng, k, 100, kk)
    packed[:, :50], packed[:, -50:] = small[:, :50], small[:, 50:]
    x, _ = activations(1, kk, 7, "f32")
    r = bl.route_experts(torch.randn(1, k, device="cuda", generator=gen), k)
    y = bl.linear_experts(x, packed, dev(gam), r, x_rows="tokens")
    want = bl.linear_experts(x, small, dev(gam), r, x_rows="tokens")
    assert torch.equal(y[:, :50], want[:, :50]) and torch.equal(y[:, -50:], want[:, 50:])
    assert int(torch.count_nonzero(y[:, 50:-50])) == 0
    del packed, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("t,e,k,kk", [(2, 9, 3, 64), (40, 9, 3, 80), (600, 9, 3, 128), (600, 70, 2, 64)])
def test_routing_of_anything_stays_in_bounds(bl, t, e, k, kk):
    """Arrays that the router would not write: the calls end and nothing beside
    the outputs changes."""
    n = 40
    rng = np.random.default_rng(t + e)
    def some(shape):
        v = rng.integers(-2 ** 31, 2 ** 31, shape)
        return dev(np.where(rng.random(shape) < 0.5, v, rng.integers(-2, t * k + 2, shape)).astype(np.int32))
    r = bl.Routing(None, torch.ones(t, k, device="cuda"), some(e + 1), some(t * k), some((t, k)))
    _, gu, gam = weights(rng, e, 2 * n, kk)
    _, dn, _ = weights(rng, e, n, kk)
    x = activations(t, kk, 1, "bf16")[0]
    xs = activations(t * k, kk, 2, "bf16")[0]
    def padded(rows, dtype):
        whole = torch.full((rows + 2, n), 7, dtype=dtype, device="cuda")
        return whole, whole[1:-1]
    # an output begins one row in: 80 or 160 bytes, a multiple of 16
    h_all, h = padded(t * k, torch.bfloat16)
    bl.gated_relu2_experts(x, gu, dev(gam), dev(gam), r, out=h)
    y_all, y = padded(t, torch.float32)
    bl.linear_experts(xs, dn, dev(gam), r, out=y)
    s_all, s = padded(t * k, torch.float32)
    bl.linear_experts(x, dn, dev(gam), r, combine=False, x_rows="tokens", out=s)
    for whole in (h_all, y_all, s_all):
        assert bool((whole[0] == 7).all()) and bool((whole[-1] == 7).all())


# ------------------------------------------------------------------ refusals of the binding

def _good(bl):
    r, *_ = routing(bl, 4, 5, 2, 1)
    return dict(x=torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"),
                gu=torch.zeros(5, 12, 16, dtype=torch.uint8, device="cuda"),
                g=torch.ones(5, device="cuda"), r=r)


@pytest.mark.parametrize("case", ["x_rows", "x_f16", "x_strided", "gu_k", "gu_odd", "gu_e", "gamma", "out", "pairs",
                                  "weights", "offsets_i64", "slots_1d"])
def test_binding_refuses(bl, case):
    v = _good(bl)
    out = None
    r = v["r"]
    if case == "x_rows": v["x"] = v["x"][:3].contiguous()
    elif case == "x_f16": v["x"] = v["x"].half()
    elif case == "x_strided": v["x"] = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")[:, ::2]
    elif case == "gu_k": v["gu"] = torch.zeros(5, 12, 12, dtype=torch.uint8, device="cuda")
    elif case == "gu_odd": v["gu"] = torch.zeros(5, 11, 16, dtype=torch.uint8, device="cuda")
    elif case == "gu_e": v["gu"] = v["gu"][:4].contiguous()
    elif case == "gamma": v["g"] = torch.ones(1, device="cuda")
    elif case == "out": out = torch.zeros(8, 5, dtype=torch.bfloat16, device="cuda")
    elif case == "pairs": r.pairs = r.pairs[:7].contiguous()
    elif case == "weights": r.weights = r.weights[:, :1].contiguous()
    elif case == "offsets_i64": r.offsets = r.offsets.long()
    elif case == "slots_1d": r.slots = r.slots.flatten()
    with pytest.raises((TypeError, ValueError)):
        bl.gated_relu2_experts(v["x"], v["gu"], v["g"], v["g"], r, out=out)


def test_calls_refused(bl):
    from bitlinear_w1_a8_amd import BitLinearError
    with pytest.raises(ValueError):
        bl.route_experts(torch.zeros(2, 4, device="cuda"), 0)
    with pytest.raises(ValueError):
        bl.route_experts(torch.zeros(2, 4, device="cuda"), 2, share="none")
    with pytest.raises(BitLinearError):
        bl.route_experts(torch.zeros(2, 4, device="cuda"), 5)
    with pytest.raises(BitLinearError):
        bl.route_experts(torch.zeros(0, 4, device="cuda"), 1)
    v = _good(bl)
    h = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    dn = torch.zeros(5, 20, 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        bl.linear_experts(h, dn, v["g"], v["r"], x_rows="pairs")
    with pytest.raises(ValueError):
        bl.linear_experts(h, dn, v["g"], v["r"], want_acc=True)
    with pytest.raises(ValueError):
        bl.linear_experts(h, dn, v["g"], v["r"], x_rows="tokens")
