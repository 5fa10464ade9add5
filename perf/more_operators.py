"""Measured cases of the residual norms with 8-bit outputs, the 8-bit floating
point product and the whole routed layer.

The plain forms below compute in binary32 (binary64 where a rounding decides an
8-bit code or a bfloat16) with elementary torch operations; with ``own`` set,
``run`` calls the package's entry points on the same tensors.

Operators (the case key ``op``):
  norm   the residual's addition and the sub-layer norm, its output in 8 bits:
         int8 codes with one scale per token (``bits`` "i8") or e4m3 with one
         scale per 128 (``bits`` "f8")
  pack   e4m3 quantisation of a matrix with one scale per block of 128 x 128
  f8     product of tokens and a matrix in e4m3, the tokens with one scale per
         128; ``raw``: of bfloat16 tokens, quantised within the call
  ffn    a routed layer, from the router's logits to the weighted sum over a
         token's experts (squared-ReLU gate); ``x``: raw activations or int8
         codes with their absmax
"""

import math

import torch

own = False

EPS = 1e-5              # floor of a token's absmax, and the norms' epsilon
TINY = 2.0 ** -100      # floor of an e4m3 group's absmax
TOP = 448.0             # largest e4m3
INF = float("inf")
_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token between two layers: a binary32 projection joins a bfloat16 residual
        {"name": "norm_t1", "op": "norm", "bits": "i8", "T": 1, "K": 2560, "x": "f32", "res": "bf16"},
        # a prompt between two layers, int8 codes for ternary projections
        {"name": "norm_t2048", "op": "norm", "bits": "i8", "T": 2048, "K": 2560, "x": "f32", "res": "bf16"},
        # a 70B-class prompt whose residual is kept in binary32, e4m3 out
        {"name": "norm_f8_t1000", "op": "norm", "bits": "f8", "T": 1000, "K": 8192, "x": "bf16", "res": "f32"},
        # a small projection, one partial row block and column block
        {"name": "pack_576x2512", "op": "pack", "N": 576, "K": 2512},
        # a 70B-class matrix
        {"name": "pack_28672x8192", "op": "pack", "N": 28672, "K": 8192},
        # vocabulary projection of one decoded token
        {"name": "f8_t1_head", "op": "f8", "T": 1, "N": 128256, "K": 2560, "raw": False, "out": "f32"},
        # a ragged decode batch from bfloat16 activations
        {"name": "f8_t13_raw", "op": "f8", "T": 13, "N": 2560, "K": 6912, "raw": True, "out": "f32"},
        # a 70B-class matrix and a batch that the weights no longer bound
        {"name": "f8_t250", "op": "f8", "T": 250, "N": 28672, "K": 8192, "raw": False, "out": "f32"},
        # a prompt of 2048 tokens
        {"name": "f8_t2048", "op": "f8", "T": 2048, "N": 6912, "K": 2560, "raw": False, "out": "bf16"},
        # one decoded token through its 8 experts, from the norm's int8 codes
        {"name": "ffn_t1", "op": "ffn", "T": 1, "E": 64, "k": 8, "F": 1024, "K": 2560, "x": "i8", "logits": "f32", "share": "chosen", "pad": 0.0},
        # a few sessions, raw activations, an odd width
        {"name": "ffn_t3_raw", "op": "ffn", "T": 3, "E": 64, "k": 6, "F": 1008, "K": 2560, "x": "bf16", "logits": "bf16", "share": "all", "pad": 0.0},
        # a decode batch of 16 sessions, some of them idle
        {"name": "ffn_t16", "op": "ffn", "T": 16, "E": 64, "k": 8, "F": 1024, "K": 2560, "x": "i8", "logits": "f32", "share": "chosen", "pad": 0.1},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "f8", "f8", "f8", "ffn", "ffn"])
    if op == "norm":
        k = 16 * _spread(rng, 8, 1792)
        return {"op": op, "bits": rng.choice(["i8", "f8"]), "T": _spread(rng, 1, max(1, min(4096, (1 << 23) // k))), "K": k,
                "x": rng.choice(["f32", "bf16"]), "res": rng.choice(["f32", "bf16", "none"])}
    if op == "pack":
        k = 16 * _spread(rng, 8, 1024)
        return {"op": op, "N": _spread(rng, 16, min(32768, 28672 * 8192 // k)), "K": k}
    if op == "f8":
        k = 16 * _spread(rng, 8, 768)
        n = _spread(rng, 16, min(131072, 2560 * 131072 // k))
        full = 250 * 28672 * 8192
        return {"op": op, "T": _spread(rng, 1, max(1, min(2048, full // (n * k)))), "N": n, "K": k, "raw": rng.random() < 0.4,
                "out": rng.choice(["f32", "bf16"])}
    e = _spread(rng, 4, 128)
    k = rng.randint(1, min(8, e))
    f, kk = 16 * _spread(rng, 4, 128), rng.choice([16, 64])
    kk *= _spread(rng, 256 // kk, 4096 // kk)
    e = max(k, min(e, 2 * 64 * 1024 * 2560 // (f * kk)))
    t = _spread(rng, 1, max(1, min(32, 16 * 8 * 1024 * 2560 // (k * f * kk))))
    return {"op": op, "T": t, "E": e, "k": k, "F": f, "K": kk, "x": rng.choice(["i8", "i8", "bf16", "f32"]),
            "logits": rng.choice(["f32", "bf16"]), "share": rng.choice(["chosen", "all"]), "pad": rng.choice([0.0, 0.1]) if t > 4 else 0.0}


# ----------------------------------------------------------------- inputs

def _hidden(g, t, k):
    # activations with a few outlying features, as a trained model's residual has
    x = torch.randn(t, k, generator=g, device="cuda")
    x[:, torch.randint(0, k, (max(1, k // 500),), generator=g, device="cuda")] *= 20
    return x


def _ternary(g, *shape):
    # packed codes 0, 1, 2 (for -1, 0, +1), about a third zeros as absmean ternarisation gives
    c = torch.randint(0, 3, (4, *shape[:-1], shape[-1] // 4), generator=g, device="cuda", dtype=torch.uint8)
    return c[0] | (c[1] << 2) | (c[2] << 4) | (c[3] << 6)


def _gammas(g, e):
    return 0.016 * (0.5 + torch.rand(e, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "norm":
        t, k = case["T"], case["K"]
        s["x"] = (0.5 * torch.randn(t, k, generator=g, device="cuda")).to(_DTYPES[case["x"]])
        s["res"] = None if case["res"] == "none" else _hidden(g, t, k).to(_DTYPES[case["res"]])
        s["gain"] = 1 + 0.2 * torch.randn(k, generator=g, device="cuda")
        s["total"] = None if s["res"] is None else torch.empty_like(s["res"])
    elif op == "pack":
        s["w"] = 0.02 * torch.randn(case["N"], case["K"], generator=g, device="cuda")
        s["w"][:130] = 0      # a block of zeros and part of another, as unused vocabulary entries leave them
    elif op == "f8":
        t, n, k = case["T"], case["N"], case["K"]
        kb = -(-k // 128)
        w = torch.randn(n, k, generator=g, device="cuda").mul_(100).clamp_(-TOP, TOP)
        s["w"] = w.to(torch.float8_e4m3fn)
        s["ws"] = 2e-4 * (0.5 + torch.rand(-(-n // 128), kb, generator=g, device="cuda"))
        if case["raw"]:
            s["x"] = _hidden(g, t, k).bfloat16()
        else:
            s["x"] = torch.randn(t, k, generator=g, device="cuda").mul_(140).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
            s["xs"] = 0.007 * (0.5 + torch.rand(kb, t, generator=g, device="cuda"))
        s["out"] = torch.empty(t, n, dtype=_DTYPES[case["out"]], device="cuda")
    else:
        t, e, f, k = case["T"], case["E"], case["F"], case["K"]
        l = torch.randn(t, e, generator=g, device="cuda") + 0.7 * torch.randn(1, e, generator=g, device="cuda")
        if case["pad"]:      # idle sessions are masked to -inf throughout
            l[torch.rand(t, generator=g, device="cuda") < case["pad"]] = -INF
        s["logits"] = l.to(_DTYPES[case["logits"]])
        x = torch.randn(t, k, generator=g, device="cuda")
        if case["x"] == "i8":
            s["x"], s["absmax"] = _codes(x)
        else:
            s["x"], s["absmax"] = x.to(_DTYPES[case["x"]]), None
        s["gu"], s["down"] = _ternary(g, e, 2 * f, k), _ternary(g, e, k, f)      # gate and up rows alternate
        s["gate"], s["up"], s["dg"] = _gammas(g, e), _gammas(g, e), _gammas(g, e)
        s["out"] = torch.empty(t, k, device="cuda")
    return s


# ------------------------------------------------------------ plain forms

def _codes(x):
    """int8 codes of each row, and its absmax."""
    x = x.float()
    a = x.abs().amax(1)
    s = (127.0 / a.clamp_min(torch.tensor(EPS, device=a.device)).double()).float()
    return (x * s[:, None]).round().clamp(-127, 127).to(torch.int8), a


def _groups(x):
    """[T, K] as [T, groups of 128, 128], zeros past K."""
    k = x.shape[1]
    return torch.nn.functional.pad(x, (0, -k % 128)).view(x.shape[0], -1, 128)


def _e4m3(v, m):
    """Values v (binary32) with group maxima m as e4m3 codes and their scale."""
    m = m.clamp_min(TINY).double()
    return (v * (TOP / m).float()).to(torch.float8_e4m3fn), (m / TOP).float()


def _quant_f8(x):
    x = x.float()
    t, k = x.shape
    v = _groups(x)
    q, s = _e4m3(v, v.abs().amax(2, keepdim=True))
    return q.reshape(t, -1)[:, :k].contiguous(), s[:, :, 0].t().contiguous()


def _norm(s):
    x, res = s["x"].float(), s["res"]
    total = None
    if res is not None:
        total = (x + res.float()).to(res.dtype)
        x = total.float()
    ms = (x.double().square().sum(1) / x.shape[1]).float()
    root = (ms + torch.tensor(EPS, device=ms.device)).double().sqrt().float()
    r = (1 / root.double()).float()
    hat = x * s["gain"] * r[:, None]
    out = {} if total is None else {"total": total}
    if s["case"]["bits"] == "f8":
        out["q"], out["scale"] = _quant_f8(hat)
    else:
        out["q"], out["scale"] = _codes(hat)
        out["rowsum"] = out["q"].sum(1, dtype=torch.int32)
    return out


def _blocks(w):
    """[N, K] as [row blocks, 128, column blocks, 128], zeros past the edges."""
    n, k = w.shape
    w = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128))
    return w.view(w.shape[0] // 128, 128, -1, 128)


def _pack(w):
    n, k = w.shape
    v = _blocks(w)
    q, s = _e4m3(v, v.abs().amax((1, 3), keepdim=True))
    return {"q": q.reshape(v.shape[0] * 128, -1)[:n, :k].contiguous(), "scale": s[:, 0, :, 0].contiguous()}


def _f8(s):
    t, n, k = (s["case"][i] for i in ("T", "N", "K"))
    q, xs = _quant_f8(s["x"]) if s["case"]["raw"] else (s["x"], s["xs"])
    x = q.float() * xs.t().repeat_interleave(128, 1)[:, :k]
    w = _blocks(s["w"].float()) * s["ws"][:, None, :, None]
    w = w.reshape(w.shape[0] * 128, -1)[:n, :k]
    return torch.matmul(x, w.t()).to(s["out"].dtype)


def _matrices(packed):
    """Ternary values, binary32, of packed rows (four codes per byte; weight 16g + 4j + i in bits 2j of byte i of word g)."""
    b = packed.view(*packed.shape[:-1], -1, 1, 4)
    j = 2 * torch.arange(4, device=b.device, dtype=torch.uint8).view(4, 1)
    return ((b >> j) & 3).float().flatten(-3) - 1


def _choices(l, k, share):
    """Experts [T, k] by falling logit (equal ones by the lower expert; -1 where there is none) and their weights."""
    v, idx = torch.sort(torch.nan_to_num(l.float(), nan=-INF, posinf=INF, neginf=-INF), dim=1, descending=True, stable=True)
    top, ids = v[:, :k], idx[:, :k]
    m = v[:, :1]
    over = top if share == "chosen" else v
    total = torch.where(over > -INF, torch.where(over == m, 1.0, torch.exp(over - m)), 0.0).sum(1, keepdim=True)
    weights = torch.where(top > -INF, torch.where(top == m, 1.0, torch.exp(top - m)) / total, 0.0)
    return torch.where(top > -INF, ids, -1), weights


def _pairs(q, packed, ids):
    """Sums of the rows q [P, K] with the matrices of their experts: [P, N]."""
    out = torch.empty(q.shape[0], packed.shape[1], device=q.device)
    step = max(1, (1 << 30) // (packed.shape[1] * q.shape[1]))
    for p in range(0, q.shape[0], step):
        out[p:p + step] = torch.matmul(_matrices(packed[ids[p:p + step]]), q[p:p + step, :, None])[:, :, 0]
    return out


def _ffn(s):
    t, k = s["case"]["T"], s["case"]["k"]
    ids, weights = _choices(s["logits"], k, s["case"]["share"])
    q, a = (s["x"], s["absmax"]) if s["absmax"] is not None else _codes(s["x"])
    floor = torch.tensor(EPS, device=a.device)
    e = ids.clamp_min(0).flatten()
    acc = _pairs(q.float().repeat_interleave(k, 0), s["gu"], e).double()
    m = a.clamp_min(floor).double().repeat_interleave(k)
    gate = (acc[:, 0::2] * s["gate"][e].double()[:, None] * m[:, None] / 127).float()
    up = (acc[:, 1::2] * s["up"][e].double()[:, None] * m[:, None] / 127).float()
    gate = gate.clamp_min(0)
    h = (gate * gate * up).bfloat16()
    q, a = _codes(h)
    y = _pairs(q.float(), s["down"], e) * (s["dg"][e] * a.clamp_min(floor) / 127)[:, None]
    return (torch.where(ids >= 0, weights, 0.0)[:, :, None] * y.view(t, k, -1)).sum(1)


# -------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import bitlinear_w1_a8_amd as bl

        if op == "norm":
            if c["bits"] == "f8":
                q, scale, total = bl.add_subln_quant_act_f8(s["x"], s["res"], s["gain"], out=s["total"])
                out = {"q": q, "scale": scale}
            else:
                q, scale, rowsum, total = bl.add_subln_quant_act(s["x"], s["res"], s["gain"], out=s["total"])
                out = {"q": q, "scale": scale, "rowsum": rowsum}
            return out if total is None else {"total": total, **out}
        if op == "pack":
            return dict(zip(("q", "scale"), bl.pack_weights_f8(s["w"])))
        if op == "f8":
            if c["raw"]:
                return {"y": bl.linear_f8(s["x"], s["w"], s["ws"], out=s["out"])}
            return {"y": bl.forward_f8(s["w"], s["ws"], s["x"], s["xs"], out=s["out"])}
        return {"y": bl.experts_ffn(s["x"], s["logits"], c["k"], s["gu"], s["gate"], s["up"], s["down"], s["dg"],
                                    absmax=s["absmax"], share=c["share"], out=s["out"])}
    if op == "norm":
        return _norm(s)
    if op == "pack":
        return _pack(s["w"])
    return {"y": _f8(s) if op == "f8" else _ffn(s)}


def work(case):
    op = case["op"]
    if op == "norm":
        t, k = case["T"], case["K"]
        size = {"f32": 4, "bf16": 2, "none": 0}
        scales = 4 * t * -(-k // 128) if case["bits"] == "f8" else 8 * t
        return {"bytes": t * k * (size[case["x"]] + 2 * size[case["res"]] + 1) + 4 * k + scales, "flops": 8 * t * k}
    if op == "pack":
        n, k = case["N"], case["K"]
        return {"bytes": 5 * n * k + 4 * -(-n // 128) * -(-k // 128), "flops": 2 * n * k}
    if op == "f8":
        t, n, k = case["T"], case["N"], case["K"]
        kb = -(-k // 128)
        x = 2 * t * k if case["raw"] else t * k + 4 * t * kb
        return {"bytes": n * k + 4 * -(-n // 128) * kb + x + t * n * (4 if case["out"] == "f32" else 2), "flops": 2 * t * n * k}
    t, e, k, f, kk = (case[i] for i in ("T", "E", "k", "F", "K"))
    live = t * (1 - case["pad"])
    hit = e * (1 - (1 - k / e) ** live)       # experts with a row, were all equally likely
    x = t * kk * {"i8": 1, "bf16": 2, "f32": 4}[case["x"]] + (4 * t if case["x"] == "i8" else 0)
    logits = t * e * (4 if case["logits"] == "f32" else 2)
    return {"bytes": logits + x + hit * 3 * f * kk / 4 + 4 * t * kk, "flops": 6 * live * k * f * kk}


# ------------------------------------------------------------------ exact

def _exact_codes(x):
    """A row's int8 codes by the rule's two binary32 roundings, and its floored absmax, in binary64."""
    x = x.double()
    m = x.abs().amax(1).clamp_min(float(torch.tensor(EPS, dtype=torch.float32)))
    scale = (127 / m).float().double()
    return torch.round((x * scale[:, None]).float()).double().clamp(-127, 127), m


def exact(case, seed):
    """The definitions in binary64: rows, blocks and experts one after the other, weights decoded bit by bit."""
    s, op = prepare(case, seed), case["op"]
    if op == "pack":
        n, k = case["N"], case["K"]
        m = torch.zeros(-(-n // 128), -(-k // 128), dtype=torch.float64, device="cuda")
        for i in range(m.shape[0]):
            most = s["w"][128 * i:128 * i + 128].abs().amax(0).double()
            for j in range(m.shape[1]):
                m[i, j] = most[128 * j:128 * j + 128].max()
        return {"q": None, "scale": torch.clamp_min(m, TINY) / TOP}
    if op == "norm":
        x = s["x"].double()
        total = x
        if s["res"] is not None:
            total = x + s["res"].double()
            x = total.float().to(s["res"].dtype).double() if case["res"] == "bf16" else total.float().double()
        hat = x * s["gain"].double() / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        out = {"q": None}
        if case["bits"] == "f8":
            out["scale"] = torch.stack([p.abs().amax(1).clamp_min(TINY) / TOP for p in hat.split(128, 1)])
        else:
            out["scale"], out["rowsum"] = hat.abs().amax(1), None
        return out if s["res"] is None else {"total": total, **out}
    if op == "f8":
        t, n, k = case["T"], case["N"], case["K"]
        x = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        for j in range(-(-k // 128)):
            at = slice(128 * j, 128 * j + 128)
            if case["raw"]:
                v = s["x"][:, at].double()
                m = v.abs().amax(1, keepdim=True).clamp_min(TINY)
                code = (v * (TOP / m).float().double()).float().to(torch.float8_e4m3fn)
                x[:, at] = code.double() * (m / TOP)
            else:
                x[:, at] = s["x"][:, at].double() * s["xs"][j].double()[:, None]
        y = torch.empty(t, n, dtype=torch.float64, device="cuda")
        for i in range(-(-n // 128)):
            w = s["w"][128 * i:128 * i + 128].double() * s["ws"][i].double().repeat_interleave(128)[:k]
            y[:, 128 * i:128 * i + 128] = x @ w.t()
        return {"y": y}
    t, k, f, kk = (case[i] for i in ("T", "k", "F", "K"))

    def matrix(rows, width):
        at = torch.arange(width, device="cuda")
        return ((rows[:, at // 16 * 4 + at % 4].int() >> (2 * (at % 16 // 4))) & 3).double() - 1

    floor = float(torch.tensor(EPS, dtype=torch.float32))
    if case["x"] == "i8":
        q, m = s["x"].double(), s["absmax"].double().clamp_min(floor)
    else:
        q, m = _exact_codes(s["x"])
    l = s["logits"].double()
    y = torch.zeros(t, kk, dtype=torch.float64, device="cuda")
    for i in range(t):
        left, best = l[i].clone(), l[i].max()
        if not bool(best > -INF):
            continue
        ids = []
        for _ in range(k):
            e = int(torch.nonzero(left == left.max())[0])      # the lowest of equal ones
            if not bool(left[e] > -INF):
                break
            ids.append(e)
            left[e] = -INF
        u = torch.exp(l[i] - best)
        u /= u[ids].sum() if case["share"] == "chosen" else u.sum()
        for e in ids:
            acc = matrix(s["gu"][e], kk) @ q[i]
            gate = (acc[0::2] * s["gate"][e].double() * m[i] / 127).float().clamp_min(0)
            up = (acc[1::2] * s["up"][e].double() * m[i] / 127).float()
            h = (gate * gate * up).bfloat16()      # as the definition rounds it: the codes below depend on its bits
            hq, hm = _exact_codes(h[None])
            y[i] += u[e] * (matrix(s["down"][e], f) @ hq[0]) * s["dg"][e].double() * hm[0] / 127
    return {"y": y}
