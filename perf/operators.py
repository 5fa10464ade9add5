"""Measured cases of the routed-expert and 4-bit operators.

The plain forms below compute in binary32 (binary64 where a rounding decides
an integer) with elementary torch operations; with ``own`` set, ``run`` calls
the package's entry points on the same tensors.

Operators (the case key ``op``):
  route    top-k routing of tokens to experts and the slot layout it gives
  gated    gate and up projections of the routed tokens, squared-ReLU gate
  down     the experts' down projection with the weighted sum over a token's
           experts (``combine``) or one output row per slot
  w4_pack  4-bit quantisation of a matrix with one scale per group of a row,
           returned as the values it stands for
  w4       product of int8 tokens with a 4-bit matrix with group scales
"""

import math

import torch

own = False

EPS = 1e-5          # floor of a token's absmax
INF = float("inf")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decoding session picks 8 of 64 experts
        {"name": "route_t1", "op": "route", "T": 1, "E": 64, "k": 8, "bf16": False, "share": "chosen", "pad": 0.0},
        # a prompt batch: 8192 tokens over 128 experts, some rows are padding
        {"name": "route_t8192", "op": "route", "T": 8192, "E": 128, "k": 8, "bf16": True, "share": "all", "pad": 0.03},
        # one decoded token: its 8 experts' gate and up matrices stream from memory
        {"name": "gated_t1", "op": "gated", "T": 1, "E": 64, "k": 8, "N": 1024, "K": 2560, "bf16": True, "pad": 0.0},
        # a ragged decode batch of 33 sessions: nearly every expert is hit, few rows each
        {"name": "gated_t33", "op": "gated", "T": 33, "E": 64, "k": 6, "N": 1000, "K": 2560, "bf16": True, "pad": 0.05},
        # a prompt of 2048 tokens: ragged products of some 256 rows per expert
        {"name": "gated_t2048", "op": "gated", "T": 2048, "E": 64, "k": 8, "N": 1024, "K": 2560, "bf16": True, "pad": 0.0},
        # the decoded token's way back: 8 experts' outputs weighted and summed
        {"name": "down_t1", "op": "down", "T": 1, "E": 64, "k": 8, "N": 2560, "K": 1024, "combine": True, "pad": 0.0},
        # the prompt's way back, some tokens routed nowhere
        {"name": "down_t2048", "op": "down", "T": 2048, "E": 64, "k": 8, "N": 2560, "K": 1024, "combine": True, "pad": 0.02},
        # a small projection packed with zero points, groups of 32
        {"name": "pack_640x2560_g32z", "op": "w4_pack", "N": 640, "K": 2560, "G": 32, "zeros": True},
        # a 70B-class matrix packed symmetrically, groups of 128
        {"name": "pack_8192x28672_g128", "op": "w4_pack", "N": 8192, "K": 28672, "G": 128, "zeros": False},
        # vocabulary projection of one decoded token
        {"name": "w4_t1_head", "op": "w4", "T": 1, "N": 128256, "K": 2560, "G": 128, "zeros": False},
        # a few sessions through a matrix with zero points and small groups
        {"name": "w4_t7_g32z", "op": "w4", "T": 7, "N": 2560, "K": 6912, "G": 32, "zeros": True},
        # a prompt of 2048 tokens
        {"name": "w4_t2048_g64", "op": "w4", "T": 2048, "N": 6912, "K": 2560, "G": 64, "zeros": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    c = _draw(rng)
    if c.get("T", 8) < 8 and "pad" in c:    # a masked row or two would leave a small case nothing to do
        c["pad"] = 0.0
    return c


def _draw(rng):
    op = rng.choice(["route", "gated", "gated", "down", "down", "w4_pack", "w4", "w4", "w4"])
    if op == "route":
        e = _spread(rng, 4, 256)
        return {"op": op, "T": _spread(rng, 1, 8192), "E": e, "k": rng.randint(1, min(8, e)), "bf16": rng.random() < 0.5,
                "share": rng.choice(["chosen", "all"]), "pad": rng.choice([0.0, 0.05, 0.3])}
    if op in ("gated", "down"):
        e = _spread(rng, 4, 128)
        c = {"op": op, "T": _spread(rng, 1, 2048), "E": e, "k": rng.randint(1, min(8, e)),
             "N": _spread(rng, 40, 2048 if op == "gated" else 4096), "K": rng.choice([16, 64, 64, 128]), "pad": rng.choice([0.0, 0.05, 0.3])}
        c["K"] *= _spread(rng, max(1, 256 // c["K"]), 4096 // c["K"])
        # no more products than the largest listed case has, no more weights than 256 M
        full = 2048 * 8 * 1024 * 2560 * (2 if op == "gated" else 1)
        c["T"] = max(1, min(c["T"], full // (c["k"] * c["N"] * c["K"] * (2 if op == "gated" else 1))))
        c["E"] = max(c["k"], min(e, (1 << 28) // (c["N"] * c["K"] * (2 if op == "gated" else 1))))
        if op == "gated":
            c["bf16"] = rng.random() < 0.7
        else:
            c["combine"] = rng.random() < 0.7
        return c
    g = rng.choice([32, 64, 128])
    k = g * _spread(rng, max(1, 256 // g), 8192 // g)
    zeros = rng.random() < 0.5
    if op == "w4_pack":
        return {"op": op, "N": _spread(rng, 16, 8192), "K": k, "G": g, "zeros": zeros}
    n = _spread(rng, 16, min(131072, 2560 * 131072 // k))
    t = _spread(rng, 1, max(1, min(2048, 2048 * 6912 * 2560 // (n * k))))
    return {"op": op, "T": t, "N": n, "K": k, "G": g, "zeros": zeros}


# ----------------------------------------------------------------- inputs

def _logits(case, g):
    # router scores of a trained gate: some experts are more popular than others
    t, e = case["T"], case["E"]
    x = torch.randn(t, e, generator=g, device="cuda") + 0.7 * torch.randn(1, e, generator=g, device="cuda")
    if case["pad"]:     # padded rows are masked to -inf throughout
        x[torch.rand(t, generator=g, device="cuda") < case["pad"]] = -INF
    return x.bfloat16() if case.get("bf16") and case["op"] == "route" else x


def _ternary(g, e, n, k):
    # packed codes 0, 1, 2 (for -1, 0, +1), about a third zeros as absmean ternarisation gives
    c = torch.randint(0, 3, (4, e, n, k // 4), generator=g, device="cuda", dtype=torch.uint8)
    return c[0] | (c[1] << 2) | (c[2] << 4) | (c[3] << 6)


def _gammas(g, e):
    return 0.016 * (0.5 + torch.rand(e, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "route":
        s["logits"] = _logits(case, g)
    elif op in ("gated", "down"):
        t, e, k, n, kk = (case[i] for i in ("T", "E", "k", "N", "K"))
        ids, weights, offsets, pairs, slots = _route(_logits(case, g), k, "chosen")
        s.update(ids=ids, weights=weights, offsets=offsets, pairs=pairs, slots=slots)
        if op == "gated":
            x = torch.randn(t, kk, generator=g, device="cuda")
            s["x"] = x.bfloat16() if case["bf16"] else x
            s["packed"] = _ternary(g, e, 2 * n, kk)      # rows 2i: gate, 2i + 1: up
            s["gate"], s["up"] = _gammas(g, e), _gammas(g, e)
            s["out"] = torch.zeros(t * k, n, dtype=torch.bfloat16, device="cuda")
        else:
            # the gated unit's output: squared ReLU leaves half of it zero
            r = torch.randn(t * k, kk, generator=g, device="cuda").clamp_min(0)
            s["x"] = (r * r * torch.randn(t * k, kk, generator=g, device="cuda")).bfloat16()
            s["packed"], s["gamma"] = _ternary(g, e, n, kk), _gammas(g, e)
            s["out"] = torch.zeros(t if case["combine"] else t * k, n, device="cuda")
    elif op == "w4_pack":
        s["w"] = 0.02 * torch.randn(case["N"], case["K"], generator=g, device="cuda")
        s["w"][:1] = 0      # a row of zeros, as an unused vocabulary entry has
    else:
        t, n, k, grp = (case[i] for i in ("T", "N", "K", "G"))
        # codes over whole blocks of 128; those past K are zero
        kp = -(-k // 128) * 128
        b = torch.randint(0, 256, (n, kp // 2), generator=g, device="cuda", dtype=torch.uint8)
        if kp > k:
            live = (torch.arange(kp, device="cuda") < k).view(kp // 128, 4, 4, 2, 4).permute(0, 2, 1, 3, 4)
            live = (live[..., 0, :] * 15 + live[..., 1, :] * 240).reshape(1, kp // 2).to(torch.uint8)
            b &= live
        s["packed"] = b
        s["scales"] = (0.004 * (0.5 + torch.rand(n, k // grp, generator=g, device="cuda"))).bfloat16()
        s["zeros"] = torch.randint(-4, 4, (n, k // grp), generator=g, device="cuda", dtype=torch.int8) if case["zeros"] else None
        s["xq"] = (torch.randn(t, k, generator=g, device="cuda") * 35).round().clamp(-127, 127).to(torch.int8)
        s["absmax"] = 1 + 3 * torch.rand(t, generator=g, device="cuda")
    return s


# ------------------------------------------------------------ plain forms

def _route(logits, k, share):
    v, idx = torch.sort(torch.nan_to_num(logits.float(), nan=-INF, posinf=INF, neginf=-INF), dim=1, descending=True, stable=True)
    top, ids = v[:, :k], idx[:, :k]
    taken = top > -INF
    m = v[:, :1]
    over = top if share == "chosen" else v
    total = torch.where(over > -INF, torch.where(over == m, 1.0, torch.exp(over - m)), 0.0).sum(1, keepdim=True)
    weights = torch.where(taken, torch.where(top == m, 1.0, torch.exp(top - m)) / total, 0.0)
    ids = torch.where(taken, ids, -1).int()
    e, p = logits.shape[1], ids.numel()
    key, order = torch.sort(torch.where(ids < 0, e, ids).flatten(), stable=True)
    offsets = torch.searchsorted(key, torch.arange(e + 1, device=key.device, dtype=key.dtype)).int()
    live = torch.arange(p, device=key.device) < offsets[-1]
    pairs = torch.where(live, order, -1).int()
    slots = torch.empty(p, dtype=torch.int64, device=key.device)
    slots[order] = torch.where(live, torch.arange(p, device=key.device), -1)
    return ids, weights, offsets, pairs, slots.int().view_as(ids)


def _quantised(x):
    """Codes of step A1 as binary32 values, and each row's absmax."""
    x = x.float()
    a = x.abs().amax(1)
    s = (127.0 / a.clamp_min(torch.tensor(EPS, device=a.device)).double()).float()
    return (x * s[:, None]).round().clamp(-127, 127), a


def _matrices(packed):
    """Ternary values, binary32, of packed rows (four codes per byte; weight 16g + 4j + i in bits 2j of byte i of word g)."""
    b = packed.view(*packed.shape[:-1], -1, 1, 4)
    j = 2 * torch.arange(4, device=b.device, dtype=torch.uint8).view(4, 1)
    return ((b >> j) & 3).float().flatten(-3) - 1


def _experts(rows, ids, offsets, live, packed):
    """Sums of every slot's row with its expert's matrix: [P, N]. `rows` [P, K] in slot order; `ids` the slots' experts."""
    p, e = rows.shape[0], packed.shape[0]
    if p <= e:          # few rows: each with a matrix of its own
        return torch.matmul(_matrices(packed[ids]), rows[:, :, None])[:, :, 0]
    count = offsets.diff()
    most = int(count.max())
    at = (offsets[:-1, None] + torch.arange(most, device=rows.device)).clamp_max(p - 1)     # [E, most]
    y = torch.matmul(rows[at], _matrices(packed).transpose(1, 2))                           # [E, most, N]
    within = torch.arange(p, device=rows.device) - offsets[ids]
    return y[ids, torch.where(live, within, 0)]


def _slots(s):
    """Of every slot: whether it is in use, its (token, rank) pair and its expert."""
    live = s["pairs"] >= 0
    pair = s["pairs"].long().clamp_min(0)
    return live, pair, torch.where(live, s["ids"].flatten()[pair], 0).long()


def _gated(s):
    live, pair, ids = _slots(s)
    q, a = _quantised(s["x"])
    token = pair // s["case"]["k"]
    acc = _experts(q[token], ids, s["offsets"], live, s["packed"])
    m = a[token].clamp_min(EPS)
    g = acc[:, 0::2] * (s["gate"][ids] * m / 127)[:, None]
    u = acc[:, 1::2] * (s["up"][ids] * m / 127)[:, None]
    r = g.clamp_min(0)
    h = (r * r * u).bfloat16()
    return torch.where(live[:, None], h, torch.zeros_like(h))


def _down(s):
    live, pair, ids = _slots(s)
    q, a = _quantised(s["x"])
    y = _experts(q, ids, s["offsets"], live, s["packed"]) * (s["gamma"][ids] * a.clamp_min(EPS) / 127)[:, None]
    if not s["case"]["combine"]:
        return torch.where(live[:, None], y, torch.zeros_like(y))
    slots = s["slots"].long()
    parts = torch.where((slots >= 0)[:, :, None], y[slots.clamp_min(0)], 0.0)
    return (s["weights"][:, :, None] * parts).sum(1)


def _w4_pack(w, grp, zeros):
    n, k = w.shape
    v = w.view(n, k // grp, grp)
    if zeros:
        lo, hi = v.amin(2).clamp_max(0), v.amax(2).clamp_min(0)
        s = ((hi - lo).double() / 15).float().bfloat16().float()
        d = torch.where(s > 0, s, 1.0).double()
        z = (-lo.double() / d).float().round().clamp(0, 15) - 8
        z = torch.where(s > 0, z, 0.0)
    else:
        s = (v.abs().amax(2).double() / 7).float().bfloat16().float()
        d = torch.where(s > 0, s, 1.0).double()
        z = torch.zeros_like(s)
    t = ((v.double() / d[:, :, None]).float().round() + z[:, :, None]).clamp(-8, 7)
    t = torch.where(s[:, :, None] > 0, t, z[:, :, None])
    return ((t - z[:, :, None]) * s[:, :, None]).view(n, k), s.bfloat16()


def _w4_values(packed, scales, zeros, k):
    """Binary32 values of a 4-bit matrix: in each block of 128, byte i of word j of 16-byte chunk q holds k = 32j + 8q + i (low four bits, two's complement) and 4 more (high)."""
    n, grp = packed.shape[0], k // scales.shape[1]
    b = packed.view(n, -1, 4, 4, 4)
    t = torch.stack((b & 15, b >> 4), 4).permute(0, 1, 3, 2, 4, 5).reshape(n, -1)[:, :k]
    t = ((t ^ 8).float() - 8).view(n, -1, grp)
    if zeros is not None:
        t = t - zeros[:, :, None].float()
    return (t * scales[:, :, None].float()).view(n, k)


def _w4(s):
    w = _w4_values(s["packed"], s["scales"], s["zeros"], s["case"]["K"])
    return torch.matmul(s["xq"].float(), w.t()) * (s["absmax"].clamp_min(EPS) / 127)[:, None]


# -------------------------------------------------------------------- run

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import bitlinear_w1_a8_amd as bl

        if op == "route":
            r = bl.route_experts(s["logits"], s["case"]["k"], share=s["case"]["share"])
            return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "pairs": r.pairs, "slots": r.slots}
        if op == "w4_pack":
            packed, scales, zeros = bl.pack_weights_w4(s["w"], s["case"]["G"], with_zeros=s["case"]["zeros"])
            return {"values": bl.unpack_weights_w4(packed, scales, zeros, s["case"]["K"]), "scales": scales}
        if op == "w4":
            return {"y": bl.forward_w4(s["packed"], s["scales"], s["xq"], s["absmax"], zeros=s["zeros"])}
        routing = bl.Routing(s["ids"], s["weights"], s["offsets"], s["pairs"], s["slots"])
        if op == "gated":
            return {"h": bl.gated_relu2_experts(s["x"], s["packed"], s["gate"], s["up"], routing, out=s["out"])[0]}
        return {"y": bl.linear_experts(s["x"], s["packed"], s["gamma"], routing, combine=s["case"]["combine"], out=s["out"])}
    if op == "route":
        return dict(zip(("ids", "weights", "offsets", "pairs", "slots"), _route(s["logits"], s["case"]["k"], s["case"]["share"])))
    if op == "w4_pack":
        return dict(zip(("values", "scales"), _w4_pack(s["w"], s["case"]["G"], s["case"]["zeros"])))
    if op == "w4":
        return {"y": _w4(s)}
    return {"h": _gated(s)} if op == "gated" else {"y": _down(s)}


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["T"], case["E"], case["k"]
        return {"bytes": t * e * (2 if case["bf16"] else 4) + 16 * t * k + 4 * (e + 1), "flops": 3 * t * e}
    if op in ("gated", "down"):
        t, e, k, n, kk = (case[i] for i in ("T", "E", "k", "N", "K"))
        p = t * k * (1 - case["pad"])
        hit = e * (1 - (1 - k / e) ** (t * (1 - case["pad"])))     # experts with a row, were all equally likely
        if op == "gated":
            return {"bytes": t * kk * (2 if case["bf16"] else 4) + hit * 2 * n * kk / 4 + 2 * p * n, "flops": 4 * p * n * kk}
        return {"bytes": 2 * p * kk + hit * n * kk / 4 + 4 * n * (t if case["combine"] else p), "flops": 2 * p * n * kk}
    n, k, g = case["N"], case["K"], case["G"]
    matrix = n * k / 2 + n * k / g * (3 if case["zeros"] else 2)
    if op == "w4_pack":     # the weights in, the packed matrix out and in again, its values out
        return {"bytes": 8 * n * k + 2 * matrix, "flops": 6 * n * k}
    t = case["T"]
    return {"bytes": matrix + t * k + 4 * t + 4 * t * n, "flops": 2 * t * n * k}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definitions in binary64; experts one after the other, weights decoded bit by bit."""
    s, op = prepare(case, seed), case["op"]
    if op == "w4_pack":
        return None      # whole codes and rounded scales: no other value than the rounded one
    if op == "route":
        l = s["logits"].double()
        l = torch.where(torch.isnan(l), torch.full_like(l, -INF), l)
        best = l.amax(1, keepdim=True)
        u = torch.where(l > -INF, torch.exp(l - torch.where(best > -INF, best, 0.0)), 0.0)
        # rank of an entry: how many come before it (larger, or equal at a lower place)
        w = torch.zeros(case["T"], case["k"], dtype=torch.float64, device="cuda")
        left, rows = l.clone(), torch.arange(case["T"], device="cuda")
        for j in range(case["k"]):
            top = left.argmax(1)
            w[:, j] = torch.where(left[rows, top] > -INF, u[rows, top], 0.0)
            left[rows, top] = -INF
        total = (w if case["share"] == "chosen" else u).sum(1, keepdim=True)
        return {"ids": None, "weights": torch.where(total > 0, w / total.clamp_min(1e-300), 0.0), "offsets": None, "pairs": None, "slots": None}
    if op == "w4":
        n, k, grp = case["N"], case["K"], case["G"]
        y = torch.zeros(case["T"], n, dtype=torch.float64, device="cuda")
        kk = torch.arange(k, device="cuda")
        word = kk % 128 % 32                                  # place within a group of 32: chunk, half, byte
        byte = kk // 128 * 64 + word // 8 * 16 + kk % 128 // 32 * 4 + word % 4
        shift = (word % 8 // 4 * 4)
        step = max(1, (1 << 27) // k)
        for r in range(0, n, step):
            c = (s["packed"][r:r + step, byte].int() >> shift) & 15
            w = torch.where(c > 7, c - 16, c).double()
            if s["zeros"] is not None:
                w -= s["zeros"][r:r + step].double().repeat_interleave(grp, 1)
            w *= s["scales"][r:r + step].double().repeat_interleave(grp, 1)
            y[:, r:r + step] = s["xq"].double() @ w.t()
        return {"y": y * s["absmax"].double().clamp_min(EPS)[:, None] / 127}
    # the A1 codes, by the rule's two binary32 roundings
    x = s["x"].double()
    a = x.abs().amax(1)
    eps = torch.tensor(EPS, device="cuda").double()
    scale = (127 / a.clamp_min(eps)).float()
    q = torch.round((x * scale.double()[:, None]).float()).double().clamp(-127, 127)
    k, kk = case["k"], case["K"]
    at = torch.arange(kk, device="cuda")
    byte, shift = at // 16 * 4 + at % 4, 2 * (at % 16 // 4)
    out = torch.zeros(case["T"] * k, case["N"], dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for e in range(case["E"]):
        mine = torch.arange(ends[e], ends[e + 1], device="cuda")
        if not len(mine):
            continue
        w = ((s["packed"][e][:, byte].int() >> shift) & 3).double() - 1
        rows = s["pairs"][mine].long() // k if op == "gated" else mine
        acc = q[rows] @ w.t() * a[rows].clamp_min(eps)[:, None] / 127
        if op == "gated":
            gate, up = acc[:, 0::2] * s["gate"][e].double(), acc[:, 1::2] * s["up"][e].double()
            out[mine] = gate.clamp_min(0) ** 2 * up
        else:
            out[mine] = acc * s["gamma"][e].double()
    if op == "gated":
        return {"h": out}
    if not case["combine"]:
        return {"y": out}
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
    for j in range(k):
        p = s["slots"][:, j].long()
        y += torch.where((p >= 0)[:, None], s["weights"][:, j, None].double() * out[p.clamp_min(0)], 0.0)
    return {"y": y}
