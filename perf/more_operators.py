"""The operators of an FFN of experts in Q4_K: their cases, their plain forms and their 64-bit values.

norm    rz.residual_rmsnorm: the residual's addition, the RMS norm of the sum, and its Q8_1 form, in one pass.
route   rz.moe_route: the top k of router logits, their softmax weights, and the rows grouped by expert.
gateup  rz.moe_swiglu: silu(gate) * up of each (token, expert) row, the products grouped by expert, Q4_K x Q8_1.
down    rz.moe_down: the product back of each row, grouped by expert, the weighted sum of a token's rows, the residual.

Q8_1 of m rows of n values: int8 codes [m][n], f32 scales [m][n / 32], f32 scale * sum of codes [m][n / 32].
Q4_K: 256 weights in 144 bytes, value = d * sc * code - dmin * m.
"""
import math

import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of one token, the hidden state padded as Qwen2-0.5B-shaped layers have it: latency alone
        dict(name="norm 1 x 896", op="norm", T=1, n=896, pad=1024, outlier=1.0),
        # a decode batch of an odd size
        dict(name="norm 33 x 2048", op="norm", T=33, n=2048, pad=2048, outlier=30.0),
        # a prompt, Llama-7B-shaped rows with an outlier channel
        dict(name="norm 4095 x 4096", op="norm", T=4095, n=4096, pad=4096, outlier=100.0),
        # one token: latency alone
        dict(name="route 1, 8 of 64", op="route", T=1, E=64, k=8, mode=1, idle=0.0, skew=0.5),
        # a prompt, some rows of the batch without a request
        dict(name="route 4095, 8 of 128", op="route", T=4095, E=128, k=8, mode=1, idle=0.1, skew=1.0),
        # decode of one token: the weights of the chosen experts are read once
        dict(name="gateup 1, 8 of 64, 2048>1024", op="gateup", T=1, E=64, k=8, n=2048, i=1024, idle=0.0, skew=0.5),
        # a decode batch on a few large experts: their weights, read once
        dict(name="gateup 16, 2 of 8, 4096>14336", op="gateup", T=16, E=8, k=2, n=4096, i=14336, idle=0.0, skew=0.5),
        # a large decode batch on many small experts, most with a few rows, some with none
        dict(name="gateup 129, 8 of 128, 2048>768", op="gateup", T=129, E=128, k=8, n=2048, i=768, idle=0.1, skew=1.0),
        # a prompt: compute
        dict(name="gateup 4096, 2 of 8, 4096>14336", op="gateup", T=4096, E=8, k=2, n=4096, i=14336, idle=0.0, skew=0.3),
        # decode of one token
        dict(name="down 1, 8 of 64, 1024>2048", op="down", T=1, E=64, k=8, n=2048, i=1024, idle=0.0, skew=0.5),
        # a decode batch of an odd size
        dict(name="down 65, 4 of 16, 4864>896", op="down", T=65, E=16, k=4, n=896, i=4864, idle=0.2, skew=1.0),
        # a prompt on many small experts
        dict(name="down 4095, 8 of 64, 1024>2048", op="down", T=4095, E=64, k=8, n=2048, i=1024, idle=0.0, skew=0.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "gateup", "gateup", "gateup", "down", "down", "down"])
    if op == "norm":
        n = _log(rng, 64, 8192)
        pad = -(-n // 256) * 256
        return dict(op=op, T=_log(rng, 1, 4095 * 4096 // pad), n=n, pad=pad, outlier=rng.choice([1.0, 10.0, 100.0]))
    E = rng.choice([4, 8, 16, 32, 64, 128])
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    idle, skew = rng.choice([0.0, 0.1, 0.5]), rng.choice([0.1, 0.5, 1.0])
    if op == "route":
        return dict(op=op, T=_log(rng, 1, 4095), E=E, k=k, mode=rng.randint(0, 1), idle=idle, skew=skew)
    # the weights of all experts stay below those of the largest listed case, and so do the products
    n = 256 * _log(rng, 1, 16)
    i = 256 * _log(rng, 1, max(1, min(56, 8 * 14336 * 4096 // (E * n * 256))))
    T = _log(rng, 1, min(4095, 4096 * 2 * 4096 * 14336 // (4 * k * n * i)))
    return dict(op=op, T=T, E=E, k=k, n=n, i=i, idle=idle, skew=skew)


def work(c):
    T = c["T"]
    if c["op"] == "norm":
        return {"bytes": T * c["n"] * 8 + c["n"] * 4 + T * c["pad"] * 37 // 4, "flops": T * c["n"] * 8}
    P, E = T * c["k"], c["E"]
    if c["op"] == "route":
        return {"bytes": T * E * 4 + P * 16 + E * 4, "flops": T * E * 8}
    met = E * (1 - (1 - c["k"] / E) ** T)  # experts that some row meets, were they all as likely
    mats = 2 if c["op"] == "gateup" else 1
    live = P * (1 - c["idle"])
    weights = met * mats * c["i"] * c["n"] * 144 / 256
    if c["op"] == "gateup":
        return {"bytes": weights + T * c["n"] * 5 / 4 + live * (c["i"] * 4 + 4), "flops": 4 * live * c["i"] * c["n"]}
    return {"bytes": weights + live * (c["i"] * 5 / 4 + 12) + T * c["n"] * 8, "flops": 2 * live * c["i"] * c["n"]}


# ---------------------------------------------------------------- Q8_1 and Q4_K in plain torch
def _q8_parts(y):
    """y f32 [m, n] -> int8 codes [m, n], f32 scales and scale * sum [m, n / 32]; halves go away from zero."""
    b = y.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1) / 127
    t = b / torch.where(d == 0, torch.ones_like(d), d).unsqueeze(-1)
    q = (torch.sign(t) * torch.floor(t.abs().double() + 0.5)).clamp(-127, 127).float()
    q = torch.where((d == 0).unsqueeze(-1), torch.zeros_like(q), q)
    return q.flatten(-2).to(torch.int8), d, d * q.sum(-1)


def _q8_buffer(q, d, s):
    return torch.cat([q.flatten().view(torch.uint8), d.flatten().view(torch.uint8), s.flatten().view(torch.uint8)])


def _q8_views(buf, m, n):
    a, b = m * n, m * n + m * n // 8
    return buf[:a].view(torch.int8).view(m, n), buf[a:b].view(torch.float32).view(m, -1), buf[b:b + m * n // 8].view(torch.float32).view(m, -1)


def _q8_values(buf, m, n, dtype=torch.float32):
    q, d, _ = _q8_views(buf, m, n)
    return (q.to(dtype).unflatten(-1, (-1, 32)) * d.to(dtype).unsqueeze(-1)).flatten(-2)


def _six(h):
    """The header's 12 bytes [..., 12] -> 8 scales and 8 mins of six bits each."""
    lo, mid, hi = h[..., 0:4], h[..., 4:8], h[..., 8:12]
    return (torch.cat([lo & 63, (hi & 15) | ((lo >> 6) << 4)], -1), torch.cat([mid & 63, (hi >> 4) | ((mid >> 6) << 4)], -1))


def _weights(w):
    """uint8 [..., blocks, 144] -> f32 [..., blocks * 256]."""
    dd = w[..., 0:4].contiguous().view(torch.float16).float()
    sc, m = _six(w[..., 4:16])
    qs = w[..., 16:144].unflatten(-1, (4, 32))
    q = torch.stack([qs & 15, qs >> 4], -2).flatten(-3, -2).float()  # [..., 8, 32]
    return ((dd[..., 0:1] * sc.float()).unsqueeze(-1) * q - (dd[..., 1:2] * m.float()).unsqueeze(-1)).flatten(-3)


# ---------------------------------------------------------------- states
def _routing(g, c):
    """Router logits of T tokens: some experts are met more often than others."""
    pop = c["skew"] * torch.randn(c["E"], generator=g, device=DEV)
    return torch.randn(c["T"], c["E"], generator=g, device=DEV) + pop


def _sequences(g, c):
    """The request of each row of the batch, -1 for a row without one."""
    idle = torch.rand(c["T"], generator=g, device=DEV) < c["idle"]
    return torch.where(idle, -1, torch.arange(c["T"], device=DEV)).int()


def _plan(logits, seq, k, mode):
    """experts, weights [T, k]; offsets [E + 1], rows [P] (token * k + choice, by expert), places [P] (of each pair among the rows)."""
    T, E = logits.shape
    order = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, :k]
    live = (seq >= 0).unsqueeze(-1)
    top = logits.gather(-1, order)
    p = torch.exp(top - logits.amax(-1, keepdim=True))
    z = p.sum(-1, keepdim=True) if mode else torch.exp(logits - logits.amax(-1, keepdim=True)).sum(-1, keepdim=True)
    weights = torch.where(live, p / z, torch.zeros_like(p))
    experts = torch.where(live, order, torch.full_like(order, -1))
    flat = torch.where(live, order, torch.full_like(order, E)).flatten()
    rows = torch.argsort(flat, stable=True)
    n = (flat.unsqueeze(0) == torch.arange(E, device=DEV).unsqueeze(1)).sum(-1)
    offsets = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    at = torch.arange(T * k, device=DEV)
    places = torch.empty_like(at).scatter(0, rows, at)
    places = torch.where(flat < E, places, torch.full_like(places, -1))
    rows = torch.where(at < offsets[-1], rows, torch.full_like(rows, -1))
    return {"experts": experts.int(), "weights": weights, "offsets": offsets.int(), "rows": rows.int(), "places": places.int()}


def _q4k(g, *shape, rows_in):
    """Q4_K weights around zero, of the size that keeps a row's products near 1: shape [..., rows, in]."""
    nb = rows_in // 256
    w = torch.randint(0, 256, (*shape, nb, 144), generator=g, device=DEV, dtype=torch.uint8)
    d = (0.5 + torch.rand(*shape, nb, generator=g, device=DEV)) / (200 * math.sqrt(rows_in))
    dmin = 7.5 * d
    w[..., 0:2] = d.half().unsqueeze(-1).view(torch.uint8)
    w[..., 2:4] = dmin.half().unsqueeze(-1).view(torch.uint8)
    w[..., 8:12] = w[..., 4:8]  # a block's min goes with its scale
    w[..., 12:16] = (w[..., 12:16] & 15) * 17
    return w


def _activations(g, m, n):
    x = torch.randn(m, n, generator=g, device=DEV)
    x[:, :: max(1, n // 7)] *= 20  # a few outlier channels
    return x


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": c}
    T = c["T"]
    if c["op"] == "norm":
        x = torch.randn(T, c["pad"], generator=g, device=DEV)
        x[:, c["n"] // 3] *= c["outlier"]
        x[:, c["n"]:] = 0
        delta = 0.3 * torch.randn(T, c["pad"], generator=g, device=DEV)
        delta[:, c["n"]:] = 0
        s |= dict(x=x, delta=delta, gamma=0.5 + torch.rand(c["n"], generator=g, device=DEV))
        return s
    logits, seq = _routing(g, c), _sequences(g, c)
    k, E, P = c["k"], c["E"], T * c["k"]
    s |= dict(seq=seq)
    if c["op"] == "route":
        s |= dict(logits=logits)
        if own:
            import quantized_q4_q8_gb300 as rz
            s["plan"] = rz.MoePlan(T, E, k, DEV)
        return s
    plan = _plan(logits, seq, k, 1)
    n, i = c["n"], c["i"]
    n_in = -(-n // 256) * 256
    s |= dict(plan=plan, most=int((plan["offsets"][1:] - plan["offsets"][:-1]).max()))
    if c["op"] == "gateup":
        s |= dict(gate=_q4k(g, E, i, rows_in=n_in), up=_q4k(g, E, i, rows_in=n_in), x=_q8_buffer(*_q8_parts(_activations(g, T, n_in))),
                  h=torch.zeros(P, i, device=DEV))
    else:
        s |= dict(down=_q4k(g, E, n, rows_in=i), h=_q8_buffer(*_q8_parts(_activations(g, P, i))), res=torch.randn(T, n, generator=g, device=DEV))
    if own:
        import quantized_q4_q8_gb300 as rz
        s["own_plan"] = rz.MoePlan(T, E, k, DEV, **plan)
        if c["op"] == "gateup":
            s["ws"] = rz.workspace(rz.moe_swiglu_workspace_bytes(T, E, k, n), DEV)
        else:
            s["ws"] = rz.workspace(rz.moe_down_workspace_bytes(T, E, k, n, i), DEV)
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    return {"norm": _norm, "route": _route, "gateup": _gateup, "down": _down}[s["c"]["op"]](s)


def _norm(s):
    c = s["c"]
    if own:
        import quantized_q4_q8_gb300 as rz
        total, y, q8 = rz.residual_rmsnorm(s["x"], s["delta"], s["gamma"], c["n"], c["pad"], 1e-6)
        q, d, qs = _q8_views(q8, c["T"], c["pad"])
        return {"sum": total, "y": y, "codes": q, "scales": d, "sums": qs}
    total = s["x"] + s["delta"]
    live = total[:, :c["n"]].double()  # in 64 bits: some values lie next to the border of two codes
    y = torch.zeros_like(total)
    y[:, :c["n"]] = (live / torch.sqrt((live * live).mean(-1, keepdim=True) + 1e-6) * s["gamma"].double()).float()
    q, d, qs = _q8_parts(y)
    return {"sum": total, "y": y, "codes": q, "scales": d, "sums": qs}


def _route(s):
    c = s["c"]
    if own:
        import quantized_q4_q8_gb300 as rz
        p = rz.moe_route(s["logits"], s["plan"], renormalise=bool(c["mode"]), row_seq=s["seq"])
        return {"experts": p.experts, "weights": p.weights, "offsets": p.offsets, "rows": p.rows, "places": p.places}
    return _plan(s["logits"], s["seq"], c["k"], c["mode"])


def _grouped(s, w, x_of):
    """w uint8 [E, rows, blocks, 144]; x_of(pairs) -> f32 [..., in]: the product of every (token, choice) row, in the order of the plan's rows.

    Few rows: each with its expert's weights; more: the experts' rows side by side, each expert's up to the most that one has."""
    p, c = s["plan"], s["c"]
    P, E = p["rows"].numel(), c["E"]
    off = p["offsets"].long()
    r = torch.arange(P, device=DEV)
    e = torch.searchsorted(off[1:], r, right=True).clamp(max=E - 1)
    real = (r < off[-1]).unsqueeze(-1)
    if P <= E // 2:
        x = x_of(p["rows"].long().clamp(min=0), r)
        return [torch.where(real, torch.matmul(_weights(m[e]), x.unsqueeze(-1)).squeeze(-1), 0.0) for m in w]
    at = (off[:-1].unsqueeze(-1) + torch.arange(max(1, s["most"]), device=DEV)).clamp(max=P - 1)  # [E, most]
    x = x_of(p["rows"].long()[at].clamp(min=0), at)
    place = (e, (r - off[e]).clamp(min=0, max=max(1, s["most"]) - 1))
    return [torch.where(real, torch.matmul(x, _weights(m).transpose(-1, -2))[place], 0.0) for m in w]


def _gateup(s):
    c = s["c"]
    T, k, i = c["T"], c["k"], c["i"]
    n = s["gate"].shape[-2] * 256
    if own:
        import quantized_q4_q8_gb300 as rz
        return rz.moe_swiglu(s["gate"], s["up"], s["x"], s["own_plan"], i, n, out=s["h"], ws=s["ws"])
    x = _q8_values(s["x"], T, n)
    gate, up = _grouped(s, (s["gate"], s["up"]), lambda pairs, places: x[pairs // k])
    return gate / (1 + torch.exp(-gate)) * up


def _down(s):
    c = s["c"]
    T, k, n, i = c["T"], c["k"], c["n"], c["i"]
    if own:
        import quantized_q4_q8_gb300 as rz
        return rz.moe_down(s["down"], s["h"], s["own_plan"], n, i, residual=s["res"], ws=s["ws"])
    h = _q8_values(s["h"], T * k, i)
    (o,) = _grouped(s, (s["down"],), lambda pairs, places: h[places])
    p = s["plan"]
    places = p["places"].long().view(T, k)
    o = torch.where((places >= 0).unsqueeze(-1), o[places.clamp(min=0)], 0.0)
    return s["res"] + (p["weights"].unsqueeze(-1) * o).sum(1)


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _code_value(w):
    """The weights of uint8 [rows, blocks, 144] in 64 bits, sub-block by sub-block."""
    b = w.long()
    half = w[..., :4].contiguous().view(torch.float16).double()
    parts = []
    for j in range(8):
        if j < 4:
            sc, m = b[..., 4 + j] % 64, b[..., 8 + j] % 64
        else:
            sc = b[..., 8 + j] % 16 + b[..., j] // 64 * 16
            m = b[..., 8 + j] // 16 + b[..., 4 + j] // 64 * 16
        q = b[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        q = (q // 16 if j % 2 else q % 16).double()
        parts.append(q * (half[..., 0] * sc).unsqueeze(-1) - (half[..., 1] * m).unsqueeze(-1))
    return torch.cat(parts, -1).flatten(-2)


def exact(c, seed):
    s = prepare(c, seed)
    T = c["T"]
    if c["op"] == "norm":
        v = s["x"].double() + s["delta"].double()
        v = v.float().double()  # the sum is held in 32 bits, and normed as it is held
        scale = torch.rsqrt(torch.linalg.vector_norm(v[:, :c["n"]], dim=-1, keepdim=True) ** 2 / c["n"] + 1e-6)
        y = torch.zeros_like(v)
        y[:, :c["n"]] = v[:, :c["n"]] * scale * s["gamma"].double()
        d = y.reshape(T, -1, 32).abs().max(-1).values / 127
        return {"sum": s["x"].double() + s["delta"].double(), "y": y, "codes": None, "scales": d, "sums": None}
    if c["op"] == "route":
        logits = s["logits"].double()
        idx = _plan(s["logits"], s["seq"], c["k"], c["mode"])["experts"].long()
        top = logits.gather(-1, idx.clamp(min=0))
        w = torch.softmax(top, -1) if c["mode"] else torch.softmax(logits, -1).gather(-1, idx.clamp(min=0))
        return {"experts": None, "weights": torch.where(idx >= 0, w, 0.0), "offsets": None, "rows": None, "places": None}
    p, k, E = s["plan"], c["k"], c["E"]
    off = p["offsets"].tolist()
    gateup = c["op"] == "gateup"
    n_in = s["gate"].shape[-2] * 256 if gateup else c["i"]
    held = _q8_values(s["x"] if gateup else s["h"], T if gateup else T * k, n_in, torch.float64)
    out = torch.zeros(T * k, c["i"] if gateup else c["n"], dtype=torch.float64, device=DEV)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if gateup:
            x = held[p["rows"][a:b].long() // k]
            gate, up = x @ _code_value(s["gate"][e]).T, x @ _code_value(s["up"][e]).T
            out[a:b] = gate * torch.sigmoid(gate) * up
        else:
            out[a:b] = held[a:b] @ _code_value(s["down"][e]).T
    if gateup:
        return out
    y = s["res"].double()
    for j in range(k):
        at = p["places"].view(T, k)[:, j].long()
        y += torch.where((at >= 0).unsqueeze(-1), out[at.clamp(min=0)] * p["weights"][:, j:j + 1].double(), 0.0)
    return y
