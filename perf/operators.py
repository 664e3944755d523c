"""The operators of a paged 4-bit KV cache: their cases, their plain forms and their 64-bit values.

plan   rz.paged_plan: request lengths -> page table, slot map, positions, row offsets.
heads  rz.qk_norm_rope: the norms of queries and keys for each head, their rotation, and the append of
       the new keys and values to the 4-bit cache, in one pass.
attend rz.attention_paged_q4: attention of each request's new tokens over its pages, read as they are held.

A page holds `page` tokens of every kv head; a record of 16 tokens of one kv head has 18 * hd bytes:
K codes | K scales | V codes | V scales (codes 4 bits, one f16 scale for 32 values: value = d * (code - 8)).
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a small batch: latency alone
        dict(name="plan 8 decodes", op="plan", n=8, ctx=4096, page=16, prompts=0, chunk=0, ended=0),
        # a full server: a thousand requests, prompts among them, some that end and return their pages
        dict(name="plan 1000 mixed", op="plan", n=1000, ctx=32768, page=16, prompts=37, chunk=777, ended=90),
        # Qwen2-0.5B-shaped heads, one token of one request
        dict(name="heads 1 x 14/2x64", op="heads", T=1, H=14, K=2, hd=64, page=16, mode=1, theta=1e6, norm=False, far=1000),
        # Llama-7B-shaped heads, one token of each of 33 requests
        dict(name="heads 33 x 32/32x128", op="heads", T=33, H=32, K=32, hd=128, page=16, mode=0, theta=1e4, norm=True, far=4096),
        # a prompt of an odd length, a head that is no power of two
        dict(name="heads 1999 x 12/4x96", op="heads", T=1999, H=12, K=4, hd=96, page=32, mode=0, theta=1e4, norm=True, far=60000),
        # a prompt chunk with shared kv heads, far into a long context
        dict(name="heads 4096 x 32/8x128", op="heads", T=4096, H=32, K=8, hd=128, page=64, mode=1, theta=1e6, norm=True, far=131072),
        # one token, a short context: latency alone
        dict(name="attend 1 at 1000, 14/2x64", op="attend", n=1, lo=1000, hi=1000, new=1, chunk=0, H=14, K=2, hd=64, page=16),
        # decode of a batch, a kv head for each head, ragged lengths
        dict(name="attend 16 to 4096, 32/32x128", op="attend", n=16, lo=130, hi=4096, new=1, chunk=0, H=32, K=32, hd=128, page=16),
        # decode of a large batch, shared kv heads, ragged lengths
        dict(name="attend 64 to 16384, 32/8x128", op="attend", n=64, lo=1000, hi=16384, new=1, chunk=0, H=32, K=8, hd=128, page=64),
        # one request with a very long context
        dict(name="attend 1 at 131071, 32/8x128", op="attend", n=1, lo=131071, hi=131071, new=1, chunk=0, H=32, K=8, hd=128, page=64),
        # five drafted tokens for each request are scored at once
        dict(name="attend 24 x 5 drafts, 14/2x64", op="attend", n=24, lo=70, hi=6000, new=5, chunk=0, H=14, K=2, hd=64, page=32),
        # a prompt chunk beside decodes
        dict(name="attend 8 with a chunk of 1000", op="attend", n=8, lo=200, hi=4001, new=1, chunk=1000, H=32, K=8, hd=128, page=64),
    ]


HEADS = [(14, 2, 64), (32, 32, 128), (32, 8, 128), (40, 40, 64), (32, 4, 64), (12, 4, 96), (8, 2, 256), (16, 1, 128)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "heads", "heads", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64])
    if op == "plan":
        n = _log(rng, 1, 1000)
        prompts = rng.randint(0, n // 8)
        return dict(op=op, n=n, ctx=_log(rng, 200, 32768), page=page, prompts=prompts, chunk=_log(rng, 20, 777) if prompts else 0,
                    ended=rng.randint(0, (n - prompts) // 8))
    H, K, hd = rng.choice(HEADS)
    if op == "heads":
        T = _log(rng, 1, min(4096, 4096 * 6144 // ((H + 2 * K) * hd)))
        return dict(op=op, T=T, H=H, K=K, hd=hd, page=page, mode=rng.randint(0, 1), theta=rng.choice([1e4, 1e6]), norm=rng.random() < 0.7,
                    far=_log(rng, max(T, 100), 131072))
    kind = rng.choice(["decode", "decode", "drafts", "chunk"])
    n = _log(rng, 1, 64)
    most = max(64, min(131072, 300000 * 1024 // (n * K * hd)))  # the keys and values of all requests stay within the largest case's
    hi = _log(rng, 20, most if n <= 2 else min(most, 20000))
    new, chunk = 1, 0
    if kind == "drafts":
        new = rng.randint(2, 9)
    elif kind == "chunk":
        hi = min(hi, 8000)
        chunk = _log(rng, 10, max(10, min(1000, hi, 3000000000 // (H * hd * hi) * 4)))
    return dict(op=op, n=n, lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi, new=new, chunk=chunk, H=H, K=K, hd=hd, page=page)


def _lengths(c):
    """(keys held, new tokens) of each request of an attend case, the new ones counted among the held."""
    r = random.Random(c["n"] * 7919 + c["hi"] * 31 + c["new"])
    held = [c["hi"]] + [_log(r, c["lo"], c["hi"]) for _ in range(c["n"] - 1)]
    new = [min(c["new"], h) for h in held]
    if c["chunk"]:
        new[0] = min(c["chunk"], held[0])
    return held, new


def _requests(c):
    """(cached, new) of each request of a plan case; new < 0: the request has ended."""
    r = random.Random(c["n"] * 104729 + c["ctx"] * 13 + c["chunk"])
    n, p, e = c["n"], c["prompts"], c["ended"]
    kind = ["prompt"] * p + ["ended"] * e + ["decode"] * (n - p - e)
    r.shuffle(kind)
    cached = [_log(r, 1, c["ctx"]) if k != "prompt" else r.choice([0, _log(r, 1, c["ctx"])]) for k in kind]
    new = [-1 if k == "ended" else 1 if k == "decode" else _log(r, 1, c["chunk"]) for k in kind]
    return cached, new


def work(c):
    if c["op"] == "plan":
        cached, new = _requests(c)
        rows = sum(max(0, x) for x in new)
        pages = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(cached, new) if b >= 0)
        back = sum(-(-a // c["page"]) for a, b in zip(cached, new) if b < 0)
        return {"bytes": c["n"] * 4 * 6 + rows * 16 + (pages + back) * 8, "flops": rows * 4 + c["n"] * 20}
    if c["op"] == "heads":
        q, kv = c["H"] * c["hd"], c["K"] * c["hd"]
        return {"bytes": c["T"] * ((q + 2 * kv) * 4 + (q + 2 * kv) * 4 + 2 * kv * 9 // 16 + 12), "flops": c["T"] * (q + kv) * 8 + c["T"] * kv * 2 * 6}
    held, new = _lengths(c)
    seen = sum(m * (h - m) + m * (m + 1) // 2 for h, m in zip(held, new))
    return {"bytes": sum(held) * c["K"] * c["hd"] * 9 // 8 + sum(-(-h // c["page"]) * 4 for h in held) + 2 * sum(new) * c["H"] * c["hd"] * 4,
            "flops": 4 * seen * c["H"] * c["hd"]}


# ---------------------------------------------------------------- the cache's layout, in plain torch
def _scales_codes(x):
    """x [..., hd] in any float type -> (f16 scales [..., hd/32], codes 0..15 uint8 [..., hd/32, 32])."""
    x = x.unflatten(-1, (-1, 32))
    top, low = x.amax(-1), x.amin(-1)
    d = (torch.where(top >= -low, top, low) / -8).float().clamp(-65504, 65504).half()
    d = torch.where(d == 0, torch.zeros_like(d), d)
    t = x / d.to(x.dtype).unsqueeze(-1)
    t = torch.where(d.unsqueeze(-1) == 0, torch.zeros_like(t), t)
    return d, (torch.round(t) + 8).clamp(0, 15).to(torch.uint8)


def _values(d, codes):
    return ((codes.float() - 8) * d.float().unsqueeze(-1)).flatten(-2)


def _word(nb):
    return 4 if nb % 2 == 0 else 2  # words of V codes that lie together


def _byte_places(hd):
    """Where byte i (low nibble value i, high value i + 16) of block b of a token lies: K [16, nb, 16], V [16, nb, 16], within a record."""
    nb = hd // 32
    tok, b, i = torch.meshgrid(torch.arange(16), torch.arange(nb), torch.arange(16), indexing="ij")
    k = tok * (hd // 2) + ((i // 4) * nb + b) * 4 + i % 4
    p, w = b * 16 + i, _word(nb)
    r, lane = p // 8, (p % 8) * 4 + tok // 4
    v = 9 * hd + ((r // w) * 32 + lane) * w * 4 + (r % w) * 4 + tok % 4
    return k.to(DEV), v.to(DEV)


def _pack_pages(x_k, x_v, page):
    """[pages, page, K, hd] twice -> uint8 [pages, K, page * hd * 9 / 8]."""
    P, _, K, hd = x_k.shape
    nb, rec = hd // 32, torch.empty(P, K, page // 16, 18 * hd, dtype=torch.uint8, device=x_k.device)
    for x, place, at in zip((x_k, x_v), _byte_places(hd), (8 * hd, 17 * hd)):
        d, c = _scales_codes(x.view(P, page // 16, 16, K, hd))
        c = c[..., :16] | (c[..., 16:] << 4)
        to = torch.empty(8 * hd, dtype=torch.int64, device=x.device)
        to[(place - place.min()).flatten()] = torch.arange(8 * hd, device=x.device)
        rec[..., place.min():place.min() + 8 * hd] = c.permute(0, 3, 1, 2, 4, 5).reshape(P, K, page // 16, -1)[..., to]
        rec[..., at:at + hd] = d.permute(0, 3, 1, 2, 4).contiguous().view(torch.uint8).reshape(P, K, page // 16, hd)
    return rec.view(P, K, -1)


def _unpack(rec, hd):
    """uint8 [..., 18 * hd] -> K and V in 32 bits, [..., 16, hd] each."""
    nb, lead = hd // 32, rec.shape[:-1]
    w = _word(nb)
    k = rec[..., :8 * hd].unflatten(-1, (16, 4, nb, 4)).movedim(-2, -3)  # token, block, 4 words, 4 bytes
    k = torch.cat([k & 15, k >> 4], -2).reshape(*lead, 16, nb, 32)
    v = rec[..., 9 * hd:17 * hd].unflatten(-1, (2 * nb // w, 8, 4, w, 4))  # r / w, p % 8, token / 4, r % w, token % 4
    d = len(lead)
    v = v.permute(*range(d), d + 2, d + 4, d, d + 3, d + 1).reshape(*lead, 16, nb, 16)
    v = torch.cat([v & 15, v >> 4], -1)
    s = [rec[..., a:a + hd].contiguous().view(torch.float16).unflatten(-1, (16, nb)) for a in (8 * hd, 17 * hd)]
    return _values(s[0], k), _values(s[1], v)


# ---------------------------------------------------------------- states
def _ints(v, t=torch.int32):
    return torch.tensor(v, dtype=t, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": c}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    if c["op"] == "plan":
        cached, new = _requests(c)
        page, n = c["page"], c["n"]
        r = random.Random(seed)  # the pages that requests hold and a request's length within its last page differ by seed
        pages = sum(-(-a // page) for a in cached) + sum(-(-max(0, m) // page) + 1 for m in new) + 5
        cached = [max(1, a - r.randint(0, 15)) if a else 0 for a in cached]
        owned = [-(-a // page) for a in cached]
        blocks = -(-(c["ctx"] + max(1, c["chunk"])) // page)
        order = torch.randperm(pages, generator=g, device=DEV).int()
        table = torch.full((n, blocks), -1, dtype=torch.int32, device=DEV)
        own_t = _ints(owned)
        at = torch.cumsum(own_t, 0) - own_t
        j = torch.arange(blocks, device=DEV)
        has = j < own_t[:, None]
        table[has] = order[(at[:, None] + j)[has]]
        free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        left = pages - sum(owned)
        free[:left] = order[sum(owned):]
        rows = sum(max(0, m) for m in new)
        s |= dict(cached=_ints(cached), new=_ints(new), table=table, owned=own_t, free=free, count=_ints([left]), rows=rows + 7,
                  owned_out=torch.empty_like(own_t), count_out=_ints([0]))
        if own:
            import quantized_q4_q8_gb300 as rz
            s["out"] = rz.PagedPlan(n, s["rows"], DEV)
        return s
    H, K, hd, page = c["H"], c["K"], c["hd"], c["page"]
    if c["op"] == "heads":
        T = c["T"]
        qkv = normal(T, (H + 2 * K) * hd)
        pages = -(-T // page) + 3
        first = int(torch.randint(0, c["far"] - min(T, c["far"]) + 1, (1,), generator=g, device=DEV))
        pos = (first + torch.arange(T, device=DEV)).int() % c["far"]
        slots = torch.randperm(pages, generator=g, device=DEV)[torch.arange(T, device=DEV) // page] * page + torch.arange(T, device=DEV) % page
        s |= dict(q=qkv[:, :H * hd], k=qkv[:, H * hd:(H + K) * hd], v=qkv[:, (H + K) * hd:], pos=pos, slots=slots,
                  gq=(0.5 + torch.rand(hd, generator=g, device=DEV)) if c["norm"] else None,
                  gk=(0.5 + torch.rand(hd, generator=g, device=DEV)) if c["norm"] else None,
                  cache=torch.zeros(pages, K, page * hd * 9 // 8, dtype=torch.uint8, device=DEV),
                  places=_byte_places(hd))
    else:
        held, new = _lengths(c)
        blocks = [-(-h // page) for h in held]
        pages = sum(blocks) + 2
        cache = _pack_pages(normal(pages, page, K, hd), normal(pages, page, K, hd), page)
        order = torch.randperm(pages, generator=g, device=DEV).int()
        table = torch.full((c["n"], max(blocks)), -1, dtype=torch.int32, device=DEV)
        b = _ints(blocks)
        j = torch.arange(max(blocks), device=DEV)
        has = j < b[:, None]
        table[has] = order[((torch.cumsum(b, 0) - b)[:, None] + j)[has]]
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        s |= dict(q=2 * normal(cu[-1], H * hd), cache=cache, table=table, held=_ints(held), cu=_ints(cu), longest=max(held), most=max(new),
                  seq=torch.repeat_interleave(torch.arange(c["n"], device=DEV), _ints(new)))
    if own:
        import quantized_q4_q8_gb300 as rz
        s["kv"] = rz.PagedKVQ4(s["cache"], page, hd)
        if c["op"] == "attend":
            s["ws"] = rz.workspace(rz.attention_paged_q4_workspace_bytes(H, K, hd), DEV)
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    return {"plan": _plan, "heads": _heads, "attend": _attend}[s["c"]["op"]](s)


def _plan(s):
    c = s["c"]
    page = c["page"]
    if own:
        import quantized_q4_q8_gb300 as rz
        p = rz.paged_plan(s["cached"], s["new"], s["table"], s["owned"], s["free"], s["count"], page, s["out"], owned_out=s["owned_out"],
                          free_count_out=s["count_out"])
        return {"cu": p.cu_rows, "len": p.kv_len, "seq": p.row_seq, "pos": p.positions, "slot": p.slots, "table": s["table"], "owned": s["owned_out"],
                "free": s["free"], "count": s["count_out"]}
    cached, new, owned, table, free = s["cached"].long(), s["new"].long(), s["owned"].long(), s["table"], s["free"]
    ended = new < 0
    m = new.clamp(min=0)
    # the pages of ended requests go back on top of the free ones
    back = torch.where(ended, owned, 0)
    back_at = torch.cumsum(back, 0) - back
    j = torch.arange(table.shape[1], device=DEV)
    gives = ended[:, None] & (j < owned[:, None])
    place = torch.where(gives, s["count"].long() + back_at[:, None] + j, free.numel())
    pool = torch.cat([free, free[:1]]).scatter(0, place.flatten(), table.flatten())[:-1]
    total = s["count"].long() + back.sum()
    # new pages are taken from the top, in order
    need = torch.where(ended, 0, (-(-(cached + m) // page) - owned).clamp(min=0))
    upto = torch.cumsum(need, 0)
    served = ~ended & ((need == 0) | (upto <= total))
    takes = served[:, None] & (j >= owned[:, None]) & (j < (owned + need)[:, None])
    number = (upto - need)[:, None] + j - owned[:, None]
    free.copy_(pool)
    table.copy_(torch.where(takes, pool[(total - 1 - number).clamp(0, pool.numel() - 1)], table))
    s["owned_out"].copy_(torch.where(ended, 0, torch.where(served, owned + need, owned)))
    s["count_out"].copy_(total - torch.where(served, need, 0).sum())
    cu = torch.cat([m.new_zeros(1), torch.cumsum(m, 0)])
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True).clamp(max=c["n"] - 1)
    real = row < cu[-1]
    pos = cached[seq] + row - cu[seq]
    put = real & served[seq]
    slot = table[seq, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    return {"cu": cu.int(), "len": torch.where(served, cached + m, 0).int(), "seq": torch.where(real, seq, -1).int(), "pos": torch.where(put, pos, -1).int(),
            "slot": torch.where(put, slot, -1), "table": table, "owned": s["owned_out"], "free": free, "count": s["count_out"]}


def _norm_rotate(x, gamma, pos, c):
    """x [T, heads, hd] -> normed and rotated, in x's type; the angles in 64 bits."""
    hd = c["hd"]
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma.to(x.dtype)
    f = torch.tensor(c["theta"], dtype=torch.float64, device=DEV) ** (-torch.arange(0, hd, 2, dtype=torch.float64, device=DEV) / hd)
    a = pos.double()[:, None, None] * f
    cos, sin = torch.cos(a).to(x.dtype), torch.sin(a).to(x.dtype)
    if c["mode"] == 0:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)
    x0, x1 = x[..., :hd // 2], x[..., hd // 2:]
    return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)


def _heads(s):
    c = s["c"]
    T, H, K, hd, page = c["T"], c["H"], c["K"], c["hd"], c["page"]
    if own:
        import quantized_q4_q8_gb300 as rz
        q, k, v = rz.qk_norm_rope(s["q"], s["k"], s["v"], s["pos"], H, K, hd, c["theta"], c["mode"], q_gamma=s["gq"], k_gamma=s["gk"], eps=1e-6,
                                  kv=s["kv"], slots=s["slots"], want_k=True, want_v=True)
        return {"q": q, "k": k, "v": v, "cache": s["cache"]}
    q = _norm_rotate(s["q"].view(T, H, hd), s["gq"], s["pos"], c)
    # the keys in 64 bits: some lie next to the border of two codes
    k = _norm_rotate(s["k"].reshape(T, K, hd).double(), s["gk"], s["pos"], c)
    cache, out = s["cache"].view(-1), []
    tok = s["slots"] % 16
    rec = ((s["slots"] // page)[:, None] * K + torch.arange(K, device=DEV)) * (page // 16) + (s["slots"] % page // 16)[:, None]
    for x, place, at in ((k, s["places"][0], 8 * hd), (s["v"].reshape(T, K, hd).double(), s["places"][1], 17 * hd)):
        d, codes = _scales_codes(x)
        cache[rec[:, :, None, None] * (18 * hd) + place[tok][:, None]] = codes[..., :16] | (codes[..., 16:] << 4)
        nb2 = hd // 16
        cache[rec[:, :, None] * (18 * hd) + at + (tok * nb2)[:, None, None] + torch.arange(nb2, device=DEV)] = d.view(torch.uint8).view(T, K, nb2)
        out.append(_values(d, codes).view(T, K * hd))
    return {"q": q.view(T, H * hd), "k": out[0], "v": out[1], "cache": s["cache"]}


def _attend(s):
    c = s["c"]
    H, K, hd, page = c["H"], c["K"], c["hd"], c["page"]
    if own:
        import quantized_q4_q8_gb300 as rz
        return rz.attention_paged_q4(s["q"], s["kv"], s["table"], s["cu"], s["held"], H, ws=s["ws"])
    n, most, L = c["n"], s["most"], s["table"].shape[1] * page
    rec = s["cache"].view(-1, K, page // 16, 18 * hd)[s["table"].long().clamp(min=0)]  # [n, blocks, K, page / 16, bytes]
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(n, K, L, hd) for x in _unpack(rec, hd))
    cu, held = s["cu"].long(), s["held"].long()
    m = cu[1:] - cu[:-1]
    i = torch.arange(most, device=DEV)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].view(n, most, K, H // K, hd).permute(0, 2, 1, 3, 4).reshape(n, K, most * (H // K), hd)
    p = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(hd)
    sees = (held - m)[:, None] + i + 1  # the keys that new token i sees
    mask = (torch.arange(L, device=DEV) < sees[..., None]).repeat_interleave(H // K, 1)[:, None]
    p = p.masked_fill(~mask, -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
    z = p.sum(-1, keepdim=True)
    # values of keys that none sees count for nothing, whatever the page holds
    v = torch.where((torch.arange(L, device=DEV) < held[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v) / torch.where(z == 0, torch.ones_like(z), z)
    o = o.view(n, K, most, H // K, hd).permute(0, 2, 1, 3, 4).reshape(n, most, H * hd)
    return o[s["seq"], torch.arange(s["q"].shape[0], device=DEV) - cu[s["seq"]]]


# ---------------------------------------------------------------- in 64 bits, from the definitions
def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers all
    s = prepare(c, seed)
    H, K, hd, page = c["H"], c["K"], c["hd"], c["page"]
    if c["op"] == "heads":
        T, half = c["T"], hd // 2
        # the rotation as a product of complex numbers
        turn = np.multiply.outer(s["pos"].cpu().numpy().astype(np.float64), np.power(float(c["theta"]), -2.0 * np.arange(half) / hd))
        turn = torch.polar(torch.ones(T, half, dtype=torch.float64), torch.from_numpy(turn)).to(DEV)[:, None]

        def rotated(x, gamma):
            x = x.double().reshape(T, -1, hd)
            if gamma is not None:
                x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / hd + 1e-6) * gamma.double()
            z = (torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) if c["mode"] == 0
                 else torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())) * turn
            return (torch.view_as_real(z).reshape(T, -1) if c["mode"] == 0 else torch.cat([z.real, z.imag], -1).reshape(T, -1))

        def held4(x):
            x = x.double().reshape(T, -1, 32)
            i = x.abs().argmax(-1, keepdim=True)
            peak = x.gather(-1, i)
            flip = ((x == peak.abs()).any(-1, keepdim=True)) & (peak < 0)  # of two peaks of one size, the positive one
            d = (torch.where(flip, -peak, peak) * -0.125).float().half().double()
            code = torch.where(d == 0, torch.zeros_like(x), torch.round(x / torch.where(d == 0, torch.ones_like(d), d)))
            return (code.clamp(-8, 7) * d).reshape(T, -1)

        return {"q": rotated(s["q"], s["gq"]), "k": held4(rotated(s["k"], s["gk"])), "v": held4(s["v"]), "cache": None}
    held, new = _lengths(c)
    if sum(held) * H * hd * max(1, max(new) // 8) > 2e13:
        return None
    kp, vp = (x.flatten() for x in _byte_places(hd))
    sc = torch.arange(hd // 32, device=DEV) * 2
    flat, table, out, at, G = s["cache"].reshape(-1), s["table"].long(), [], 0, H // K
    for r, (n, m) in enumerate(zip(held, new)):
        t = torch.arange(n, device=DEV)
        rec = ((table[r, t // page][:, None] * K + torch.arange(K, device=DEV)) * (page // 16) + (t % page // 16)[:, None]) * (18 * hd)

        def read(places, scales):
            byte = flat[rec[:, :, None] + places.view(16, -1)[t % 16][:, None]].view(n, K, -1, 16)
            where = rec[:, :, None] + scales + (t % 16 * (hd // 16))[:, None, None] + sc
            bits = flat[where].int() | (flat[where + 1].int() << 8)
            d = bits.to(torch.int16).view(torch.float16).double()
            return (torch.cat([byte % 16, byte // 16], -1).double() - 8).mul(d[..., None]).reshape(n, K, hd)

        k, v = read(kp, 8 * hd), read(vp, 17 * hd)
        q = s["q"][at:at + m].double().view(m, K, G, hd)
        o = torch.empty(m, K, G, hd, dtype=torch.float64, device=DEV)
        hidden = t[None, None] > (n - m + torch.arange(m, device=DEV))[:, None, None]
        for h in range(K):
            w = torch.softmax((torch.einsum("mgd,td->mgt", q[:, h], k[:, h]) * hd ** -0.5).masked_fill(hidden, -math.inf), -1)
            o[:, h] = torch.einsum("mgt,td->mgd", w, v[:, h])
        out.append(o.view(m, H * hd))
        at += m
    return torch.cat(out)
