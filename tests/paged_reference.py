"""The paged 4-bit KV cache in numpy and f64, written from the format's definition in
include/rz.h: quantisation, record layout, page plan, norm and rotation, attention."""
import numpy as np


def quantise(x):
    """x f64 [..., hd] -> (f16 scales [..., nb], codes [..., nb, 32], values f32 [..., hd])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    hi, lo = b.max(-1), b.min(-1)
    with np.errstate(all="ignore"):
        s = np.where(hi >= -lo, hi, lo)
        d = np.clip((s / -8.0).astype(np.float32), -65504, 65504).astype(np.float16)
        d = np.where(d == 0, np.float16(0), d)
        fine = np.isfinite(b).all(-1)
        d = np.where(fine, d, np.float16(np.nan))
        t = b / d.astype(np.float64)[..., None]
    zero = (d == 0) | ~fine
    t = np.where(zero[..., None], 0.0, t)
    codes = np.clip(np.rint(t) + 8, 0, 15).astype(np.int64)
    v = (codes - 8).astype(np.float32) * d.astype(np.float32)[..., None]
    return d, codes, v.reshape(x.shape)


def k_place(nb, tok, b, i):
    return tok * 16 * nb + ((i // 4) * nb + b) * 4 + i % 4


def v_place(nb, tok, b, i):
    p, run = 16 * b + i, 4 if nb % 2 == 0 else 2
    r, lane = p // 8, (p % 8) * 4 + tok // 4
    return 9 * 32 * nb + ((r // run) * 32 + lane) * run * 4 + (r % run) * 4 + tok % 4


def record_of(page_size, n_kv_heads, hd, slot, head):
    """Byte offset of the record that holds a slot of one kv head."""
    page, inside = slot // page_size, slot % page_size
    return ((page * n_kv_heads + head) * (page_size // 16) + inside // 16) * 18 * hd


def store(cache, page_size, n_kv_heads, hd, slot, head, k, v):
    """(scales, codes) of one token's key and value into a flat uint8 cache."""
    nb, tok, at = hd // 32, slot % 16, record_of(page_size, n_kv_heads, hd, slot, head)
    for (d, codes), place, scales in ((k, k_place, 8 * hd), (v, v_place, 17 * hd)):
        for b in range(nb):
            for i in range(16):
                cache[at + place(nb, tok, b, i)] = codes[b, i] | (codes[b, i + 16] << 4)
        cache[at + scales + tok * nb * 2:at + scales + (tok + 1) * nb * 2] = np.ascontiguousarray(d).view(np.uint8)


def pack(k, v, page_size):
    """k, v f64 [slots, heads, hd] (slots: whole pages) -> (flat uint8 cache, f32 values of k and of v)."""
    n, heads, hd = k.shape
    nb = hd // 32
    out = np.zeros(n * heads * hd * 9 // 8, np.uint8).reshape(n // page_size, heads, page_size // 16, 18 * hd)
    vals = []
    tok, b, i = np.meshgrid(np.arange(16), np.arange(nb), np.arange(16), indexing="ij")
    for x, place, scales in ((k, k_place, 8 * hd), (v, v_place, 17 * hd)):
        d, c, val = quantise(x)
        byte = (c[..., :16] | (c[..., 16:] << 4)).astype(np.uint8)  # [slots, heads, nb, 16]
        byte = byte.reshape(n // page_size, page_size // 16, 16, heads, nb, 16).transpose(0, 3, 1, 2, 4, 5)
        out[..., place(nb, tok, b, i)] = byte
        d8 = np.ascontiguousarray(d.reshape(n // page_size, page_size // 16, 16, heads, nb).transpose(0, 3, 1, 2, 4)).view(np.uint8)
        out[..., scales:scales + hd] = d8.reshape(n // page_size, heads, page_size // 16, hd)
        vals.append(val)
    return out.reshape(-1), vals[0], vals[1]


def rotate(x, pos, theta, mode):
    """x f64 [n, heads, hd] rotated by pos [n]."""
    hd = x.shape[-1]
    ang = pos.astype(np.float64)[:, None] * np.power(float(theta), -2.0 * np.arange(hd // 2) / hd)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = np.empty_like(x)
    if mode == 0:
        a, b = x[..., 0::2], x[..., 1::2]
        y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        y[..., :hd // 2], y[..., hd // 2:] = a * c - b * s, a * s + b * c
    return y


def norm(x, gamma, eps):
    if gamma is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * gamma.astype(np.float64)


def plan(cached, fresh, owned, table, free, count, page, max_rows):
    """One step, request after request.  Returns a dict of the outputs and the new state."""
    n, max_blocks = table.shape
    table, free = table.copy(), free.copy()
    owned_out = owned.copy()
    total, bad = count, False
    for i in range(n):
        if fresh[i] < 0 and 0 <= owned[i] <= max_blocks:
            free[total:total + owned[i]] = table[i, :owned[i]]
            total += owned[i]
    cu, kv_len, seq, pos, slot = [0], np.zeros(n, np.int32), [], [], []
    wanted = taken = rows = 0
    refused = False
    for i in range(n):
        m = max(int(fresh[i]), 0)
        rows += m
        fits = rows <= max_rows
        ok = 0 <= owned[i] <= max_blocks and (cached[i] >= 0 or fresh[i] < 0) and (fits or m == 0)
        need = 0
        if fresh[i] < 0:
            owned_out[i] = 0
            bad |= not 0 <= owned[i] <= max_blocks
        else:
            if ok:
                blocks = -(-(int(cached[i]) + m) // page)
                ok = blocks <= max_blocks and cached[i] <= owned[i] * page
                need = max(0, blocks - int(owned[i])) if ok else 0
            bad |= not ok
            wanted += need
            served = ok and (need == 0 or wanted <= total)
            refused |= ok and not served
            if served:
                for b in range(need):
                    table[i, owned[i] + b] = free[total - 1 - taken]
                    taken += 1
                owned_out[i] += need
                kv_len[i] = cached[i] + m
            if fits:
                for r in range(m):
                    p = int(cached[i]) + r if served else -1
                    seq.append(i)
                    pos.append(p)
                    slot.append(int(table[i, p // page]) * page + p % page if served else -1)
        cu.append(len(seq))
    pad = [-1] * (max_rows - len(seq))
    return dict(cu_rows=np.array(cu), kv_len=kv_len, row_seq=np.array(seq + pad), positions=np.array(pos + pad),
                slots=np.array(slot + pad), table=table, owned=owned_out, free=free, count=total - taken, bad=bad, refused=refused)


def attention(q, k, v, sees, scale):
    """q f64 [rows, hd], k and v f64 [tokens, hd], sees [rows] -> (out [rows, hd], weights [rows, tokens])."""
    s = (q @ k.T) * scale
    hidden = np.arange(k.shape[0])[None] >= np.asarray(sees)[:, None]
    s = np.where(hidden, -np.inf, s)
    with np.errstate(all="ignore"):
        p = np.exp(s - np.where(np.isinf(s.max(-1, initial=-np.inf)), 0, s.max(-1, initial=-np.inf))[:, None])
        z = p.sum(-1, keepdims=True)
        p = np.where(z == 0, 0, p / np.where(z == 0, 1, z))
    return np.where(hidden, 0, p) @ v, p
