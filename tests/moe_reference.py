"""Plain numpy forms, in 64 bits, of the operators of an FFN of experts."""
import numpy as np


def q8_quantize(y, multiplied=False):
    """y f32 [m, n] -> int8 codes, f32 scales, f32 scale * sum: the format's definition, step by step in f32.  multiplied: the
    scale is max|y| * (1 / 127), as rz_residual_rmsnorm has it."""
    b = y.astype(np.float32).reshape(y.shape[0], y.shape[1] // 32, 32)
    top = np.abs(b).max(-1)
    d = top * (np.float32(1) / np.float32(127)) if multiplied else top / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(d[..., None] == 0, np.float32(0), b / d[..., None])
    q = np.clip(np.sign(t) * np.floor(np.abs(t).astype(np.float64) + 0.5), -127, 127).astype(np.int32)
    return q.reshape(y.shape).astype(np.int8), d, (d * q.sum(-1).astype(np.float32)).astype(np.float32)


def q8_buffer(q, d, s):
    return np.concatenate([q.reshape(-1).view(np.uint8), np.ascontiguousarray(d, np.float32).reshape(-1).view(np.uint8),
                           np.ascontiguousarray(s, np.float32).reshape(-1).view(np.uint8)])


def q8_parts(buf, m, n):
    nb = n // 32
    q = buf[:m * n].view(np.int8).reshape(m, n)
    d = buf[m * n:m * n + 4 * m * nb].view(np.float32).reshape(m, nb)
    s = buf[m * n + 4 * m * nb:].view(np.float32).reshape(m, nb)
    return q, d, s


def q8_values(q, d):
    return (q.astype(np.float64).reshape(*d.shape, 32) * d.astype(np.float64)[..., None]).reshape(q.shape)


def weights(w):
    """uint8 [..., blocks, 144] -> (values, |d sc code| + |dmin m|), f64 [..., blocks * 256]."""
    d = w[..., 0:2].copy().view(np.float16).astype(np.float64)
    dmin = w[..., 2:4].copy().view(np.float16).astype(np.float64)
    b = w.astype(np.int64)
    val, size = [], []
    for j in range(8):
        if j < 4:
            sc, mn = b[..., 4 + j] & 63, b[..., 8 + j] & 63
        else:
            sc = (b[..., 8 + j] & 15) | ((b[..., j] >> 6) << 4)
            mn = (b[..., 8 + j] >> 4) | ((b[..., 4 + j] >> 6) << 4)
        qs = b[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        q = (qs >> 4) if j & 1 else (qs & 15)
        up, down = d * sc[..., None] * q, dmin * mn[..., None]
        val.append(up - down)
        size.append(np.abs(up) + np.abs(down))
    return tuple(np.concatenate(p, -1).reshape(*w.shape[:-2], -1) for p in (val, size))


def route(logits, k, renormalise, scale=1.0, row_seq=None):
    """experts, weights, offsets, rows, places as rz.h has them; weights in 64 bits."""
    T, E = logits.shape
    experts, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        if row_seq is not None and row_seq[t] < 0:
            continue
        v = logits[t].astype(np.float64)
        key = [(1 if np.isnan(x) else 0, -x if not np.isnan(x) else 0.0, e) for e, x in enumerate(v) if x != -np.inf]
        ids = [e for _, _, e in sorted(key)][:k]
        experts[t, :len(ids)] = ids
        if not ids:
            continue
        with np.errstate(invalid="ignore"):
            top = np.exp(v[ids] - v[ids[0]])
            z = top.sum() if renormalise else np.exp(v[v != -np.inf] - v[ids[0]]).sum()
            w[t, :len(ids)] = top / z * scale
        if np.isnan(v).any():
            w[t, :len(ids)] = np.nan
    flat = experts.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    used = int((flat >= 0).sum())
    rows = np.where(np.arange(T * k) < used, order, -1).astype(np.int32)
    places = np.full(T * k, -1, np.int32)
    places[order[:used]] = np.arange(used)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    return experts, w, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), rows, places


def experts_of(offsets, n_pairs):
    """The expert of each row, -1 behind the last."""
    e = np.full(n_pairs, -1)
    for i in range(len(offsets) - 1):
        e[offsets[i]:offsets[i + 1]] = i
    return e


# How far a product may be off, in units of 2^-24 of the sum of |weight part| * |x| over the row (both parts of each weight, code and min):
# the grouped products round, or cut, what they add. A super-block on the tensor cores is 34 additions, each off by 2^-23 of the
# sum so far at most; activations enter with 22 bits (2^-22: 4 units) and the mins' ratios with 22 (4); a rounded
# product for the scale, one for the block; then one rounded addition a super-block, and the few of a join.
# The integer kernel stays within that: 4 rounded operations for 64 weights, 5 additions of a warp.
def units(in_dim):
    return 2 * 34 + 4 + 4 + 2 + in_dim // 256 + 8


def swiglu(gate, up, x, rows, expert, k):
    """(h, tolerance) f64 [pairs, inter]; gate, up (values, sizes) [E, inter, in]; x f64 [T, in]."""
    h, tol = np.zeros((len(rows), gate[0].shape[1])), np.zeros((len(rows), gate[0].shape[1]))
    eps = units(x.shape[1]) * 2.0 ** -24
    for r, e in enumerate(expert):
        if e < 0:
            continue
        v = x[rows[r] // k]
        g, u = gate[0][e] @ v, up[0][e] @ v
        dg, du = eps * (gate[1][e] @ np.abs(v)), eps * (up[1][e] @ np.abs(v))
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        h[r] = silu * u
        # |silu'| < 1.1; then, in half-ulps of h (2^-24): e^-g within 3 + 1.173 |g| ulp, which 1 + e^-g does not make larger (twice that in
        # half-ulps), an addition (1), a division within 2 ulp (4), a product (1)
        tol[r] = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + (12 + 2.4 * np.abs(g)) * 2.0 ** -24 * np.abs(h[r]) + 1e-37
    return h, tol


def down(w, h, places, expert, weight, residual):
    """(y, tolerance) f64 [T, out]; w (values, sizes) [E, out, in]; h f64 [pairs, in]."""
    T, k = weight.shape
    y = np.zeros((T, w[0].shape[1])) if residual is None else residual.astype(np.float64).copy()
    tol, eps = np.zeros_like(y), units(h.shape[1]) * 2.0 ** -24
    size = np.abs(y)
    for t in range(T):
        for j in range(k):
            r = places[t * k + j]
            if r < 0:
                continue
            o = w[0][expert[r]] @ h[r]
            y[t] += weight[t, j] * o
            size[t] += np.abs(weight[t, j] * o)
            tol[t] += np.abs(weight[t, j]) * eps * (w[1][expert[r]] @ np.abs(h[r]))
    return y, tol + (k + 1) * 2.0 ** -24 * size + 1e-37
