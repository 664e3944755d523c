"""The paged 4-bit KV cache on the GPU against numpy in f64 (paged_reference.py)."""
import numpy as np
import pytest

import paged_reference as R
from gpu_common import check_no_device_error, to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half an f32 step


@pytest.fixture(scope="module")
def rz():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_q4_q8_gb300 as rz
    rz.load()
    return rz


@pytest.fixture(autouse=True)
def no_error_left(rz):
    yield
    check_no_device_error()


def device_error(rz):
    st, code = rz.check_device_error()
    assert st in (0, 7)
    return code


def ints(a, t=np.int32):
    return to_dev(np.asarray(a, t))


# ------------------------------------------------------------------ plan
def random_pool(rng, n, max_blocks, page, spare, cached):
    owned = -(-cached // page)
    pages = int(owned.sum()) + spare
    order = rng.permutation(max(pages, 1)).astype(np.int32)
    table = np.full((n, max_blocks), -7, np.int32)
    at = 0
    for i in range(n):
        table[i, :owned[i]] = order[at:at + owned[i]]
        at += owned[i]
    free = np.full(max(pages, 1), -9, np.int32)
    free[:spare] = order[at:]
    return owned.astype(np.int32), table, free


def run_plan(rz, cached, fresh, owned, table, free, count, page, max_rows, in_place=True, ld=0):
    import torch
    n, max_blocks = table.shape
    t = torch.full((n, max_blocks + ld), -77, dtype=torch.int32, device="cuda")
    tv = t[:, :max_blocks]
    tv.copy_(to_dev(table))
    o, f, c = ints(owned), ints(free), ints([count])
    o2, c2 = (o, c) if in_place else (torch.full_like(o, -5), torch.full_like(c, -5))
    out = rz.PagedPlan(n, max_rows)
    rz.paged_plan(ints(cached), ints(fresh), tv, o, f, c, page, out, owned_out=o2, free_count_out=c2)
    got = {k: getattr(out, k).cpu().numpy() for k in ("cu_rows", "kv_len", "row_seq", "positions", "slots")}
    got |= dict(table=tv.cpu().numpy(), owned=o2.cpu().numpy(), free=f.cpu().numpy(), count=int(c2.item()))
    if ld:
        assert (t[:, max_blocks:] == -77).all()
    if not in_place:
        assert np.array_equal(o.cpu().numpy(), owned) and int(c.item()) == count
    return got


def check_plan(rz, *args, **kw):
    want = R.plan(*args)
    got = run_plan(rz, *args, **kw)
    code = device_error(rz)
    assert code == (0x203 if want["bad"] else 0x204 if want["refused"] else 0) or (want["bad"] and want["refused"] and code in (0x203, 0x204))
    for k, v in got.items():
        assert np.array_equal(v, want[k]), k
    return want


@pytest.mark.parametrize("n,page,max_rows,spare,in_place", [
    (1, 16, 1, 3, True), (1, 128, 300, 5, False), (7, 16, 64, 40, True), (33, 32, 500, 60, False), (255, 64, 2048, 400, True),
    (512, 16, 2100, 3000, True), (513, 16, 700, 3000, False), (1000, 16, 20000, 9000, True), (1024, 128, 3000, 3000, False)])
def test_plan_matches_reference(rz, n, page, max_rows, spare, in_place):
    rng = np.random.default_rng(n * 100 + page)
    cached = rng.integers(0, 40 * page, n).astype(np.int32)
    fresh = rng.choice([0, 1, 1, 1, 5, -1], n).astype(np.int32)
    if n > 4:
        fresh[rng.integers(0, n, 3)] = rng.integers(1, 60, 3)
    owned, table, free = random_pool(rng, n, 48, page, spare, cached)
    check_plan(rz, cached, fresh, owned, table, free, spare, page, max_rows, in_place=in_place, ld=0 if n % 2 else 3)


@pytest.mark.parametrize("spare,ended", [(0, 0), (1, 0), (3, 0), (3, 2), (0, 5)])
def test_plan_pool_runs_out(rz, spare, ended):
    rng = np.random.default_rng(spare)
    cached = np.array([16, 15, 32, 3, 48, 0, 64, 16], np.int32)
    fresh = np.array([1, 1, 17, 1, 1, 33, 0, 2], np.int32)
    fresh[len(fresh) - ended:] = -1
    owned, table, free = random_pool(rng, 8, 9, 16, spare, cached)
    w = check_plan(rz, cached, fresh, owned, table, free, spare, 16, 80)
    assert w["refused"] == (spare + ended < 4 or not ended)


def test_plan_owned_pages_beyond_the_length_are_used_first(rz):
    # a request shortened by rejected drafts keeps its pages
    table = np.array([[5, 6, 7, -1], [1, 2, -1, -1]], np.int32)
    w = check_plan(rz, np.array([17, 0]), np.array([20, 33]), np.array([3, 2], np.int32), table, np.array([9, 8, 0, 0], np.int32), 2, 16, 64)
    assert list(w["slots"][:3]) == [6 * 16 + 1, 6 * 16 + 2, 6 * 16 + 3] and w["owned"][0] == 3 and w["owned"][1] == 3


@pytest.mark.parametrize("what", ["cached", "owned", "owned_big", "long", "held_nowhere", "rows", "count", "count_big", "overfull"])
def test_plan_bad_lengths_are_refused_and_reported(rz, what):
    cached, fresh = np.array([10, 20, 30, 0], np.int32), np.array([1, 2, 1, 1], np.int32)
    rng = np.random.default_rng(1)
    owned, table, free = random_pool(rng, 4, 4, 16, 6, cached)
    count, rows = 6, 20
    if what == "cached":
        cached[1] = -4
    elif what == "owned":
        owned[1] = -1
    elif what == "owned_big":
        owned[1] = 5
    elif what == "long":
        fresh[1], rows = 60, 100
    elif what == "held_nowhere":
        cached[1] = 60
    elif what == "rows":
        rows = 2
    elif what == "count":
        count = -1
    elif what == "count_big":
        count = len(free) + 1
    elif what == "overfull":
        fresh[1], count = -1, len(free)
    if what in ("count", "count_big"):
        got = run_plan(rz, cached, fresh, owned, table, free, count, 16, rows)
        assert device_error(rz) in (0x203, 0x204)
        assert got["count"] == 0 and got["kv_len"][3] == 0 and got["kv_len"][0] == 11  # nothing to hand out
    elif what == "overfull":
        got = run_plan(rz, cached, fresh, owned, table, free, count, 16, rows)
        assert device_error(rz) == 0x203 and got["count"] <= len(free)
    else:
        check_plan(rz, cached, fresh, owned, table, free, count, 16, rows)


# ------------------------------------------------------------------ norm, rotation, append
def heads_case(rng, T, H, K, hd, page, spread=1.0):
    qkv = (rng.standard_normal((T, (H + 2 * K) * hd)) * spread).astype(np.float32)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    return qkv, pages, slots


def run_heads(rz, qkv, H, K, hd, page, pages, slots, pos, theta, mode, gq, gk, eps=1e-6, fill=0xAB, q_out=None):
    import torch
    d = to_dev(qkv)
    q, k, v = d[:, :H * hd], d[:, H * hd:(H + K) * hd], d[:, (H + K) * hd:]
    kv = rz.PagedKVQ4(torch.full((pages, K, page * hd * 9 // 8), fill, dtype=torch.uint8, device="cuda"), page, hd)
    out = rz.qk_norm_rope(q, k, v, ints(pos), H, K, hd, theta, mode, q_gamma=None if gq is None else to_dev(gq),
                          k_gamma=None if gk is None else to_dev(gk), eps=eps, kv=kv, slots=ints(slots, np.int64), want_k=True, want_v=True,
                          q_out=q if q_out == "q" else None)
    return [x.cpu().numpy() for x in out] + [kv.pages.cpu().numpy().reshape(-1)]


def want_heads(qkv, H, K, hd, pos, theta, mode, gq, gk, eps=1e-6):
    T = qkv.shape[0]
    x = qkv.astype(np.float64).reshape(T, H + 2 * K, hd)
    q = R.rotate(R.norm(x[:, :H], gq, eps), pos, theta, mode)
    k = R.rotate(R.norm(x[:, H:H + K], gk, eps), pos, theta, mode)
    return q, k, x[:, H + K:]


def check_cache(flat, page, K, hd, slots, k, v, fill=0xAB):
    want = np.full_like(flat, fill)
    qk, qv = R.quantise(k), R.quantise(v)
    for t, s in enumerate(slots):
        if s >= 0:
            for h in range(K):
                R.store(want, page, K, hd, int(s), h, (qk[0][t, h], qk[1][t, h]), (qv[0][t, h], qv[1][t, h]))
    assert np.array_equal(flat, want)


@pytest.mark.parametrize("hd", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("normed", [True, False])
def test_heads_all_head_dims(rz, hd, mode, normed):
    rng = np.random.default_rng(hd + mode)
    T, H, K, page = 21, 6, 3, 32
    qkv, pages, slots = heads_case(rng, T, H, K, hd, page)
    pos = rng.integers(0, 100000, T)
    pos[0] = 0
    gq, gk = (rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32)) if normed else (None, None)
    q, k, v, flat = run_heads(rz, qkv, H, K, hd, page, pages, slots, pos, 1e4, mode, gq, gk)
    wq, wk, wv = want_heads(qkv, H, K, hd, pos, 1e4, mode, gq, gk)
    # the error of a value is below 2^-20 of its pair's |y0| + |y1| (see the kernel), which the largest value of a head bounds
    bound = 2.0 ** -20 * 2 * np.abs(wq).max(-1, keepdims=True) * 2 ** 0.5
    assert (np.abs(q.reshape(wq.shape) - wq) <= bound).all()
    assert np.array_equal(k, R.quantise(wk)[2].reshape(k.shape))
    assert np.array_equal(v, R.quantise(wv)[2].reshape(v.shape))
    check_cache(flat, page, K, hd, slots, wk, wv)


@pytest.mark.parametrize("T,H,K,hd,page", [(1, 14, 2, 64, 16), (2, 32, 32, 128, 16), (3, 1, 1, 32, 128), (700, 8, 4, 128, 64), (65, 40, 40, 64, 32),
                                           (400, 71, 1, 64, 16)])
def test_heads_shapes_and_in_place(rz, T, H, K, hd, page):
    rng = np.random.default_rng(T)
    qkv, pages, slots = heads_case(rng, T, H, K, hd, page)
    slots[T // 2] = -1 if T > 2 else slots[T // 2]
    pos = rng.integers(0, 4096, T)
    g = rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32)
    q, k, v, flat = run_heads(rz, qkv, H, K, hd, page, pages, slots, pos, 1e6, 1, g[0], g[1], q_out="q")
    wq, wk, wv = want_heads(qkv, H, K, hd, pos, 1e6, 1, g[0], g[1])
    assert (np.abs(q.reshape(wq.shape) - wq) <= 2.0 ** -20 * 3 * np.abs(wq).max(-1, keepdims=True)).all()
    assert np.array_equal(k, R.quantise(wk)[2].reshape(k.shape))
    check_cache(flat, page, K, hd, slots, wk, wv)


def test_heads_padding_rows_are_left_as_they_were(rz):
    import torch
    rng = np.random.default_rng(0)
    T, H, K, hd, page = 9, 4, 2, 64, 16
    qkv, pages, slots = heads_case(rng, T, H, K, hd, page)
    pos = np.arange(T)
    pos[[2, 7, 8]] = -1
    d = to_dev(qkv)
    kv = rz.PagedKVQ4(torch.full((pages, K, page * hd * 9 // 8), 0x5C, dtype=torch.uint8, device="cuda"), page, hd)
    out = torch.full((T, H * hd), 3.25, device="cuda")
    rz.qk_norm_rope(d[:, :H * hd], d[:, H * hd:(H + K) * hd], d[:, (H + K) * hd:], ints(pos), H, K, hd, 1e4, 0, kv=kv,
                    slots=ints(slots, np.int64), q_out=out)
    assert (out[[2, 7, 8]] == 3.25).all() and not (out[[0, 1, 3]] == 3.25).any()
    wq, wk, wv = want_heads(qkv, H, K, hd, pos, 1e4, 0, None, None)
    check_cache(kv.pages.cpu().numpy().reshape(-1), page, K, hd, np.where(pos < 0, -1, slots), wk, wv, 0x5C)


def test_heads_slot_beyond_the_cache_is_reported_and_skipped(rz):
    rng = np.random.default_rng(0)
    qkv, pages, slots = heads_case(rng, 3, 2, 2, 64, 16)
    slots = np.array([5, pages * 16, 7])
    q, k, v, flat = run_heads(rz, qkv, 2, 2, 64, 16, pages, slots, np.arange(3), 1e4, 1, None, None)
    assert device_error(rz) == 0x205
    wq, wk, wv = want_heads(qkv, 2, 2, 64, np.arange(3), 1e4, 1, None, None)
    check_cache(flat, 16, 2, 64, [5, -1, 7], wk, wv)


def test_heads_without_a_cache(rz):
    rng = np.random.default_rng(5)
    T, H, K, hd = 13, 5, 2, 96
    x = rng.standard_normal((T, (H + K) * hd)).astype(np.float32)
    d = to_dev(x)
    pos = rng.integers(0, 1 << 20, T)
    q, k, v = rz.qk_norm_rope(d[:, :H * hd], d[:, H * hd:], None, ints(pos), H, K, hd, 1e4, 1)
    assert v is None
    w = R.rotate(x.astype(np.float64).reshape(T, H + K, hd), pos, 1e4, 1)
    got = np.concatenate([q.cpu().numpy(), k.cpu().numpy()], 1).reshape(w.shape)
    assert (np.abs(got - w) <= 2.0 ** -20 * 3 * np.abs(w).max(-1, keepdims=True)).all()


@pytest.mark.parametrize("normed", [True, False])
def test_heads_special_values(rz, normed):
    """Zeros, ties of two peaks, exact borders between codes, subnormal and huge scales, NaN and infinities."""
    rng = np.random.default_rng(9)
    H, K, hd, page = 1, 1, 64, 16
    rows = [np.zeros(64), np.full(64, 1e-30), np.full(64, 3e38), np.full(64, -1e-42)]
    a = rng.standard_normal(64)
    a[3], a[9] = 5.0, -5.0
    rows.append(a)
    b = np.arange(64) / 16.0 - 2.0          # many values half-way between codes: the peak is -2, a step 1/4
    rows.append(b)
    rows.append(np.where(np.arange(64) % 2 == 0, 8.0, -7.5))
    for bad in (np.nan, np.inf, -np.inf):
        c = rng.standard_normal(64)
        c[40] = bad
        rows.append(c)
    rows.append(rng.standard_normal(64) * 1e25)
    rows.append(rng.standard_normal(64) * 1e-25)
    rows.append(rng.standard_normal(64) * 4e5)
    rows.append(rng.standard_normal(64) * 3e-7)
    x = np.array(rows, np.float32)
    T = len(rows)
    qkv = np.concatenate([x, x, x], 1)
    pos = np.zeros(T, int)
    g = rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32) if normed else (None, None)
    slots = np.arange(T)
    with np.errstate(all="ignore"):
        q, k, v, flat = run_heads(rz, qkv, H, K, hd, page, 2, slots, pos, 1e4, 1, g[0], g[1])
        wq, wk, wv = want_heads(qkv, H, K, hd, pos, 1e4, 1, g[0], g[1])
        assert np.array_equal(v, R.quantise(wv)[2].reshape(v.shape), equal_nan=True)
        assert np.array_equal(k, R.quantise(wk)[2].reshape(k.shape), equal_nan=True)
        fine = np.isfinite(wq).all(-1).reshape(T) & (np.abs(wq).max(-1).reshape(T) < 3e38)
        assert (np.abs(q[fine] - wq.reshape(T, -1)[fine]) <= 2.0 ** -20 * 3 * np.abs(wq.reshape(T, -1)[fine]).max(-1, keepdims=True) + 1e-44).all()
        # a NaN in any value of a scale: the bits may differ, so only the others are compared
    want = np.full_like(flat, 0xAB)
    qk, qv = R.quantise(wk), R.quantise(wv)
    for t in range(T):
        if np.isfinite(x[t]).all():
            R.store(want, page, K, hd, t, 0, (qk[0][t, 0], qk[1][t, 0]), (qv[0][t, 0], qv[1][t, 0]))
            nb = 2
            for place in (R.k_place, R.v_place):
                for bb in range(nb):
                    for i in range(16):
                        at = R.record_of(page, K, hd, t, 0) + place(nb, t % 16, bb, i)
                        assert flat[at] == want[at], (t, bb, i)


def test_heads_codes_hold_next_to_borders(rz):
    """Many keys: without the second look in f64 some codes would differ from the definition's."""
    rng = np.random.default_rng(77)
    T, H, K, hd, page = 2000, 1, 8, 64, 64
    qkv, pages, slots = heads_case(rng, T, H, K, hd, page)
    pos = rng.integers(0, 131072, T)
    g = rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32)
    q, k, v, flat = run_heads(rz, qkv, H, K, hd, page, pages, slots, pos, 1e4, 0, g[0], g[1])
    wq, wk, wv = want_heads(qkv, H, K, hd, pos, 1e4, 0, g[0], g[1])
    assert np.array_equal(k, R.quantise(wk)[2].reshape(k.shape))
    assert np.array_equal(v, R.quantise(wv)[2].reshape(v.shape))


# ------------------------------------------------------------------ attention
class Setup:
    """Requests (held, new) over a cache of random pages; what no request holds is NaN."""

    def __init__(self, seed, H, K, hd, page, reqs, spread=1.0, sharp=1.0, v_mean=0.0, ld=0, extra_rows=0, ld_table=0,
                 key_size=None):
        import torch
        rng = np.random.default_rng(seed)
        self.H, self.K, self.hd, self.page, self.reqs = H, K, hd, page, reqs
        blocks = [-(-n // page) for n, _ in reqs]
        pages = sum(blocks) + 3
        k = rng.standard_normal((pages * page, K, hd)) * sharp
        v = (rng.standard_normal((pages * page, K, hd)) + v_mean) * spread
        order = rng.permutation(pages)
        self.max_blocks = max(max(blocks), 1) + 1
        self.table = np.full((len(reqs), self.max_blocks), 2 ** 31 - 1, np.int64)
        at, self.slots = 0, []
        used = np.zeros(pages * page, bool)
        for i, (n, _) in enumerate(reqs):
            self.table[i, :blocks[i]] = order[at:at + blocks[i]]
            at += blocks[i]
            s = self.table[i, np.arange(n) // page] * page + np.arange(n) % page
            self.slots.append(s)
            used[s] = True
            if key_size is not None:
                k[s] *= key_size(np.arange(n))[:, None, None]
        k[~used], v[~used] = np.nan, np.nan
        with np.errstate(all="ignore"):
            flat, self.kval, self.vval = R.pack(k, v, page)
        self.kd, self.vd = (np.abs(x.reshape(-1, K, hd // 32, 32)).max(-1) / 7 for x in (self.kval, self.vval))  # at least |d|
        rows = [m for _, m in reqs]
        self.cu = np.concatenate([[0], np.cumsum(rows)])
        self.T = int(self.cu[-1]) + extra_rows
        q = rng.standard_normal((self.T, H * hd + ld)).astype(np.float32)
        if extra_rows:
            q[self.cu[-1]:] = np.nan
        self.q = q[:, :H * hd]
        self.qd = to_dev(q)[:, :H * hd]
        import quantized_q4_q8_gb300 as rz
        self.kv = rz.PagedKVQ4(to_dev(flat.reshape(pages, K, -1)), page, hd)
        t = torch.full((len(reqs), self.max_blocks + ld_table), -1, dtype=torch.int32, device="cuda")
        t[:, :self.max_blocks] = ints(self.table)
        self.td = t[:, :self.max_blocks]
        self.cud, self.lend = ints(self.cu), ints([n for n, _ in reqs])
        self.ws = rz.workspace(rz.attention_paged_q4_workspace_bytes(H, K, hd), "cuda")

    def run(self, rz, **kw):
        kw.setdefault("ws", self.ws)
        return rz.attention_paged_q4(self.qd, self.kv, self.td, self.cud, self.lend, self.H, **kw)

    def check(self, got, scale=0.0, reqs=None):
        """Against f64, within the bound that follows from the kernel's arithmetic:
        a score is off by delta <= scale 2^-20 sum_b |d_b| 23 sum |q_b| (two pieces of q to 2^-22 of
        its row's largest value, at most nb + 8 roundings of sums of codes up to 15 and of 8 sum q), and by
        2^-24 (|s| log2 e + 40) in the exponent; exp to 2^-21; a weighted sum to 2^-22 (pieces) + 2^-23 for
        each of its tokens / 16 + 40 steps, of A = 23 sum_j p_j |d_j| of the block (codes up to 15, and 8).
        The output is off by at most (2 delta + the rest) A."""
        H, K, hd, G = self.H, self.K, self.hd, self.H // self.K
        sc = scale or hd ** -0.5
        got = np.asarray(got, np.float64)
        worst = off2 = all2 = 0.0
        for i, (n, m) in enumerate(self.reqs):
            if m == 0:
                continue
            s = self.slots[i]
            for h in range(K):
                q = self.q[self.cu[i]:self.cu[i] + m].reshape(m, H, hd)[:, h * G:(h + 1) * G].astype(np.float64).reshape(m * G, hd)
                sees = np.repeat(np.clip(n - m + np.arange(m) + 1, 0, n), G)
                k, v = self.kval[s, h].astype(np.float64), self.vval[s, h].astype(np.float64)
                want, p = R.attention(q, k, v, sees, sc)
                out = got[self.cu[i]:self.cu[i] + m].reshape(m, H, hd)[:, h * G:(h + 1) * G].reshape(m * G, hd)
                if n == 0:
                    assert not out.any()
                    continue
                qb = np.abs(q).reshape(m * G, -1, 32).sum(-1) + 2.0 ** -2 * np.abs(q).max(-1, keepdims=True)
                delta = (sc * 2.0 ** -20 * 23 * (qb @ self.kd[s, h].T)).max(-1, initial=0)
                top = np.abs(q @ k.T * sc).max(-1, initial=0)
                rel = 2 * (delta + U * (top * 1.45 + 40)) + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -23 * (n / 16 + 40)
                A = 23 * np.repeat(p @ self.vd[s, h], 32, axis=-1)
                err = np.abs(out - want)
                assert (err <= rel[:, None] * A + 1e-38).all(), (i, h, (err / (rel[:, None] * A + 1e-38)).max())
                worst = max(worst, (err / (rel[:, None] * A + 1e-38)).max())
                off2, all2 = off2 + (err ** 2).sum(), all2 + (want ** 2).sum()
        assert off2 <= (1e-5) ** 2 * all2 or self.T == 0
        return worst


SHAPES = [(hd, H, K) for hd in (32, 64, 96, 128, 160, 192, 224, 256) for H, K in ((4, 2),)] + [
    (64, 14, 2), (128, 8, 8), (128, 8, 1), (64, 16, 1), (64, 33, 1), (96, 9, 3), (256, 16, 2)]


@pytest.mark.parametrize("hd,H,K", SHAPES)
@pytest.mark.parametrize("page", [16, 64])
def test_attention_shapes(rz, hd, H, K, page):
    reqs = [(1, 1), (15, 1), (16, 1), (17, 2), (177, 1), (0, 0), (100, 0), (300, 5), (40, 40), (700, 1)]
    s = Setup(hd + H, H, K, hd, page, reqs)
    s.check(s.run(rz).cpu().numpy())


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 175, 176, 177, 352, 353, 1000, 4100])
def test_attention_lengths(rz, page, n):
    s = Setup(n, 4, 2, 64, page, [(n, 1), (max(n - 1, 1), 1)])
    s.check(s.run(rz).cpu().numpy())


@pytest.mark.parametrize("m", [1, 2, 3, 4, 6, 7, 10, 11, 21, 22, 23, 64, 129])
def test_attention_new_tokens(rz, m):
    # groups of 4 heads: items of 1, 2, 3, 5 and 11 row groups, and several items
    s = Setup(m, 8, 2, 64, 32, [(m + 250, m), (m, m), (m + 5000, m)])
    s.check(s.run(rz).cpu().numpy())


@pytest.mark.parametrize("hd,H,K", [(128, 8, 2), (64, 14, 2), (128, 4, 4), (128, 16, 1), (64, 7, 1), (96, 4, 2)])
@pytest.mark.parametrize("page", [16, 128])
def test_attention_prompt_chunks(rz, hd, H, K, page):
    """Many rows: whole prompts, chunks behind a context, odd sizes, beside decodes and empty requests."""
    s = Setup(hd + H + page, H, K, hd, page, [(130, 130), (1000, 65), (129, 128), (5, 5), (700, 1), (0, 0), (257, 256), (1500, 33)])
    s.check(s.run(rz).cpu().numpy())


@pytest.mark.parametrize("n,m", [(64, 64), (65, 65), (127, 127), (128, 128), (129, 129), (4000, 1000), (20, 200), (3, 150), (0, 150), (2999, 300)])
def test_attention_one_prompt_chunk(rz, n, m):
    s = Setup(n + m, 4, 2, 128, 64, [(n, m)])
    out = s.run(rz).cpu().numpy()
    assert not out[:max(m - n, 0)].any()
    s.check(out)


@pytest.mark.parametrize("spread,sharp,v_mean", [(1e-4, 0.01, 0.0), (3e4, 12.0, 0.0), (1.0, 12.0, 4.0), (1.0, 1.0, 4.0)])
def test_attention_prompt_chunk_scales(rz, spread, sharp, v_mean):
    s = Setup(8, 4, 2, 128, 16, [(900, 200), (33, 33), (2500, 100)], spread=spread, sharp=sharp, v_mean=v_mean)
    s.check(s.run(rz).cpu().numpy())


@pytest.mark.parametrize("first,then", [(0.05, 16.0), (16.0, 0.05)])
@pytest.mark.parametrize("hd,H,K", [(64, 4, 1), (128, 4, 2)])
def test_attention_prompt_chunk_maximum_moves(rz, hd, H, K, first, then):
    """The rows' maxima grow by about 2^70 at token 2100 (or never again after it), far within the parts of an
    item: sums that were put aside before are as good as nothing (or all there is)."""
    s = Setup(hd, H, K, hd, 32, [(5000, 1500)], key_size=lambda j: np.where(j < 2100, first, then))
    s.check(s.run(rz).cpu().numpy())


def test_attention_prompt_chunk_nan_and_padding(rz):
    """NaN keys and values reach the rows that see them and no others; rows behind the last stay; q8; repeats."""
    import torch
    s = Setup(13, 4, 2, 64, 16, [(500, 200), (60, 1)], extra_rows=5)
    out = torch.full((s.T, 256), 2.5, device="cuda")
    q8 = torch.full((rz.q8_1_size(s.T, 256),), 0x55, dtype=torch.uint8, device="cuda")
    good = s.run(rz, out=out, att_q8=q8).clone()
    assert (good[201:] == 2.5).all()
    assert torch.equal(q8.view(-1)[:201 * 256], rz.q8_1_quantize(good[:201].contiguous())[:201 * 256])
    ds = q8[s.T * 256:].view(torch.float32).view(2, s.T, 8)
    want = rz.q8_1_quantize(good[:201].contiguous())[201 * 256:].view(torch.float32).view(2, 201, 8)
    assert torch.equal(ds[:, :201], want) and (q8[s.T * 256:].view(2, s.T, 32)[:, 201:] == 0x55).all()
    for _ in range(3):
        assert torch.equal(s.run(rz, out=out), good)
    # token 450's value scale in kv head 1, token 470's key scale in kv head 0 (rows 150 and 170 are the first that see them)
    for token, head, scales in ((450, 1, 17), (470, 0, 8)):
        at = R.record_of(16, 2, 64, int(s.slots[0][token]), head) + scales * 64 + (token % 16) * 4
        s.kv.pages.view(-1)[at:at + 4] = torch.tensor([0, 0x7e, 0, 0x7e], dtype=torch.uint8, device="cuda")
    bad = s.run(rz, out=out)
    seen = torch.zeros_like(good, dtype=torch.bool)
    seen[150:200, 128:] = True
    seen[170:200, :128] = True
    assert torch.isnan(bad[seen]).all() and torch.equal(bad[~seen], good[~seen])


def test_attention_long_and_split_over_all_ctas(rz):
    s = Setup(2, 4, 1, 128, 64, [(40001, 1)])
    s.check(s.run(rz).cpu().numpy())


def test_attention_many_requests(rz):
    rng = np.random.default_rng(4)
    reqs = [(int(n), int(m)) for n, m in zip(rng.integers(1, 90, 1024), rng.integers(0, 2, 1024))]
    s = Setup(3, 2, 1, 32, 16, reqs)
    s.check(s.run(rz).cpu().numpy())


@pytest.mark.parametrize("hd", [128, 256])
def test_attention_most_requests_of_wide_heads(rz, hd):
    """1024 requests, whose rows of the plan take shared memory from the ring of units."""
    rng = np.random.default_rng(hd)
    reqs = [(int(n), 1) for n in rng.integers(1, 80, 1023)] + [(700, 3)]
    s = Setup(hd, 2, 1, hd, 16, reqs)
    s.check(s.run(rz).cpu().numpy())


def test_attention_shared_pages(rz):
    """A prefix whose pages stand in the rows of several requests; with row counts of every width of an item."""
    H, K, hd, page = 8, 2, 64, 16
    s = Setup(5, H, K, hd, page, [(333, 1), (1, 1), (1, 1), (1, 1)])
    prefix = s.table[0, :20]
    reqs, s.slots = [(333, 1), (322, 2), (336, 4), (330, 9)], [s.slots[0]]
    for i in (1, 2, 3):
        own = s.table[i, 0]
        s.table[i, :20], s.table[i, 20] = prefix, own
        n = reqs[i][0]
        s.slots.append(s.table[i, np.arange(n) // page] * page + np.arange(n) % page)
    # the requests' own last pages hold one token each so far: give them sixteen
    rng = np.random.default_rng(6)
    pages = s.kv.pages.shape[0]
    k, v = s.kval.reshape(pages, page, K, hd).copy(), s.vval.reshape(pages, page, K, hd).copy()
    for i in (1, 2, 3):
        k[s.table[i, 20]], v[s.table[i, 20]] = rng.standard_normal((2, page, K, hd))
    flat, s.kval, s.vval = R.pack(k.reshape(-1, K, hd), v.reshape(-1, K, hd), page)
    s.kd, s.vd = (np.abs(x.reshape(-1, K, hd // 32, 32)).max(-1) / 7 for x in (s.kval, s.vval))
    s.reqs, s.cu = reqs, np.concatenate([[0], np.cumsum([m for _, m in reqs])])
    s.T = int(s.cu[-1])
    s.q = rng.standard_normal((s.T, H * hd)).astype(np.float32)
    s.qd, s.td, s.cud, s.lend = to_dev(s.q), ints(s.table), ints(s.cu), ints([n for n, _ in reqs])
    s.kv = rz.PagedKVQ4(to_dev(flat.reshape(pages, K, -1)), page, hd)
    s.check(s.run(rz).cpu().numpy())


def test_attention_more_new_rows_than_held_tokens(rz):
    """Rows that see nothing come out as zeros, whatever their neighbours see."""
    s = Setup(6, 4, 2, 64, 16, [(3, 8), (0, 5), (20, 33)])
    out = s.run(rz).cpu().numpy()
    assert not out[:5].any() and not out[8:13].any()
    s.check(out)


@pytest.mark.parametrize("spread", [1e-4, 1.0, 3e4])
@pytest.mark.parametrize("sharp", [0.01, 1.0, 12.0])
def test_attention_scales(rz, spread, sharp):
    s = Setup(8, 4, 2, 128, 16, [(900, 1), (33, 3), (2500, 30)], spread=spread, sharp=sharp)
    s.check(s.run(rz).cpu().numpy())


def test_attention_values_of_one_sign(rz):
    s = Setup(8, 4, 2, 128, 16, [(9000, 1), (700, 9)], v_mean=4.0)
    s.check(s.run(rz).cpu().numpy())


def test_attention_scale_argument_and_strides(rz):
    s = Setup(10, 4, 2, 64, 32, [(200, 2), (77, 1)], ld=20, ld_table=5)
    s.check(s.run(rz, scale=0.25).cpu().numpy(), scale=0.25)


def test_attention_rows_behind_the_last_are_left_as_they_were(rz):
    import torch
    s = Setup(11, 4, 2, 96, 16, [(200, 2), (77, 3)], extra_rows=6)
    out = torch.full((s.T, 4 * 96), 2.5, device="cuda")
    q8 = torch.full((rz.q8_1_size(s.T, 512),), 0x77, dtype=torch.uint8, device="cuda")
    s.run(rz, out=out, att_q8=q8)
    assert (out[5:] == 2.5).all()
    codes = q8[:s.T * 512].view(s.T, 512)
    assert (codes[5:] == 0x77).all() and not (codes[:5, 384:] != 0).any()
    ds = q8[s.T * 512:].view(2, s.T, 64)
    assert (ds[:, 5:] == 0x77).all()
    s.check(out.cpu().numpy())


@pytest.mark.parametrize("hd,H,K,page", [(64, 14, 2, 16), (128, 32, 8, 64), (96, 3, 3, 32), (32, 7, 1, 16), (256, 4, 2, 16)])
def test_attention_q8_is_the_quantised_output(rz, hd, H, K, page):
    import torch
    s = Setup(12, H, K, hd, page, [(200, 2), (1, 1), (3000, 1), (0, 2), (500, 40)])
    q_pad = -(-H * hd // 256) * 256
    q8 = torch.full((rz.q8_1_size(s.T, q_pad),), 0x55, dtype=torch.uint8, device="cuda")
    out = s.run(rz, att_q8=q8)
    padded = torch.zeros(s.T, q_pad, device="cuda")
    padded[:, :H * hd] = out
    assert torch.equal(q8, rz.q8_1_quantize(padded))
    alone = torch.zeros_like(q8)
    rz.rz_attention_paged_q4(s.qd, s.qd.stride(0), s.T, s.kv, s.td, s.td.stride(0), s.max_blocks, s.cud, s.lend, len(s.reqs), H, 0.0, None, alone,
                             s.ws, s.ws.numel())
    assert torch.equal(alone, q8)


def test_attention_nan_rows_stay_with_their_request(rz):
    """A NaN key or value of a request reaches the rows that see it and no others; an infinite query its own row."""
    import torch
    s = Setup(13, 4, 2, 64, 16, [(50, 4), (60, 1), (200, 20)])
    good = s.run(rz).clone()
    # token 48 of request 0 gets a NaN value scale in kv head 1: rows 2 and 3 see it (they see 49 and 50 tokens)
    at = R.record_of(16, 2, 64, int(s.slots[0][48]), 1) + 17 * 64 + (48 % 16) * 4
    s.kv.pages.view(-1)[at:at + 4] = torch.tensor([0, 0x7e, 0, 0x7e], dtype=torch.uint8, device="cuda")
    out = s.run(rz)
    seen = torch.zeros_like(out, dtype=torch.bool)
    seen[2:4, 128:] = True
    assert torch.isnan(out[seen]).all() and torch.equal(out[~seen], good[~seen])
    q = s.qd.clone()
    q[4, 7] = float("inf")
    out2 = rz.attention_paged_q4(q, s.kv, s.td, s.cud, s.lend, 4, ws=s.ws)
    assert torch.isnan(out2[4, :64]).all()
    seen[4, :64] = True
    assert torch.equal(out2[~seen], out[~seen])


def test_attention_repeats_bit_for_bit(rz):
    import torch
    s = Setup(14, 8, 2, 128, 32, [(3000, 1), (20, 1), (5000, 7), (800, 100)])
    first = s.run(rz).clone()
    for _ in range(5):
        assert torch.equal(s.run(rz), first)
    assert not s.ws[:1024].any()  # its counters are zero again
    rz.set_pdl(False)
    try:
        assert torch.equal(s.run(rz), first)
    finally:
        rz.set_pdl(True)


@pytest.mark.parametrize("what", ["page", "negative_page", "length", "offsets", "rows"])
def test_attention_bad_device_data_is_reported(rz, what):
    import torch
    s = Setup(15, 4, 2, 64, 16, [(50, 1), (60, 1), (70, 1)])
    good = s.run(rz).clone()
    if what == "page":
        s.td[1, 2] = s.kv.pages.shape[0]
    elif what == "negative_page":
        s.td[1, 0] = -5
    elif what == "length":
        s.lend[1] = s.max_blocks * 16 + 1
    elif what == "offsets":
        s.cud[1], s.cud[2] = 2, 1
    elif what == "rows":
        s.cud[3] = 4
    out = torch.zeros_like(good)
    s.run(rz, out=out)
    assert device_error(rz) == (0x206 if "page" in what else 0x203)
    if "page" in what:
        assert torch.equal(out[[0, 2]], good[[0, 2]])
    elif what == "length":
        s.reqs[1] = (0, 1)  # an empty request: zeros, and the others by the usual bound (their work is split elsewhere)
        s.check(out.cpu().numpy())
    check_no_device_error()


def test_attention_workspace_size_is_checked(rz):
    import torch
    s = Setup(16, 4, 2, 64, 16, [(50, 1)])
    with pytest.raises(rz.RzError, match="workspace"):
        s.run(rz, ws=torch.zeros(1024, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ together
def test_step_after_step_matches_dense_attention(rz):
    """Requests join with a prompt, decode, get drafts scored and rejected, end; one captured graph of
    plan -> norm, rotation, append -> attention serves every step, on a stream of its own."""
    import torch
    rng = np.random.default_rng(21)
    n, H, K, hd, page, max_rows, max_blocks, n_pages = 5, 6, 2, 64, 16, 96, 8, 26
    kv = rz.PagedKVQ4(torch.randint(0, 256, (n_pages, K, page * hd * 9 // 8), dtype=torch.uint8, device="cuda"), page, hd)
    table = torch.full((n, max_blocks), -1, dtype=torch.int32, device="cuda")
    owned, count = torch.zeros(n, dtype=torch.int32, device="cuda"), ints([n_pages])
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    cached, fresh = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    plan = rz.PagedPlan(n, max_rows)
    qkv = torch.zeros(max_rows, (H + 2 * K) * hd, device="cuda")
    g = rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32)
    gq, gk = to_dev(g[0]), to_dev(g[1])
    q_out = torch.zeros(max_rows, H * hd, device="cuda")
    att = torch.zeros(max_rows, H * hd, device="cuda")
    ws = rz.workspace(rz.attention_paged_q4_workspace_bytes(H, K, hd), "cuda")

    def step():
        rz.paged_plan(cached, fresh, table, owned, free, count, page, plan)
        rz.qk_norm_rope(qkv[:, :H * hd], qkv[:, H * hd:(H + K) * hd], qkv[:, (H + K) * hd:], plan.positions, H, K, hd, 1e4, 1, q_gamma=gq,
                        k_gamma=gk, kv=kv, slots=plan.slots, q_out=q_out)
        rz.attention_paged_q4(q_out, kv, table, plan.cu_rows, plan.kv_len, H, out=att, ws=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()  # no request has anything to do
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    held = [(np.zeros((0, K, hd)), np.zeros((0, K, hd))) for _ in range(n)]  # values as the cache holds them
    lens = [0] * n
    script = [[20, 3, 0, 0, 0], [1, 1, 33, 0, 0], [5, 1, 1, 16, 0], [5, -1, 1, 1, 2], [-1, 47, 1, 4, 1], [9, 1, 17, 1, 1], [1, 1, -1, 1, 1]]
    for i, news in enumerate(script):
        x = rng.standard_normal((max_rows, (H + 2 * K) * hd)).astype(np.float32)
        with torch.cuda.stream(stream):
            cached.copy_(ints(lens))
            fresh.copy_(ints(news))
            qkv.copy_(to_dev(x))
            graph.replay()
        stream.synchronize()
        check_no_device_error()
        out = att.cpu().numpy().astype(np.float64)
        at = 0
        for r, m in enumerate(news):
            if m < 0:
                held[r], lens[r] = (np.zeros((0, K, hd)), np.zeros((0, K, hd))), 0
                continue
            if m == 0:
                continue
            pos = lens[r] + np.arange(m)
            wq, wk, wv = want_heads(x[at:at + m], H, K, hd, pos, 1e4, 1, g[0], g[1])
            k = np.concatenate([held[r][0][:lens[r]], R.quantise(wk)[2]])
            v = np.concatenate([held[r][1][:lens[r]], R.quantise(wv)[2]])
            held[r] = (k, v)
            for h in range(H):
                want, _ = R.attention(wq[:, h], k[:, h // 3], v[:, h // 3], pos + 1, hd ** -0.5)
                # q is f32 here: 2^-20 of it, over scores of up to |q| |k| = 64 scale ... 8, on top of the attention's own error
                assert np.abs(out[at:at + m, h * hd:(h + 1) * hd] - want).max() <= 2.0 ** -16 * np.abs(v).max()
            lens[r] += m
            at += m
        if i == 2:
            lens[0] -= 3  # three of request 0's drafts are rejected: its pages stay its own
    assert int(count.item()) + int(owned.sum()) == n_pages
    pages = torch.cat([free[:int(count.item())]] + [table[r, :int(owned[r])] for r in range(n)])
    assert torch.equal(torch.sort(pages).values, torch.arange(n_pages, dtype=torch.int32, device="cuda"))


def test_calls_on_two_streams_with_two_workspaces(rz):
    import torch
    a, b = Setup(31, 4, 2, 64, 16, [(3000, 1), (100, 3)]), Setup(32, 4, 2, 64, 16, [(2000, 2), (900, 1)])
    wa, wb = a.run(rz).clone(), b.run(rz).clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        oa = a.run(rz, stream=sa)
        ob = b.run(rz, stream=sb.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


# ------------------------------------------------------------------ the decode layer over the paged cache
@pytest.mark.parametrize("normed", [False, True])
def test_decode_layer_paged_is_its_steps(rz, normed):
    """Bit for bit the composition of the public calls, for a prompt's rows, drafts and single tokens."""
    import torch

    import rz_synth as S
    sh = S.QWEN2
    L = S.layer(sh, "paged.l0")
    w = {k: to_dev(v) for k, v in L.w.items()} | {"attn_gamma": to_dev(L.attn_gamma), "ffn_gamma": to_dev(L.ffn_gamma)}
    layer = rz.DeviceLayer(w, sh.hidden, sh.hidden_pad, sh.n_heads, sh.n_kv_heads, sh.head_dim, sh.inter, sh.eps, sh.rope_theta, sh.rope_mode)
    H, K, hd, page, n = sh.n_heads, sh.n_kv_heads, sh.head_dim, 16, 3
    rng = np.random.default_rng(2)
    gq, gk = (to_dev(rng.uniform(0.5, 1.5, (2, hd)).astype(np.float32))) if normed else (None, None)
    kvs = [rz.PagedKVQ4.empty(9, page, K, hd) for _ in range(2)]
    for kv in kvs:
        kv.pages.zero_()
    table = torch.full((n, 4), -1, dtype=torch.int32, device="cuda")
    owned, count, free = torch.zeros(n, dtype=torch.int32, device="cuda"), ints([9]), torch.arange(9, dtype=torch.int32, device="cuda")
    lens = np.zeros(n, np.int32)
    q_pad = -(-H * hd // 256) * 256
    ws = rz.workspace(rz.decode_layer_paged_workspace_bytes(layer, 16), "cuda")
    for news in ([11, 4, 0], [1, 3, 9], [0, 1, 1]):
        m = sum(news)
        plan = rz.PagedPlan(n, m)
        rz.paged_plan(ints(lens), ints(news), table, owned, free, count, page, plan)
        x = to_dev(S.hidden_input(f"paged.x{m}", m, sh.hidden, sh.hidden_pad))
        out = rz.decode_layer_paged(x, layer, kvs[0], table, plan, q_gamma=gq, k_gamma=gk, ws=ws)
        # the same from its steps (the FFN of the layer's own workspace-free form)
        if m <= 3:
            qkv = rz.rmsnorm_q4k_gemv(x, w["attn_gamma"], sh.hidden, sh.eps, [w["wq"], w["wk"], w["wv"]], [H * hd, K * hd, K * hd], sh.hidden_pad)
        else:
            x8 = rz.rmsnorm(x, w["attn_gamma"], sh.hidden, sh.hidden_pad, sh.eps, want_y=False)[1]
            qkv = rz.q4k_q8_gemv_multi(x8, [w["wq"], w["wk"], w["wv"]], [H * hd, K * hd, K * hd], m, sh.hidden_pad)
        q, _, _ = rz.qk_norm_rope(qkv[:, :H * hd], qkv[:, H * hd:(H + K) * hd], qkv[:, (H + K) * hd:], plan.positions, H, K, hd, sh.rope_theta,
                                  sh.rope_mode, q_gamma=gq, k_gamma=gk, eps=sh.eps, kv=kvs[1], slots=plan.slots)
        a8 = torch.empty(rz.q8_1_size(m, q_pad), dtype=torch.uint8, device="cuda")
        rz.attention_paged_q4(q, kvs[1], table, plan.cu_rows, plan.kv_len, H, att_q8=a8)
        res = torch.zeros(m, sh.hidden_pad, device="cuda")
        rz.q4k_q8_gemv_ex(w["wo"], a8, m, sh.hidden, q_pad, residual=x, out=res, ld=sh.hidden_pad)
        res[:, sh.hidden:] = 0
        want = rz.swiglu_ffn(res, w["ffn_gamma"], w["wgate"], w["wup"], w["wdown"], sh.hidden, sh.hidden_pad, sh.inter, sh.eps)
        assert torch.equal(out, want), news
        assert torch.equal(kvs[0].pages, kvs[1].pages)
        lens = lens + np.array(news, np.int32)


def test_decode_layer_paged_refusals(rz):
    import torch

    import rz_synth as S
    sh = S.QWEN2
    L = S.layer(sh, "paged.l0")
    w = {k: to_dev(v) for k, v in L.w.items()} | {"attn_gamma": to_dev(L.attn_gamma), "ffn_gamma": to_dev(L.ffn_gamma)}
    layer = rz.DeviceLayer(w, sh.hidden, sh.hidden_pad, sh.n_heads, sh.n_kv_heads, sh.head_dim, sh.inter, sh.eps, sh.rope_theta, sh.rope_mode)
    x = torch.zeros(2, sh.hidden_pad, device="cuda")
    table, plan = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), rz.PagedPlan(1, 2)
    kv = rz.PagedKVQ4.empty(4, 16, sh.n_kv_heads, sh.head_dim)
    with pytest.raises(rz.RzError, match="cache holds"):
        rz.decode_layer_paged(x, layer, rz.PagedKVQ4.empty(4, 16, sh.n_kv_heads, 2 * sh.head_dim), table, plan)
    with pytest.raises(rz.RzError, match="workspace"):
        rz.decode_layer_paged(x, layer, kv, table, plan, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="fewer rows"):
        rz.decode_layer_paged(torch.zeros(3, sh.hidden_pad, device="cuda"), layer, kv, table, plan)
    with pytest.raises(ValueError, match="q_gamma"):
        rz.decode_layer_paged(x, layer, kv, table, plan, q_gamma=torch.zeros(5, device="cuda"))
    assert rz.decode_layer_paged_workspace_bytes(layer, 17) == 0
