"""The operators of an FFN of experts on the GPU against plain forms in 64 bits."""
import numpy as np
import pytest

import moe_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import quantized_q4_q8_gb300 as m
    yield m
    st, code = m.check_device_error()
    assert st == 0, f"device error word 0x{code:x}"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().cpu().numpy()


# ---------------------------------------------------------------- residual + norm
def norm_inputs(m, n, n_pad, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x, d = rng.normal(0, 1, (2, m, n_pad)).astype(np.float32)
    x *= np.exp(rng.uniform(-spread, spread, (m, 1))).astype(np.float32)
    x[:, n // 2] *= 50
    x[:, n:], d[:, n:] = np.nan, np.nan  # not read
    return x, d, rng.uniform(0.5, 1.5, n).astype(np.float32)


def norm_reference(x, d, gamma, n, eps):
    """(sum f32, y f64): the padding is 0."""
    s = np.zeros_like(x)
    s[:, :n] = x[:, :n] + d[:, :n] if d is not None else x[:, :n]
    v = s.astype(np.float64)[:, :n]
    y = np.zeros(x.shape)
    y[:, :n] = v / np.sqrt((v * v).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * gamma.astype(np.float64)
    return s, y


@pytest.mark.parametrize("m,n,n_pad", [(1, 1, 32), (3, 31, 32), (1, 896, 1024), (2, 1000, 1024), (33, 1025, 1056), (5, 2048, 2048), (7, 2049, 2304),
                                       (300, 4096, 4096), (2, 4097, 4352), (3, 8190, 8192), (1, 8193, 16384), (2, 16384, 16384)])
@pytest.mark.parametrize("with_delta", [True, False])
def test_norm(rz, m, n, n_pad, with_delta):
    x, d, gamma = norm_inputs(m, n, n_pad, 7 * n + m)
    d = d if with_delta else None
    s_ref, y_ref = norm_reference(x, d, gamma, n, 1e-5)
    s, y, q8 = rz.residual_rmsnorm(dev(x), None if d is None else dev(d), dev(gamma), n, n_pad, 1e-5)
    assert np.array_equal(host(s), s_ref)
    # the nearest f32, or its neighbour where the value lies within 2^-40 of the middle
    assert np.all(np.abs(host(y) - y_ref) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(y_ref))
    q, dd, ss = R.q8_quantize(host(y), multiplied=True)
    assert np.array_equal(host(q8), R.q8_buffer(q, dd, ss))
    # and so the codes are those of the formula
    assert np.array_equal(R.q8_quantize(y_ref.astype(np.float32), multiplied=True)[0], q)
    # the scales are within an ulp of the division's
    assert np.all(np.abs(dd - R.q8_quantize(host(y))[1]) <= 2.0 ** -23 * dd)


def test_norm_in_place_and_single_outputs(rz):
    m, n, n_pad = 5, 900, 1024
    x, d, gamma = norm_inputs(m, n, n_pad, 3)
    s0, y0, q0 = rz.residual_rmsnorm(dev(x), dev(d), dev(gamma), n, n_pad, 1e-6)
    for which in (0, 1):
        ins = [dev(x), dev(d)]
        s, y, q8 = rz.residual_rmsnorm(ins[0], ins[1], dev(gamma), n, n_pad, 1e-6, sum_out=ins[which], want_y=which == 0, want_q8=which == 1)
        assert s is ins[which] and torch.equal(s, s0)
        assert torch.equal(y, y0) if which == 0 else y is None
        assert torch.equal(q8, q0) if which == 1 else q8 is None
    ins = [dev(x), dev(d)]
    g = dev(gamma)  # y over x, sum over delta, by the C entry point
    rz.rz_residual_rmsnorm(ins[0], ins[1], g, ins[1], ins[0], None, m, n, n_pad, 1e-6)
    assert torch.equal(ins[0], y0) and torch.equal(ins[1], s0)
    ins = [dev(x), dev(d)]
    rz.rz_residual_rmsnorm(ins[0], ins[1], g, None, ins[1], None, m, n, n_pad, 1e-6)
    assert torch.equal(ins[1], y0)


def test_norm_rows_of_zeros_and_extremes(rz):
    n = 256
    x = np.zeros((6, n), np.float32)
    x[1] = 1e-20           # squares underflow: eps alone
    x[2] = 1e15
    x[3, 5] = np.inf
    x[4, 7] = np.nan
    x[5] = 1e-3
    gamma = np.ones(n, np.float32)
    s, y, q8 = rz.residual_rmsnorm(dev(x), dev(np.zeros_like(x)), dev(gamma), n, n, 1e-6)
    y = host(y)
    with np.errstate(all="ignore"):
        _, ref = norm_reference(x, None, gamma, n, 1e-6)
    ok = [0, 1, 2, 5]
    assert np.all(np.abs(y[ok] - ref[ok]) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(ref[ok]))
    assert not np.isfinite(y[3]).all() and np.isnan(y[4]).all()
    ok = [0, 1, 2, 5]
    for a, b in zip(R.q8_parts(host(q8), 6, n), R.q8_quantize(y[ok], multiplied=True)):
        assert np.array_equal(a[ok], b)


def test_norm_refuses_wrong_tensors(rz):
    x, d, gamma = (dev(a) for a in norm_inputs(2, 64, 64, 1))
    with pytest.raises(ValueError):
        rz.residual_rmsnorm(x, d[:1], gamma, 64, 64, 1e-6)
    with pytest.raises(ValueError):
        rz.residual_rmsnorm(x.t().contiguous().t(), d, gamma, 64, 64, 1e-6)
    with pytest.raises(TypeError):
        rz.residual_rmsnorm(x.double(), d, gamma, 64, 64, 1e-6)
    with pytest.raises(ValueError):
        rz.residual_rmsnorm(x, d, gamma[:63], 64, 64, 1e-6)
    with pytest.raises(TypeError):
        rz.residual_rmsnorm(x.cpu(), d, gamma, 64, 64, 1e-6)
    with pytest.raises(rz.RzError):
        rz.residual_rmsnorm(x, d, gamma, 64, 64, -1.0)


# ---------------------------------------------------------------- routing
def check_route(rz, logits, k, renorm, scale=1.0, row_seq=None, plan=None, ld=None):
    T, E = logits.shape
    plan = plan or rz.MoePlan(T, E, k)
    plan.rows.fill_(12345)
    t = dev(logits)
    if ld:
        wide = torch.full((T, ld), 1e9, device="cuda")
        wide[:, :E] = t
        t = wide[:, :E]
    rz.moe_route(t, plan, renormalise=renorm, scale=scale, row_seq=None if row_seq is None else dev(row_seq))
    e, w, off, rows, places = R.route(logits, k, renorm, scale, row_seq)
    assert np.array_equal(host(plan.experts), e)
    assert np.array_equal(host(plan.offsets), off) and np.array_equal(host(plan.rows), rows) and np.array_equal(host(plan.places), places)
    got = host(plan.weights).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(w))
    # exp within 2 ulp of a difference rounded once (relative 2^-24 |logit - top|, at most 100 here), sums of up to 512
    # such in f32 (4 a lane in turn, 5 halvings: 21 roundings), a division and a product
    ok = ~np.isnan(w)
    assert np.all(np.abs(got[ok] - w[ok]) <= (2 * (4 + 100) + 21 + 2) * 2.0 ** -24 * np.abs(w[ok]) + 1e-44)
    return plan


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 8, 2), (16, 65, 6), (17, 128, 8), (129, 32, 32), (200, 512, 32), (512, 16, 3),
                                   (513, 512, 32), (1000, 128, 8), (4097, 8, 2), (9000, 33, 5), (70, 256, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(rz, T, E, k, renorm):
    rng = np.random.default_rng(T + E)
    logits = (3 * rng.normal(size=(T, E))).astype(np.float32)
    check_route(rz, logits, k, renorm, 1.0 if renorm else 2.5)
    # ties, zeros of both signs
    check_route(rz, np.round(logits).astype(np.float32) * np.where(rng.random((T, E)) < 0.5, -1, 1).astype(np.float32), k, renorm)


@pytest.mark.parametrize("T", [6, 300])
def test_route_masks(rz, T):
    rng = np.random.default_rng(T)
    E, k = 40, 4
    logits = rng.normal(size=(T, E)).astype(np.float32)
    logits[rng.random((T, E)) < 0.8] = -np.inf
    logits[0] = -np.inf              # nothing left
    logits[1, :] = -np.inf
    logits[1, 39] = -3e38            # one left, next to the lowest number
    logits[2, 3] = np.nan
    logits[3, :3] = [np.nan, 2, np.inf]
    logits[4] = np.nan
    row_seq = np.where(rng.random(T) < 0.3, -1, 7).astype(np.int32)
    row_seq[:5] = 0
    row_seq[5] = -5
    logits[5] = np.nan               # not read
    for renorm in (True, False):
        check_route(rz, logits, k, renorm, row_seq=row_seq)
    check_route(rz, logits, k, True, row_seq=np.full(T, -1, np.int32))


def test_route_strided_logits_and_used_plan(rz):
    rng = np.random.default_rng(1)
    plan = None
    for _ in range(3):
        plan = check_route(rz, rng.normal(size=(150, 16)).astype(np.float32), 3, True, plan=plan, ld=37)


# ---------------------------------------------------------------- products
def q4k(rng, *shape, in_dim, spread=0.0):
    nb = in_dim // 256
    w = rng.integers(0, 256, (*shape, nb, 144), dtype=np.uint8)
    grow = np.exp(rng.uniform(-spread, spread, (*shape, nb)))
    for at in (0, 2):
        w[..., at:at + 2] = (rng.uniform(1e-3, 1e-2, (*shape, nb)) * grow).astype(np.float16)[..., None].view(np.uint8)
    return w


def activations(rng, m, n, spread=0.0):
    x = rng.normal(size=(m, n)).astype(np.float32)
    x = (x.reshape(m, -1, 32) * np.exp(rng.uniform(-spread, spread, (m, n // 32, 1)))).reshape(m, n).astype(np.float32)
    return R.q8_quantize(x)


def make_plan(rz, rng, T, E, k, skew=1.0, idle=0.1):
    logits = (rng.normal(size=(T, E)) + skew * rng.normal(size=E)).astype(np.float32)
    row_seq = np.where(rng.random(T) < idle, -1, 1).astype(np.int32)
    plan = rz.MoePlan(T, E, k)
    rz.moe_route(dev(logits), plan, row_seq=dev(row_seq))
    return plan, R.experts_of(host(plan.offsets), T * k)


def within(got, ref, tol, what):
    bad = ~(np.abs(got.astype(np.float64) - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.max(np.abs(got - ref) / tol)))


SHAPES = [  # T, E, k, inter, in
    (1, 1, 1, 1, 256), (1, 8, 3, 33, 256), (2, 4, 4, 32, 512), (5, 3, 2, 100, 768), (9, 2, 2, 160, 2304), (17, 64, 8, 64, 256),
    (33, 4, 1, 129, 512), (40, 3, 3, 256, 1024), (130, 8, 2, 130, 256), (150, 2, 2, 320, 512), (300, 16, 4, 96, 256), (270, 1, 1, 200, 768),
    (64, 32, 2, 640, 256), (240, 8, 1, 2600, 256), (1700, 8, 1, 2560, 512),  # more tiles than SMs, for each of the tiles' sizes
    (7, 8, 2, 65, 1280), (6, 16, 1, 40, 2560), (9, 256, 32, 32, 256),
    (40, 8, 2, 2208, 512), (17, 2, 1, 3001, 1280), (100, 64, 2, 1024, 256), (10, 4, 4, 2000, 1536),  # tiles of 16 rows: many outputs
]


@pytest.mark.parametrize("T,E,k,inter,in_dim", SHAPES)
def test_swiglu(rz, T, E, k, inter, in_dim):
    rng = np.random.default_rng(T * E + inter)
    plan, expert = make_plan(rz, rng, T, E, k)
    # f16 scales of gate and up that keep silu in its curved part
    gate, up = q4k(rng, E, inter, in_dim=in_dim, spread=1.0), q4k(rng, E, inter, in_dim=in_dim, spread=1.0)
    q, d, s = activations(rng, T, in_dim, 2.0)
    d = (d * np.float32(0.01)).astype(np.float32)
    s = (s * np.float32(0.01)).astype(np.float32)  # both as a user's own quantiser may scale them: s and d * sum(q) agree to 2^-23
    out = torch.full((T * k, inter), 7.5, device="cuda")
    with_q8 = inter % 32 == 0
    q8 = torch.full((rz.q8_1_size(T * k, inter),), 99, dtype=torch.uint8, device="cuda") if with_q8 else None
    rz.moe_swiglu(dev(gate), dev(up), dev(R.q8_buffer(q, d, s)), plan, inter, in_dim, out=out, out_q8=q8)
    x = R.q8_values(q, d)
    h, tol = R.swiglu(R.weights(gate), R.weights(up), x, host(plan.rows), expert, k)
    # s enters as it is given: off from d * sum(q) by 2^-23 of it
    got, live = host(out), expert >= 0
    within(got[live], h[live], 1.2 * tol[live], "h")
    assert np.all(got[~live] == 7.5)
    if with_q8:
        qr, dr, sr = R.q8_quantize(got)
        qg, dg, sg = R.q8_parts(host(q8), T * k, inter)
        for a, b in ((qr, qg), (dr, dg), (sr, sg)):
            assert np.array_equal(a[live], b[live])
        assert np.all(qg[~live].view(np.uint8) == 99)
        only = torch.empty_like(q8)
        assert rz.moe_swiglu(dev(gate), dev(up), dev(R.q8_buffer(q, d, s)), plan, inter, in_dim, out_q8=only, want_h=False) is None
        assert np.array_equal(R.q8_parts(host(only), T * k, inter)[0][live], qg[live])


@pytest.mark.parametrize("T,E,k,out_dim,in_dim", SHAPES)
def test_down(rz, T, E, k, out_dim, in_dim):
    rng = np.random.default_rng(T * E + out_dim + 1)
    plan, expert = make_plan(rz, rng, T, E, k)
    w = q4k(rng, E, out_dim, in_dim=in_dim, spread=1.0)
    q, d, s = activations(rng, T * k, in_dim, 2.0)
    pad = out_dim + 8 + T % 3
    res = rng.normal(size=(T, pad)).astype(np.float32)
    ref, tol = R.down(R.weights(w), R.q8_values(q, d), host(plan.places), expert, host(plan.weights).astype(np.float64), res[:, :out_dim])
    args = (dev(w), dev(R.q8_buffer(q, d, s)), plan, out_dim, in_dim)
    y = rz.moe_down(*args, residual=dev(res), out_pad=pad)
    within(host(y)[:, :out_dim], ref, tol, "y")
    assert np.all(host(y)[:, out_dim:] == 0)
    inplace = dev(res)
    assert rz.moe_down(*args, residual=inplace, out=inplace, out_pad=pad) is inplace and torch.equal(inplace, y)
    none = host(rz.moe_down(*args))
    idle = (host(plan.experts) < 0).all(-1)
    assert none.shape == (T, out_dim) and np.all(none[idle] == 0)
    ref0, tol0 = R.down(R.weights(w), R.q8_values(q, d), host(plan.places), expert, host(plan.weights).astype(np.float64), None)
    within(none, ref0, tol0, "y without a residual")


PARTS = [  # few tiles and a long in_dim: 4 to 19 super-blocks, in parts of equal and unequal lengths
    (60, 4, 2, 300, 1024), (33, 8, 2, 1000, 4864), (65, 16, 4, 130, 2304), (60, 2, 1, 257, 2816), (200, 1, 1, 700, 2560), (130, 1, 1, 1, 1280),
    (52, 4, 1, 2049, 1792),
]


@pytest.mark.parametrize("T,E,k,out_dim,in_dim", PARTS)
def test_down_in_parts(rz, T, E, k, out_dim, in_dim):
    test_down(rz, T, E, k, out_dim, in_dim)


def test_down_parts_workspace(rz):
    """Nothing behind the workspace is written, nothing of an earlier call is read, and every call gives the same bits."""
    rng = np.random.default_rng(77)
    T, E, k, out_dim, in_dim = 33, 8, 2, 1000, 4864
    plan, _ = make_plan(rz, rng, T, E, k)
    args = (dev(q4k(rng, E, out_dim, in_dim=in_dim, spread=1.0)), dev(R.q8_buffer(*activations(rng, T * k, in_dim, 2.0))), plan, out_dim, in_dim)
    size = rz.moe_down_workspace_bytes(T, E, k, out_dim, in_dim)
    room = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    first = rz.moe_down(*args, ws=room[:size])
    for fill in (0, 127, 255):
        room.fill_(fill)
        assert torch.equal(rz.moe_down(*args, ws=room[:size]), first)
        assert torch.all(room[size:] == fill)
    res = torch.randn(T, out_dim, device="cuda")
    rz.moe_route(torch.zeros(T, E, device="cuda"), plan, row_seq=torch.full((T,), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(rz.moe_down(*args, residual=res, ws=room[:size]), res)  # no row at all


@pytest.mark.parametrize("T,inter", [(3, 64), (9, 2240), (90, 64), (200, 64)])  # integer dots, and tiles of 16, 32 and 128 rows
def test_products_of_extreme_blocks(rz, T, inter):
    """Super-blocks without a scale, without a min, with mins far above or below the scale; blocks of x far apart."""
    rng = np.random.default_rng(T)
    E, k, in_dim = 2, 2, 1024
    plan, expert = make_plan(rz, rng, T, E, k, idle=0.0)
    w = q4k(rng, E, inter, in_dim=in_dim)
    d, dmin = w[..., 0:2].view(np.float16)[..., 0], w[..., 2:4].view(np.float16)[..., 0]
    d[:, 0::8], dmin[:, 1::8] = 0, 0
    d[:, 2::8], dmin[:, 3::8] = np.float16(6e-8), np.float16(6e-8)       # the least f16
    d[:, 4::8], dmin[:, 5::8] = np.float16(900.0), np.float16(900.0)
    d[:, 6::8] *= -1
    d[:, 7::8] = 0
    dmin[:, 7::8] = 0
    q, dd, s = activations(rng, T, in_dim, 12.0)
    out = host(rz.moe_swiglu(dev(w), dev(w), dev(R.q8_buffer(q, dd, s)), plan, inter, in_dim))
    wv = R.weights(w)
    h, tol = R.swiglu(wv, wv, R.q8_values(q, dd), host(plan.rows), expert, k)
    fine = np.abs(h) < 1e37
    within(out[fine], h[fine], 1.2 * tol[fine], "h")


def test_values_that_are_no_numbers_stay_in_their_rows(rz):
    rng = np.random.default_rng(11)
    for T, out_dim in ((4, 70), (31, 2600), (140, 70), (620, 70)):  # integer dots, and tiles of 16, 32 and 128 rows
        E, k, in_dim = 3, 1, 512
        plan, expert = make_plan(rz, rng, T, E, k, idle=0.0)
        w = q4k(rng, E, out_dim, in_dim=in_dim)
        q, d, s = activations(rng, T, in_dim)
        args = dev(R.q8_buffer(q, d, s)), plan, out_dim, in_dim
        before = host(rz.moe_down(dev(w), *args))
        bad = w.copy()
        bad[1, 33, 0, 0:2] = np.float16(np.nan).reshape(1).view(np.uint8)
        y = host(rz.moe_down(dev(bad), *args))
        meets = host(plan.experts)[:, 0] == 1
        assert np.isnan(y[meets, 33]).all()
        keep = np.ones_like(y, bool)
        keep[meets, 33] = False
        assert np.array_equal(y[keep], before[keep])
        d2, s2 = d.copy(), s.copy()
        d2[1, 3], s2[1, 3] = np.nan, np.nan
        hq = dev(R.q8_buffer(q, d2, s2))
        y = host(rz.moe_down(dev(w), hq, plan, out_dim, in_dim))
        token = int(np.where(host(plan.places) == 1)[0][0])
        assert np.isnan(y[token]).all()
        others = np.arange(T) != token
        assert np.array_equal(y[others], before[others])


def test_bad_plans_are_reported(rz):
    rng = np.random.default_rng(2)
    for T, E in ((3, 8), (4, 4), (200, 4)):
        k, out_dim, in_dim = 2, 64, 256
        plan, _ = make_plan(rz, rng, T, E, k, idle=0.0)
        w, x = dev(q4k(rng, E, out_dim, in_dim=in_dim)), dev(R.q8_buffer(*activations(rng, T, in_dim)))
        h8 = dev(R.q8_buffer(*activations(rng, T * k, in_dim)))
        ref = rz.moe_swiglu(w, w, x, plan, out_dim, in_dim)
        y = rz.moe_down(w, h8, plan, out_dim, in_dim)
        good = plan.rows.clone()
        plan.rows[1] = T * k
        plan.rows[2] = -1
        h = rz.moe_swiglu(w, w, x, plan, out_dim, in_dim)
        st, code = rz.check_device_error()
        assert st == 7 and code == 0x203
        assert torch.equal(h[3:], ref[3:]) and torch.equal(h[0], ref[0])
        plan.rows.copy_(good)
        at = int(plan.places[0])
        plan.places[0] = T * k
        rz.moe_down(w, h8, plan, out_dim, in_dim)
        st, code = rz.check_device_error()
        assert st == 7 and code == 0x203
        plan.places[0] = at
        off = plan.offsets.clone()
        last = int((off[1:] > off[:-1]).nonzero()[-1])
        plan.offsets[last + 1:] = T * k + 5  # the last rows end outside
        out = torch.full_like(ref, 3.0)
        rz.moe_swiglu(w, w, x, plan, out_dim, in_dim, out=out)
        first = int(off[last])
        assert torch.equal(out[:first], ref[:first]) and bool((out[first:] == 3.0).all())
        plan.offsets.copy_(off)
        rz.check_device_error()
        assert torch.equal(rz.moe_down(w, h8, plan, out_dim, in_dim), y)


def test_no_rows(rz):
    plan = rz.MoePlan(3, 4, 2)
    rz.moe_route(torch.randn(3, 4, device="cuda"), plan, row_seq=torch.full((3,), -1, dtype=torch.int32, device="cuda"))
    rng = np.random.default_rng(1)
    w = dev(q4k(rng, 4, 64, in_dim=256))
    out = torch.full((6, 64), 2.0, device="cuda")
    rz.moe_swiglu(w, w, dev(R.q8_buffer(*activations(rng, 3, 256))), plan, 64, 256, out=out)
    assert bool((out == 2.0).all())
    res = torch.randn(3, 64, device="cuda")
    y = rz.moe_down(w, dev(R.q8_buffer(*activations(rng, 6, 256))), plan, 64, 256, residual=res)
    assert torch.equal(y, res)


# ---------------------------------------------------------------- together
class Block:
    """An FFN of experts of random weights, as a caller keeps it."""

    def __init__(self, rz, T, E, k, n, n_pad, inter, seed):
        rng = np.random.default_rng(seed)
        self.rz, self.T, self.E, self.k, self.n, self.n_pad, self.inter = rz, T, E, k, n, n_pad, inter
        self.gate, self.up, self.down = q4k(rng, E, inter, in_dim=n_pad), q4k(rng, E, inter, in_dim=n_pad), q4k(rng, E, n, in_dim=inter)
        self.gamma, self.router = rng.uniform(0.001, 0.003, n).astype(np.float32), rng.normal(size=(E, n_pad)).astype(np.float32) * 50
        self.d = {k: dev(v) for k, v in (("gate", self.gate), ("up", self.up), ("down", self.down), ("gamma", self.gamma), ("router", self.router))}
        self.plan = rz.MoePlan(T, E, k)
        self.h8 = torch.empty(rz.q8_1_size(T * k, inter), dtype=torch.uint8, device="cuda")
        self.ws = rz.workspace(max(rz.moe_down_workspace_bytes(T, E, k, n, inter), rz.moe_swiglu_workspace_bytes(T, E, k, n_pad),
                                   rz.moe_route_workspace_bytes(T, E)), "cuda")
        self.h8.zero_()

    def run(self, x, delta, seq):
        rz = self.rz
        s, y, q8 = rz.residual_rmsnorm(x, delta, self.d["gamma"], self.n, self.n_pad, 1e-6)
        rz.moe_route(y @ self.d["router"].t(), self.plan, row_seq=seq, ws=self.ws)
        rz.moe_swiglu(self.d["gate"], self.d["up"], q8, self.plan, self.inter, self.n_pad, out_q8=self.h8, want_h=False, ws=self.ws)
        return rz.moe_down(self.d["down"], self.h8, self.plan, self.n, self.inter, residual=s, out_pad=self.n_pad, ws=self.ws)

    def reference(self, x, delta, plan, h8):
        """From the sum, the plan and the quantised h as they are on the GPU (their codes may turn on an ulp of h)."""
        s, y = norm_reference(x, delta, self.gamma, self.n, 1e-6)
        q, d, _ = R.q8_quantize(y.astype(np.float32), multiplied=True)
        expert = R.experts_of(host(plan.offsets), self.T * self.k)
        h, tol = R.swiglu(R.weights(self.gate), R.weights(self.up), R.q8_values(q, d), host(plan.rows), expert, self.k)
        hq, hd, _ = R.q8_parts(h8, self.T * self.k, self.inter)
        live = expert >= 0
        # what is held of h is within half a step, and what h may be off
        held = R.q8_values(hq, hd)
        within(held[live], h[live], 1.2 * tol[live] + np.repeat(hd[live], 32, -1) * (0.5 + 1e-3), "held h")
        w = host(plan.weights).astype(np.float64)
        return R.down(R.weights(self.down), held, host(plan.places), expert, w, s[:, :self.n])


@pytest.mark.parametrize("T,E,k,n,n_pad,inter", [(1, 8, 2, 200, 256, 256), (7, 4, 3, 512, 512, 512), (33, 16, 4, 900, 1024, 256), (160, 4, 2, 256, 256, 768)])
def test_block(rz, T, E, k, n, n_pad, inter):
    b = Block(rz, T, E, k, n, n_pad, inter, T)
    rng = np.random.default_rng(T + 1)
    x, delta = rng.normal(size=(2, T, n_pad)).astype(np.float32)
    x[:, n:], delta[:, n:] = 0, 0
    seq = np.where(rng.random(T) < 0.2, -1, 0).astype(np.int32)
    y = host(b.run(dev(x), dev(delta), dev(seq)))
    ref, tol = b.reference(x, delta, b.plan, host(b.h8))
    within(y[:, :n], ref, tol, "y")
    assert np.all(y[:, n:] == 0)


@pytest.mark.parametrize("T,E,k,n,n_pad,inter", [(1, 8, 2, 200, 256, 256), (7, 4, 3, 512, 512, 512), (130, 16, 4, 900, 1024, 256), (160, 4, 2, 256, 256, 768),
                                                 (300, 3, 1, 130, 256, 256)])
def test_ffn_is_its_steps(rz, T, E, k, n, n_pad, inter):
    b = Block(rz, T, E, k, n, n_pad, inter, T + 3)
    rng = np.random.default_rng(T + 1)
    logits, res = dev(rng.normal(size=(T, E)).astype(np.float32)), dev(rng.normal(size=(T, n_pad)).astype(np.float32))
    seq = dev(np.where(rng.random(T) < 0.2, -1, 0).astype(np.int32))
    q8 = dev(R.q8_buffer(*activations(rng, T, n_pad)))
    d = b.d
    for renorm, scale, r in ((True, 1.0, res), (False, 2.5, None)):
        rz.moe_route(logits, b.plan, renormalise=renorm, scale=scale, row_seq=seq)
        h8 = torch.zeros_like(b.h8)
        h = rz.moe_swiglu(d["gate"], d["up"], q8, b.plan, inter, n_pad, out_q8=h8)
        live = R.experts_of(host(b.plan.offsets), T * k) >= 0
        assert np.array_equal(R.q8_quantize(host(h)[live])[0], R.q8_parts(host(h8), T * k, inter)[0][live])
        want = rz.moe_down(d["down"], h8, b.plan, n, inter, residual=r, out_pad=n_pad)
        plan = rz.MoePlan(T, E, k)
        got = rz.moe_ffn(logits, q8, d["gate"], d["up"], d["down"], plan, n, n_pad, inter, renormalise=renorm, scale=scale, row_seq=seq, residual=r)
        assert torch.equal(got, want)
        for name in ("experts", "weights", "offsets", "rows", "places"):
            assert torch.equal(getattr(plan, name), getattr(b.plan, name)), name
    out = res.clone()
    rz.moe_route(logits, b.plan, row_seq=seq)
    want = rz.moe_ffn(logits, q8, d["gate"], d["up"], d["down"], plan, n, n_pad, inter, row_seq=seq, residual=res)
    ws = rz.workspace(rz.moe_ffn_workspace_bytes(T, E, k, n, n_pad, inter), "cuda")
    ws.fill_(255)
    assert rz.moe_ffn(logits, q8, d["gate"], d["up"], d["down"], plan, n, n_pad, inter, row_seq=seq, residual=out, out=out, ws=ws) is out
    assert torch.equal(out, want)


def test_block_in_a_graph_and_on_another_stream(rz):
    T, E, k, n, inter = 37, 8, 2, 512, 256
    b = Block(rz, T, E, k, n, n, inter, 5)
    ins = [torch.randn(2, T, n, device="cuda") for _ in range(3)]
    seqs = [torch.where(torch.rand(T, device="cuda") < 0.3, -1, 0).int() for _ in range(3)]
    eager = [b.run(i[0], i[1], s).clone() for i, s in zip(ins, seqs)]
    x, seq = ins[0].clone(), seqs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            b.run(x[0], x[1], seq)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.run(x[0], x[1], seq)
    for i, s, want in list(zip(ins, seqs, eager)) * 2:
        x.copy_(i)
        seq.copy_(s)
        g.replay()
        assert torch.equal(out, want)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        got = b.run(ins[1][0], ins[1][1], seqs[1])
    side.synchronize()
    assert torch.equal(got, eager[1])


def test_two_streams_at_once(rz):
    """Calls that share weights and input, each with its own plan, workspace and outputs."""
    rng = np.random.default_rng(3)
    T, E, k, n, inter = 33, 8, 2, 1024, 2048
    gate, up, down = (dev(q4k(rng, E, *s, in_dim=i)) for s, i in (((inter,), n), ((inter,), n), ((n,), inter)))
    x8, logits = dev(R.q8_buffer(*activations(rng, T, n))), torch.randn(4, T, E, device="cuda")
    plans = [rz.MoePlan(T, E, k) for _ in logits]
    run = lambda i: rz.moe_ffn(logits[i], x8, gate, up, down, plans[i], n, n, inter)
    want = [run(i).clone() for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i in range(4):
            with torch.cuda.stream(streams[i % 2]):
                got.append(run(i))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[j % 4]) for j, g in enumerate(got))
    assert rz.check_device_error() == (0, 0)


def test_two_graphs_share_a_workspace(rz):
    """Replayed one after another; the smaller call leaves what the larger one must not read."""
    rng = np.random.default_rng(4)
    E, k, n, inter = 8, 2, 1024, 2048
    gate, up, down = (dev(q4k(rng, E, *s, in_dim=i)) for s, i in (((inter,), n), ((inter,), n), ((n,), inter)))
    sizes = (33, 3, 700)
    ws = rz.workspace(max(rz.moe_ffn_workspace_bytes(T, E, k, n, n, inter) for T in sizes), "cuda")
    graphs = []
    for T in sizes:
        args = torch.randn(T, E, device="cuda"), dev(R.q8_buffer(*activations(rng, T, n))), gate, up, down, rz.MoePlan(T, E, k), n, n, inter
        want = rz.moe_ffn(*args, ws=ws).clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = rz.moe_ffn(*args, ws=ws)
        graphs.append((g, out, want, args))
    for i in (0, 1, 2, 1, 0, 2, 2, 0):
        g, out, want, _ = graphs[i]
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert rz.check_device_error() == (0, 0)


def test_more_than_2_31_values(rz):
    rng = np.random.default_rng(5)
    T, E, k, out_dim, in_dim = 74900, 4, 2, 14400, 256
    plan, expert = make_plan(rz, rng, T, E, k, idle=0.0)
    w = q4k(rng, E, out_dim, in_dim=in_dim, spread=1.0)
    wv = R.weights(w)
    q, d, s = activations(rng, T, in_dim)
    d, s = (d * np.float32(0.01)).astype(np.float32), (s * np.float32(0.01)).astype(np.float32)
    h = rz.moe_swiglu(dev(w), dev(w), dev(R.q8_buffer(q, d, s)), plan, out_dim, in_dim)
    assert h.numel() > 2 ** 31 and expert[-1] >= 0
    some = np.array([0, 1, 74901, T * k - 129, T * k - 1])
    ref, tol = R.swiglu(wv, wv, R.q8_values(q, d), host(plan.rows)[some], expert[some], k)
    within(host(h[torch.from_numpy(some).cuda()]), ref, 1.2 * tol, "h")
    del h
    q, d, s = activations(rng, T * k, in_dim)
    y = rz.moe_down(dev(w), dev(R.q8_buffer(q, d, s)), plan, out_dim, in_dim)
    places = host(plan.places).reshape(T, k)
    some = np.array([0, T - 1, int(places.max(1).argmax()), 40000])
    ref, tol = R.down(wv, R.q8_values(q, d), places[some].reshape(-1), expert, host(plan.weights)[some].astype(np.float64), None)
    within(host(y[torch.from_numpy(some).cuda()]), ref, tol, "y")
    assert rz.check_device_error() == (0, 0)


@pytest.mark.parametrize("T,E,out_dim", [(20, 4, 2304), (60, 4, 384), (300, 2, 384)])
def test_wait_that_runs_out(rz, T, E, out_dim):
    """The first weights of CTA 0 are left uncopied: the product reports it, ends, and the next is as before."""
    rng = np.random.default_rng(T)
    k, in_dim = 2, 1024
    plan, _ = make_plan(rz, rng, T, E, k, idle=0.0)
    w, x = dev(q4k(rng, E, out_dim, in_dim=in_dim)), dev(R.q8_buffer(*activations(rng, T, in_dim)))
    want = rz.moe_swiglu(w, w, x, plan, out_dim, in_dim)
    assert rz.check_device_error() == (0, 0)
    rz.rz_debug_stall_next_moe(1 << 12)
    got = rz.moe_swiglu(w, w, x, plan, out_dim, in_dim)
    assert rz.check_device_error() == (5, 0x120)
    # the first item is the first expert's first tile; other CTAs' outputs are whole
    assert torch.equal(got[:, 128:], want[:, 128:])
    for _ in range(3):
        assert torch.equal(rz.moe_swiglu(w, w, x, plan, out_dim, in_dim), want)
    assert rz.check_device_error() == (0, 0)


def test_stall_limit_is_checked_on_the_host(rz):
    from quantized_q4_q8_gb300 import _lib
    assert _lib.status("rz_debug_stall_next_moe", 10) == 1
    assert _lib.status("rz_debug_stall_next_moe", 1 << 30) == 1
