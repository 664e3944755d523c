"""The operators of an FFN of experts on the GPU at their edges: plans that no routing makes, weights and activations whose parts are
far apart or no numbers, waits that run out."""
import numpy as np
import pytest

import moe_reference as R
from test_gpu_moe import activations, dev, host, make_plan, q4k, rz, within  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# rows, experts, outputs: tiles of 16, 32 and 128 rows for both products (of in_dim 512)
TILES = [(80, 8, 2208), (400, 8, 640), (1536, 8, 384)]


def one_expert(rz, n, E, offsets):
    """A plan of n tokens of one choice, expert 0, and the offsets given."""
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    return rz.MoePlan(n, E, 1, experts=torch.zeros(n, 1, dtype=torch.int32, device="cuda"), weights=torch.ones(n, 1, device="cuda"),
                      offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), rows=ids, places=ids.clone())


def in_the_middle(size):
    """(a buffer, a workspace of `size` bytes inside it): 4 MB before and behind."""
    room = torch.empty((8 << 20) + size, dtype=torch.uint8, device="cuda")
    return room, room[4 << 20:(4 << 20) + size]


@pytest.mark.parametrize("n,E,out_dim", TILES)
def test_overlapping_offsets(rz, n, E, out_dim):
    """Every other expert has all rows, more tiles than the workspace holds; with the same weights for each the values are those
    of one expert, whatever lies around the workspace."""
    rng = np.random.default_rng(n)
    in_dim = 512
    w = dev(np.repeat(q4k(rng, 1, out_dim, in_dim=in_dim), E, 0))
    x = dev(R.q8_buffer(*activations(rng, n, in_dim)))
    plain, over = (one_expert(rz, n, E, o) for o in ([0] + [n] * E, [0, n] * (E // 2) + [0]))
    h, y = rz.moe_swiglu(w, w, x, plain, out_dim, in_dim), rz.moe_down(w, x, plain, out_dim, in_dim)
    room, ws = in_the_middle(rz.moe_swiglu_workspace_bytes(n, E, 1, in_dim))
    room2, ws2 = in_the_middle(rz.moe_down_workspace_bytes(n, E, 1, out_dim, in_dim))
    assert ws.numel() and ws2.numel()
    for fill in (0, 127, 255):
        room.fill_(fill)
        room2.fill_(fill)
        assert torch.equal(rz.moe_swiglu(w, w, x, over, out_dim, in_dim, ws=ws), h)
        assert torch.equal(rz.moe_down(w, x, over, out_dim, in_dim, ws=ws2), y)
        for r in (room, room2):
            assert bool((r[:4 << 20] == fill).all()) and bool((r[-(4 << 20):] == fill).all())
    assert rz.check_device_error() == (0, 0)


# rows, experts, choices, outputs: integer dots, then tiles of 16, 32 and 128 rows (of in_dim 512; parts of in_dim are the next)
DOWNS = [(5, 8, 2, 96, 512), (40, 8, 2, 2208, 512), (200, 8, 2, 640, 512), (800, 8, 2, 384, 512), (33, 8, 2, 1000, 4864)]


@pytest.mark.parametrize("T,E,k,out_dim,in_dim", DOWNS)
@pytest.mark.parametrize("bad", ["past the rows", "below 0", "decreasing", "a place of another expert", "no expert", "no place"])
def test_down_of_bad_plans(rz, T, E, k, out_dim, in_dim, bad):
    """An expert whose offsets are none has no rows, and a place that is not among its expert's is left out: both are reported, and
    nothing of the workspace shows."""
    rng = np.random.default_rng(T + 1)
    plan, expert = make_plan(rz, rng, T, E, k, idle=0.2)
    w = q4k(rng, E, out_dim, in_dim=in_dim)
    q, d, s = activations(rng, T * k, in_dim)
    res = rng.normal(size=(T, out_dim)).astype(np.float32)
    off, ids, places = host(plan.offsets).copy(), host(plan.experts).copy().reshape(-1), host(plan.places).copy()
    full = np.flatnonzero(np.diff(off))
    last, some = int(full[-1]), int(full[len(full) // 2])
    if bad == "past the rows":
        off[last + 1:] = T * k + 3
        lost = ids == last
    elif bad == "below 0":
        off[:full[0] + 1] = -1
        lost = ids == full[0]
    elif bad == "decreasing":
        off[some + 1:] = off[some] - 1  # `some` ends before it starts, those behind it have none
        lost = ids >= some
    else:
        lost = np.zeros(T * k, bool)
        pair = int(np.flatnonzero(ids == last)[-1])
        lost[pair] = True
        if bad == "a place of another expert":
            places[pair] = off[last] - 1
        elif bad == "no expert":
            ids[pair] = -1
        else:
            places[pair] = -1
    plan.offsets.copy_(dev(off))
    plan.experts.copy_(dev(ids).view(T, k))
    plan.places.copy_(dev(places))
    keep = np.where(lost, -1, host(plan.places))
    ref, tol = R.down(R.weights(w), R.q8_values(q, d), keep, expert, host(plan.weights).astype(np.float64), res)
    room, ws = in_the_middle(rz.moe_down_workspace_bytes(T, E, k, out_dim, in_dim))
    args = dev(w), dev(R.q8_buffer(q, d, s)), plan, out_dim, in_dim
    got = []
    for fill in (0, 127, 255):
        room.fill_(fill)
        got.append(rz.moe_down(*args, residual=dev(res), ws=ws if ws.numel() else None))
        assert rz.check_device_error() == (7, 0x203)
    within(host(got[0]), ref, tol, "y")
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ---------------------------------------------------------------- values that are no numbers
@pytest.mark.parametrize("T,inter", [(4, 256), (31, 2560), (140, 256), (620, 256)])  # integer dots, and tiles of 16, 32 and 128 rows
def test_no_number_reaches_the_q8_of_its_block(rz, T, inter):
    """One value of h is NaN: so are the scale and the sum of its block of 32, not those of the others, and what is made of it."""
    rng = np.random.default_rng(T)
    E, k, n = 3, 1, 512
    plan, expert = make_plan(rz, rng, T, E, k, idle=0.0)
    gate, up, down = q4k(rng, E, inter, in_dim=n), q4k(rng, E, inter, in_dim=n), q4k(rng, E, n, in_dim=inter)
    x = dev(R.q8_buffer(*activations(rng, T, n)))
    bad = gate.copy()
    bad[1, 33, 0, 0:2] = np.float16(np.nan).reshape(1).view(np.uint8)
    meets, block = expert == 1, np.arange(inter // 32) == 1
    assert meets.any()
    q8 = [torch.zeros(rz.q8_1_size(T, inter), dtype=torch.uint8, device="cuda") for _ in range(2)]
    h0 = host(rz.moe_swiglu(dev(gate), dev(up), x, plan, inter, n, out_q8=q8[0]))
    h1 = host(rz.moe_swiglu(dev(bad), dev(up), x, plan, inter, n, out_q8=q8[1]))
    keep = np.ones_like(h0, bool)
    keep[meets, 33] = False
    assert np.isnan(h1[~keep]).all() and np.array_equal(h1[keep], h0[keep])
    (q0, d0, s0), (q1, d1, s1) = (R.q8_parts(host(b), T, inter) for b in q8)
    hit = meets[:, None] & block
    assert np.isnan(d1[hit]).all() and np.isnan(s1[hit]).all()
    assert np.array_equal(d1[~hit], d0[~hit]) and np.array_equal(s1[~hit], s0[~hit])
    same = np.repeat(~hit, 32, -1)
    assert np.array_equal(q1[same], q0[same])
    # through the whole FFN, its tokens and no other
    logits = dev(np.where(np.arange(E) == host(plan.experts), 1, 0).astype(np.float32))
    out = [host(rz.moe_ffn(logits, x, dev(g), dev(up), dev(down), rz.MoePlan(T, E, k), n, n, inter)) for g in (gate, bad)]
    token = host(plan.experts)[:, 0] == 1
    assert np.isfinite(out[0]).all() and np.isnan(out[1][token]).all() and np.array_equal(out[1][~token], out[0][~token])


@pytest.mark.parametrize("m,n,n_pad", [(1, 96, 96), (3, 900, 1024), (2, 5000, 5120)])
def test_no_number_reaches_the_norms_q8(rz, m, n, n_pad):
    rng = np.random.default_rng(n)
    x, gamma = rng.normal(size=(m, n_pad)).astype(np.float32), rng.uniform(0.5, 1.5, n).astype(np.float32)
    bad = gamma.copy()
    bad[70] = np.nan
    (_, y0, b0), (_, y1, b1) = (rz.residual_rmsnorm(dev(x), None, dev(g), n, n_pad, 1e-6) for g in (gamma, bad))
    y0, y1, hit = host(y0), host(y1), np.arange(n_pad // 32) == 2
    assert np.isnan(y1[:, 70]).all() and np.array_equal(np.delete(y1, 70, 1), np.delete(y0, 70, 1))
    (q0, d0, s0), (q1, d1, s1) = (R.q8_parts(host(b), m, n_pad) for b in (b0, b1))
    assert np.isnan(d1[:, hit]).all() and np.isnan(s1[:, hit]).all()
    assert np.array_equal(d1[:, ~hit], d0[:, ~hit]) and np.array_equal(s1[:, ~hit], s0[:, ~hit])
    assert np.array_equal(q1[:, np.repeat(~hit, 32)], q0[:, np.repeat(~hit, 32)])


# ---------------------------------------------------------------- parts that are far apart
@pytest.mark.parametrize("T,inter", [(3, 64), (31, 2560), (90, 64), (640, 64)])  # integer dots, and tiles of 16, 32 and 128 rows
@pytest.mark.parametrize("d,dmin", [(2.0 ** -10, 9.0), (2.0 ** -14, 1.5), (3.1e-5, 33.0), (2.0 ** -14, 1000.0), (5e-7, 60.0), (1.2e-7, 8000.0),
                                    (6e-8, 8000.0), (-3.1e-5, 33.0), (3.1e-5, -33.0)])
@pytest.mark.parametrize("mins", ["none", "one", "all but one"])
def test_codes_beside_a_large_scale_of_the_mins(rz, T, inter, d, dmin, mins):
    """A scale of the mins 2^13 to 2^37 times the codes', where sub-blocks that x meets have no min: their codes are what a row is.  Usual
    rows stand between."""
    rng = np.random.default_rng(T + len(mins))
    E, k, in_dim = 3, 1, 512
    plan, expert = make_plan(rz, rng, T, E, k, idle=0.0)
    w = q4k(rng, E, inter, in_dim=in_dim)
    wide = np.arange(inter) % 5 != 4
    w[..., 0:2] = np.float16(d).reshape(1).view(np.uint8)
    w[..., 2:4] = w[..., 0:2]
    w[:, wide, :, 2:4] = np.float16(dmin).reshape(1).view(np.uint8)
    q, dd, _ = activations(rng, T, in_dim)
    blocks = q.reshape(T, -1, 32)
    at = np.arange(in_dim // 32)
    if mins == "all but one":  # sub-block 1 has none, and x is 0 elsewhere
        w[:, wide, :, 9] &= 0xc0
        blocks[:, at % 8 != 1] = 0
    else:  # the codes of the mins: bytes 8 to 11 and the upper halves of 12 to 15
        w[:, wide, :, 8:12] = 0
        w[:, wide, :, 12:16] &= 15
        if mins == "one":  # the least there is, in sub-block 2 of the second super-block, where x is 0
            w[:, wide, 1, 10] = 1
            blocks[:, at == 10] = 0
    dd = dd * np.float32(1 / (4000 * abs(float(np.float16(d)))))  # products of about 1
    s = (dd * blocks.astype(np.float32).sum(-1)).astype(np.float32)
    wv = R.weights(w)
    h, tol = R.swiglu(wv, wv, R.q8_values(q, dd), host(plan.rows), expert, k)
    out = host(rz.moe_swiglu(dev(w), dev(w), dev(R.q8_buffer(q, dd, s)), plan, inter, in_dim))
    within(out, h, tol, "h")


@pytest.mark.parametrize("n,E,out_dim", [(3, 8, 64)] + TILES)
def test_codes_beside_the_largest_scale_of_the_mins(rz, n, E, out_dim):
    """The least scale beside the largest: 2^40. What f16 steps cost is less than 2^-33 of the mins' scale for a weight."""
    rng = np.random.default_rng(n)
    in_dim, plan = 512, one_expert(rz, n, E, [0] + [n] * E)
    for d, dmin in ((6e-8, 65504.0), (1.2e-7, 40000.0), (0.0, 65504.0)):
        w = q4k(rng, 1, out_dim, in_dim=in_dim)
        w[..., 0:2], w[..., 2:4] = (np.float16(v).reshape(1).view(np.uint8) for v in (d, dmin))
        w[:, ::2, :, 8:12] = 0  # every other row without mins
        w[:, ::2, :, 12:16] &= 15
        q, dd, s = activations(rng, n, in_dim)
        x = R.q8_values(q, dd)
        ref, tol = R.down(R.weights(w), x, np.arange(n), np.zeros(n, int), np.ones((n, 1)), None)
        y = host(rz.moe_down(dev(np.repeat(w, E, 0)), dev(R.q8_buffer(q, dd, s)), plan, out_dim, in_dim))
        within(y, ref, tol + 2.0 ** -33 * dmin * np.abs(x).sum(-1, keepdims=True), (d, dmin))


def exact_gates(E, inter, in_dim):
    """(gate, up, g): with x one code of 1 in front, gate row i gives g[i] <= 0 and up gives 1, both without any rounding."""
    gate, up = np.zeros((2, E, inter, in_dim // 256, 144), np.uint8)
    i = np.arange(inter)
    sc, code = 1 + i % 63, 1 + i // 63 % 15
    gate[:, :, 0, 0:2] = np.float16(-0.125).reshape(1).view(np.uint8)
    up[:, :, 0, 0:2] = np.float16(1).reshape(1).view(np.uint8)
    gate[:, :, 0, 4], gate[:, :, 0, 16] = sc, code
    up[:, :, 0, 4], up[:, :, 0, 16] = 1, 1
    return gate, up, -0.125 * (sc * code).astype(np.float64)


def test_silu_of_exact_gates(rz):
    """Gates that are exact, -0.125 to -118, so that only silu rounds.  In half-ulps, integer dots: e^-g within 2 ulp (4), an addition, a
    division and the product with up (1 each); tensor cores: e^g within 2 ulp (4), its product with g and an addition (1 each), a division within
    2 ulp (4), the product with up (1).  The same for every row."""
    E, k, in_dim, inter = 3, 1, 256, 2560
    gate, up, g = exact_gates(E, inter, in_dim)
    with np.errstate(over="ignore"):
        ref = g / (1 + np.exp(-g))
    for T, half_ulps in ((2, 7), (31, 11), (90, 11), (640, 11)):  # integer dots, tiles of 16, 32 and 128 rows
        tol = half_ulps * 2.0 ** -24 * np.abs(ref) + 2.7e-37  # e^88.73 and more is infinite in f32, where silu is 88.73 / 2^128
        plan, _ = make_plan(rz, np.random.default_rng(T), T, E, k, idle=0.0)
        q, d = np.zeros((T, in_dim), np.int8), np.zeros((T, in_dim // 32), np.float32)
        q[:, 0], d[:, 0] = 1, 1
        out = host(rz.moe_swiglu(dev(gate), dev(up), dev(R.q8_buffer(q, d, d)), plan, inter, in_dim))
        assert np.array_equal(out, np.broadcast_to(out[0], out.shape))
        within(out, np.broadcast_to(ref, out.shape), np.broadcast_to(tol, out.shape), T)


# ---------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("T,E,out_dim", [(20, 4, 2304), (60, 4, 512), (300, 2, 512)])  # tiles of 16, 32 and 128 rows
def test_waits_that_run_out_before_other_outputs(rz, T, E, out_dim):
    """The same as with f32 outputs of gate and up, for their Q8_1 form and for the product back: reported, other CTAs' outputs whole, and
    the next calls as before."""
    rng = np.random.default_rng(T + 1)
    k, in_dim = 2, 1024
    plan, _ = make_plan(rz, rng, T, E, k, idle=0.0)
    w, x = dev(q4k(rng, E, out_dim, in_dim=in_dim)), dev(R.q8_buffer(*activations(rng, T, in_dim)))
    h8 = dev(R.q8_buffer(*activations(rng, T * k, in_dim)))
    q8 = torch.zeros(rz.q8_1_size(T * k, out_dim), dtype=torch.uint8, device="cuda")

    def gate_up():
        rz.moe_swiglu(w, w, x, plan, out_dim, in_dim, out_q8=q8, want_h=False)
        return q8[:T * k * out_dim].view(T * k, out_dim).clone()

    for run, first in ((gate_up, 128), (lambda: rz.moe_down(w, h8, plan, out_dim, in_dim), 256)):
        want = run()
        assert rz.check_device_error() == (0, 0)
        for limit in (1 << 10, 1 << 12, 1 << 14):
            rz.rz_debug_stall_next_moe(limit)
            got = run()
            assert rz.check_device_error() == (5, 0x120)
            assert torch.equal(got[:, first:], want[:, first:])
            for _ in range(2):
                assert torch.equal(run(), want)
        assert rz.check_device_error() == (0, 0)


@pytest.mark.parametrize("k", [1, 4, 8, 12, 16, 20])
@pytest.mark.parametrize("n,E,out_dim", [(3, 8, 64)] + TILES)
def test_small_blocks_beside_a_large_one(rz, n, E, out_dim, k):
    """Block 0 of each super-block of x has a scale 2^k times the others', and meets weights of 0.  On the tensor cores a value of the others is off
    by up to 2^(k - 24) of its block's largest: steps of 2^-24 where the largest scale is 1/2 .. 1."""
    rng = np.random.default_rng(n + k)
    in_dim, plan = 512, one_expert(rz, n, E, [0] + [n] * E)
    w = q4k(rng, 1, out_dim, in_dim=in_dim)
    w[..., 4] &= 0xc0
    w[..., 8] &= 0xc0
    q, d, _ = activations(rng, n, in_dim)
    d[:] = rng.uniform(0.5, 1, d.shape) * 2.0 ** -k
    d[:, ::8] = 1
    s = (d * q.reshape(n, -1, 32).astype(np.float32).sum(-1)).astype(np.float32)
    x, (wv, size) = R.q8_values(q, d), R.weights(w)
    ref, tol = R.down((wv, size), x, np.arange(n), np.zeros(n, int), np.ones((n, 1)), None)
    top = np.repeat(127 * d.astype(np.float64), 32, -1)  # of a block of 256 weights of 0 nothing counts
    y = host(rz.moe_down(dev(np.repeat(w, E, 0)), dev(R.q8_buffer(q, d, s)), plan, out_dim, in_dim))
    # the scale of a block may be half of 2^-k: once more
    within(y, ref, tol + (0 if n == 3 else 2 * 1.02 * 2.0 ** (k - 24)) * (top @ size[0].T), "y")
