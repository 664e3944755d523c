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
