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
