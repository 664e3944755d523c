"""Host-side checks of the paged 4-bit cache at its limits (no GPU: no refused call gets that far)."""
import numpy as np
import pytest

import paged_reference as R
from test_paged_host import ATT, HEADS, kv, lib  # noqa: F401


@pytest.mark.parametrize("heads", [1 << 24, 1 << 30, 65536 + 2])
def test_attention_refuses_rows_beyond_32_bits(lib, heads):
    """2^24 heads of 128 are 2^31 values a row, which the kernels count in 32 bits."""
    a = {**ATT, "kv": kv(lib, hd=128), "H": heads, "ld_q": heads * 128, "n": 1}
    assert lib.status("rz_attention_paged_q4", *a.values()) == 2 and "n_heads" in lib.last_error()
    assert lib.load().rz_attention_paged_q4_workspace_bytes(heads, 2, 128) == 0 and "n_heads" in lib.last_error()


def test_heads_refuses_as_many(lib):
    a = {**HEADS, "kv": kv(lib), "H": 65537, "ld_q": 1 << 30, "ld_qo": 1 << 30}
    assert lib.status("rz_qk_norm_rope", *a.values()) == 2 and "n_heads" in lib.last_error()


def test_heads_in_place_needs_one_row_stride(lib):
    """Rows written at another stride would run into rows that are still to be read."""
    a = {**HEADS, "kv": kv(lib), "ld_qo": 512}
    assert lib.status("rz_qk_norm_rope", *a.values()) == 2 and "ld_qo" in lib.last_error()


def carried(torch, rz, cached, fresh, w):
    plan = rz.PagedPlan(len(cached), 8, "cpu")
    plan.kv_len.copy_(torch.from_numpy(w["kv_len"]))
    c, f = (torch.from_numpy(np.asarray(x, np.int32)) for x in (cached, fresh))
    new = plan.next_cached(c, f)
    assert plan.next_cached(c, f, out=c) is c and torch.equal(c, new)
    return new.numpy()


def test_lengths_carried_over_a_refusing_step():
    """A request that a step refuses goes on where it was, as soon as there are pages again."""
    torch = pytest.importorskip("torch")
    import quantized_q4_q8_gb300 as rz
    cached, owned = np.array([16, 16, 32], np.int32), np.array([1, 1, 2], np.int32)
    table, free, count = np.array([[0, -1, -1], [1, -1, -1], [2, 3, -1]], np.int32), np.full(5, -9, np.int32), 1
    free[0] = 4
    w = R.plan(cached, np.array([1, 2, 0]), owned, table, free, count, 16, 8)
    assert w["refused"] and list(w["kv_len"]) == [17, 0, 32] and list(w["positions"][:3]) == [16, -1, -1]
    cached = carried(torch, rz, cached, [1, 2, 0], w)
    assert list(cached) == [17, 16, 32]
    for news, want, positions in (([0, 0, -1], [17, 16, 0], []), ([1, 2, 0], [18, 18, 0], [17, 16, 17])):
        w = R.plan(cached, np.array(news), w["owned"], w["table"], w["free"], w["count"], 16, 8)
        assert not w["refused"] and not w["bad"]
        cached = carried(torch, rz, cached, news, w)
        assert list(cached) == want and list(w["positions"][:len(positions)]) == positions


def test_bad_lengths_are_carried_as_they_are():
    torch = pytest.importorskip("torch")
    import quantized_q4_q8_gb300 as rz
    assert list(carried(torch, rz, [-4, 5, 0], [1, -1, 0], {"kv_len": np.zeros(3, np.int32)})) == [-4, 0, 0]
