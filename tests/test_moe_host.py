"""Host-side checks of the entry points of an FFN of experts: every refusal returns its
status and a message before any device work (no GPU here, and no pointer is one)."""
import ctypes as C

import numpy as np
import pytest

import moe_reference as R


@pytest.fixture(scope="module")
def lib():
    from quantized_q4_q8_gb300 import _lib
    from quantized_q4_q8_gb300.build import build
    build()
    _lib.load()
    return _lib


NORM = dict(x=16, delta=32, gamma=48, sum=64, y=80, q8=96, m=3, n=900, n_pad=1024, eps=1e-6, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(gamma=None), 1), (dict(y=None, q8=None), 1), (dict(m=0), 1), (dict(n=0), 1), (dict(n=1025), 1),
    (dict(m=(1 << 30) + 1), 2), (dict(n_pad=1000), 2), (dict(n_pad=16416), 6), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(y=64), 1), (dict(x=20), 3), (dict(delta=8), 3), (dict(gamma=4), 3), (dict(sum=40), 3), (dict(y=84), 3),
    (dict(q8=100), 3),
])
def test_norm_refusals(lib, change, status):
    st = lib.status("rz_residual_rmsnorm", *{**NORM, **change}.values())
    assert st == status and lib.last_error(), (st, lib.last_error())


PLAN = dict(experts=16, weights=32, offsets=48, rows=64, places=80, n_tokens=200, n_experts=8, top_k=2)
PLAN_CHANGES = [
    (dict(experts=None), 1), (dict(weights=None), 1), (dict(offsets=None), 1), (dict(rows=None), 1), (dict(places=None), 1),
    (dict(weights=18), 3), (dict(rows=65), 3), (dict(n_tokens=0), 1), (dict(n_tokens=1 << 27), 2), (dict(n_experts=0), 2),
    (dict(n_experts=513), 2), (dict(top_k=0), 2), (dict(top_k=9), 2), (dict(n_experts=64, top_k=33), 2),
]


def plan(lib, change):
    return C.byref(lib.MoePlanStruct(*{**PLAN, **change}.values()))


ROUTE = dict(logits=16, ld=8, row_seq=16, plan={}, renormalise=1, scale=1.0, ws=16, ws_bytes=1 << 20, stream=None)
SWIGLU = dict(gate=16, up=32, x=48, plan={}, inter=512, in_dim=256, h=64, h_q8=80, ws=96, ws_bytes=1 << 30, stream=None)
DOWN = dict(down=16, h=32, plan={}, residual=48, y=64, out_dim=100, out_pad=128, in_dim=512, ws=80, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("name,base", [("rz_moe_route", ROUTE), ("rz_moe_swiglu", SWIGLU), ("rz_moe_down", DOWN)])
@pytest.mark.parametrize("change,status", PLAN_CHANGES)
def test_plan_refusals(lib, name, base, change, status):
    st = lib.status(name, *{**base, "plan": plan(lib, change)}.values())
    assert st == status and lib.last_error(), (st, lib.last_error())
    st = lib.status(name, *{**base, "plan": None}.values())
    assert st == 1 and lib.last_error()


def refused(lib, name, base, change, status):
    a = {**base, **change}
    a["plan"] = plan(lib, a["plan"])
    st = lib.status(name, *a.values())
    assert st == status and lib.last_error(), (st, lib.last_error())


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(logits=18), 3), (dict(row_seq=17), 3), (dict(ld=7), 2), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(ws=None), 1), (dict(ws=24), 3), (dict(ws_bytes=16), 1),
])
def test_route_refusals(lib, change, status):
    refused(lib, "rz_moe_route", ROUTE, change, status)


@pytest.mark.parametrize("change,status", [
    (dict(gate=None), 1), (dict(up=None), 1), (dict(x=None), 1), (dict(h=None, h_q8=None), 1), (dict(inter=0), 2),
    (dict(inter=(1 << 20) + 1, h_q8=None), 2), (dict(inter=48), 2), (dict(in_dim=0), 2), (dict(in_dim=300), 2), (dict(in_dim=1 << 21), 2),
    (dict(gate=20), 3), (dict(up=8), 3), (dict(x=4), 3), (dict(h=72), 3), (dict(h_q8=88), 3), (dict(ws=None), 1), (dict(ws=88), 3), (dict(ws_bytes=200 * 1060 - 1), 1),
])
def test_swiglu_refusals(lib, change, status):
    refused(lib, "rz_moe_swiglu", SWIGLU, change, status)


@pytest.mark.parametrize("change,status", [
    (dict(down=None), 1), (dict(h=None), 1), (dict(y=None), 1), (dict(out_dim=0), 2), (dict(out_pad=99), 2),
    (dict(out_pad=1 << 21), 2), (dict(in_dim=0), 2), (dict(in_dim=100), 2), (dict(down=8), 3), (dict(h=36), 3), (dict(residual=52), 3),
    (dict(y=68), 3), (dict(ws=None), 1), (dict(ws=88), 3), (dict(ws_bytes=200 * 2 * 100 * 4 - 1), 1),
])
def test_down_refusals(lib, change, status):
    refused(lib, "rz_moe_down", DOWN, change, status)


FFN = dict(logits=16, ld=8, row_seq=16, x=16, gate=32, up=48, down=64, residual=80, out=96, plan={}, renormalise=1, scale=1.0, hidden=900,
           hidden_pad=1024, inter=512, ws=16, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(x=None), 1), (dict(gate=None), 1), (dict(up=None), 1), (dict(down=None), 1), (dict(out=None), 1),
    (dict(ld=7), 2), (dict(scale=float("nan")), 1), (dict(hidden=0), 2), (dict(hidden=1025), 2), (dict(hidden_pad=1000), 2), (dict(inter=500), 2),
    (dict(logits=18), 3), (dict(row_seq=18), 3), (dict(x=24), 3), (dict(gate=20), 3), (dict(down=8), 3), (dict(residual=88), 3), (dict(out=100), 3),
    (dict(ws=None), 1), (dict(ws=8), 3), (dict(ws_bytes=200 * 2 * 512), 1),
])
def test_ffn_refusals(lib, change, status):
    refused(lib, "rz_moe_ffn", FFN, change, status)


@pytest.mark.parametrize("change,status", PLAN_CHANGES)
def test_ffn_plan_refusals(lib, change, status):
    st = lib.status("rz_moe_ffn", *{**FFN, "plan": plan(lib, change)}.values())
    assert st == status and lib.last_error()


def test_workspace_sizes(lib):
    L = lib.load()
    assert L.rz_moe_route_workspace_bytes(16, 512) == 0 and not lib.last_error()
    assert L.rz_moe_route_workspace_bytes(17, 8) > 0
    assert L.rz_moe_route_workspace_bytes(0, 8) == 0 and lib.last_error()
    assert L.rz_moe_route_workspace_bytes(5, 600) == 0 and lib.last_error()
    assert L.rz_moe_swiglu_workspace_bytes(1, 64, 8, 2048) == 0 and not lib.last_error()
    assert L.rz_moe_swiglu_workspace_bytes(200, 8, 2, 512) >= 200 * 512 * 4
    assert L.rz_moe_swiglu_workspace_bytes(200, 8, 2, 100) == 0 and lib.last_error()
    assert L.rz_moe_down_workspace_bytes(1, 64, 8, 100, 512) == 0 and not lib.last_error()
    assert L.rz_moe_down_workspace_bytes(200, 8, 2, 100, 512) >= 200 * 2 * (100 * 4 + 512 * 4)
    assert L.rz_moe_down_workspace_bytes(200, 8, 0, 100, 512) == 0 and lib.last_error()
    assert L.rz_moe_down_workspace_bytes(200, 8, 2, 0, 512) == 0 and lib.last_error()
    assert L.rz_moe_down_workspace_bytes(200, 8, 2, 100, 500) == 0 and lib.last_error()
    assert L.rz_moe_ffn_workspace_bytes(1, 64, 8, 900, 1024, 512) >= 8 * 512 * 5 // 4 and not lib.last_error()
    assert L.rz_moe_ffn_workspace_bytes(1, 64, 8, 900, 800, 512) == 0 and lib.last_error()
    assert L.rz_moe_ffn_workspace_bytes(1, 64, 8, 900, 1024, 500) == 0 and lib.last_error()


# ---------------------------------------------------------------- the reference itself
def test_reference_weights_are_the_oracles(orc):
    rng = np.random.default_rng(5)
    w = rng.integers(0, 256, (3, 2, 144), dtype=np.uint8)
    w[..., 0:2] = rng.uniform(1e-3, 1e-2, (3, 2)).astype(np.float16)[..., None].view(np.uint8)
    w[..., 2:4] = rng.uniform(1e-3, 1e-2, (3, 2)).astype(np.float16)[..., None].view(np.uint8)
    got, size = R.weights(w)
    ref = orc.q4k_dequantize(w.reshape(3, -1)).reshape(3, 512)
    # the oracle's values are f32: two roundings of each part at most
    assert np.all(np.abs(got - ref) <= 3 * 2.0 ** -24 * size)


def test_reference_quantisation_is_the_oracles(orc):
    y = np.random.default_rng(6).normal(0, 3, (5, 96)).astype(np.float32)
    y[1, 32:64] = 0
    assert np.array_equal(R.q8_buffer(*R.q8_quantize(y)), orc.q8_1_quantize(y))


def test_reference_route():
    logits = np.array([[1, 3, 3, -np.inf], [0, -0.0, 5, 5], [-np.inf] * 4, [1, 2, 3, 4]], np.float32)
    e, w, off, rows, places = R.route(logits, 2, True, row_seq=np.array([0, 1, 2, -1]))
    assert e.tolist() == [[1, 2], [2, 3], [-1, -1], [-1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [0.5, 0.5], [0, 0], [0, 0]])
    assert off.tolist() == [0, 0, 1, 3, 4] and rows.tolist() == [0, 1, 2, 3, -1, -1, -1, -1]
    assert places.tolist() == [0, 1, 2, 3, -1, -1, -1, -1]
