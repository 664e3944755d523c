"""Host-side checks of the paged 4-bit cache's entry points: every refusal returns its
status and a message before any device work (no GPU here, and no pointer is one)."""
import ctypes as C

import numpy as np
import pytest

import paged_reference as R


@pytest.fixture(scope="module")
def lib():
    from quantized_q4_q8_gb300 import _lib
    from quantized_q4_q8_gb300.build import build
    build()
    _lib.load()
    return _lib


def kv(lib, pages=16, n_pages=4, page=16, heads=2, hd=64):
    return C.byref(lib.KvQ4Struct(pages, n_pages, page, heads, hd))


PLAN = dict(cached=16, fresh=32, n_seqs=2, owned=48, owned_out=48, free_count=64, free_count_out=64, free_pages=80, n_pages=8,
            table=96, ld_table=4, max_blocks=4, page=16, max_rows=8, cu=112, kv_len=128, row_seq=144, positions=160, slots=176,
            stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(cached=None), 1), (dict(fresh=None), 1), (dict(owned_out=None), 1), (dict(slots=None), 1), (dict(kv_len=None), 1),
    (dict(cached=18), 3), (dict(positions=161), 3), (dict(slots=180), 3),
    (dict(n_seqs=0), 2), (dict(n_seqs=1025), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2),
    (dict(max_blocks=0), 2), (dict(ld_table=3), 2), (dict(max_blocks=1 << 27, ld_table=1 << 27), 2),
    (dict(n_pages=0), 2), (dict(n_pages=1 << 31), 2), (dict(max_rows=0), 2), (dict(max_rows=1 << 31), 2),
    (dict(kv_len=16), 1), (dict(kv_len=32), 1),
])
def test_plan_refusals(lib, change, status):
    st = lib.status("rz_paged_plan", *{**PLAN, **change}.values())
    assert st == status and lib.last_error(), (st, lib.last_error())


HEADS = dict(q=16, ld_q=256, k=16, ld_k=128, v=16, ld_v=128, qg=None, kg=None, eps=1e-6, pos=16, slots=16, kv=True, n=3, H=4, K=2,
             hd=64, theta=1e4, mode=0, qo=16, ld_qo=256, ko=None, vo=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(pos=None), 1), (dict(qo=None), 1), (dict(v=None), 1), (dict(slots=None), 1),
    (dict(kv=None), 1), (dict(kv=None, ko=16, vo=16), 1),
    (dict(q=18), 3), (dict(qg=17), 3), (dict(slots=12), 3), (dict(n=0), 1), (dict(n=1 << 31), 1),
    (dict(hd=48), 2), (dict(hd=0), 2), (dict(hd=288), 2), (dict(H=0), 2), (dict(K=0), 2), (dict(K=3), 2), (dict(hd=32), 2),
    (dict(mode=2), 1), (dict(theta=0.0), 1), (dict(theta=float("nan")), 1), (dict(theta=float("inf")), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(ld_q=255), 2), (dict(ld_k=127), 2), (dict(ld_v=127), 2), (dict(ld_qo=255), 2),
    (dict(kv=dict(pages=None)), 1), (dict(kv=dict(pages=8)), 3), (dict(kv=dict(page=20)), 2), (dict(kv=dict(n_pages=0)), 2),
    (dict(kv=dict(n_pages=1 << 31)), 2), (dict(kv=dict(heads=0)), 2), (dict(kv=dict(heads=1025)), 2),
])
def test_heads_refusals(lib, change, status):
    a = {**HEADS, **change}
    a["kv"] = kv(lib, **(a["kv"] if isinstance(a["kv"], dict) else {})) if a["kv"] else None
    st = lib.status("rz_qk_norm_rope", *a.values())
    assert st == status and lib.last_error(), (st, lib.last_error())


ATT = dict(q=16, ld_q=256, n=5, kv=True, table=16, ld_table=4, max_blocks=4, cu=16, kv_len=16, n_seqs=2, H=4, scale=0.0, att=16, q8=None,
           ws=16, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(kv_len=None), 1), (dict(att=None), 1), (dict(kv=None), 1),
    (dict(kv=dict(hd=40)), 2), (dict(ld_table=3), 2), (dict(max_blocks=0), 2), (dict(n_seqs=0), 2), (dict(n_seqs=1025), 2),
    (dict(H=0), 2), (dict(H=3), 2), (dict(n=0), 1), (dict(n=1 << 31), 2), (dict(n=1 << 30), 2), (dict(ld_q=252), 2), (dict(ld_q=258), 2),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q=20), 3), (dict(att=24), 3), (dict(q8=8), 3), (dict(table=17), 3), (dict(cu=18), 3), (dict(ws=None), 1), (dict(ws=8), 3),
])
def test_attention_refusals(lib, change, status):
    a = {**ATT, **change}
    a["kv"] = kv(lib, **(a["kv"] if isinstance(a["kv"], dict) else {})) if a["kv"] else None
    st = lib.status("rz_attention_paged_q4", *a.values())
    assert st == status and lib.last_error(), (st, lib.last_error())


WEIGHTS = dict(wq=16, wk=32, wv=48, wo=64, wgate=80, wup=96, wdown=112, attn_gamma=128, ffn_gamma=144, hidden=256, hidden_pad=256,
               n_heads=4, n_kv_heads=2, head_dim=64, inter=512, eps=1e-6, rope_theta=1e4, rope_mode=0, bq=None, bk=None, bv=None)
LAYER = dict(input=16, w=True, qg=None, kg=None, kv=True, positions=16, slots=16, table=16, ld_table=4, max_blocks=4, cu=16, kv_len=16,
             n_seqs=2, m=5, output=32, ws=16, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(input=None), 1), (dict(output=None), 1), (dict(positions=None), 1), (dict(slots=None), 1), (dict(table=None), 1),
    (dict(cu=None), 1), (dict(kv_len=None), 1), (dict(w=None), 1), (dict(kv=None), 1),
    (dict(input=20), 3), (dict(output=24), 3), (dict(qg=17), 3), (dict(kg=18), 3), (dict(slots=12), 3), (dict(table=17), 3), (dict(cu=18), 3),
    (dict(kv_len=19), 3), (dict(positions=21), 3),
    (dict(n_seqs=0), 2), (dict(n_seqs=1025), 2), (dict(ld_table=3), 2), (dict(max_blocks=0), 2), (dict(m=0), 2), (dict(m=17), 2),
    (dict(kv=dict(hd=40)), 2), (dict(kv=dict(hd=32)), 2), (dict(kv=dict(heads=1)), 2), (dict(kv=dict(page=20)), 2), (dict(kv=dict(pages=8)), 3),
    (dict(w=dict(wo=None)), 1), (dict(w=dict(wk=None)), 1), (dict(w=dict(wq=24)), 3), (dict(w=dict(n_kv_heads=3)), 2),
])
def test_layer_refusals(lib, change, status):
    a = {**LAYER, **change}
    a["kv"] = kv(lib, **(a["kv"] if isinstance(a["kv"], dict) else {})) if a["kv"] else None
    a["w"] = C.byref(lib.LayerWeightsStruct(**{**WEIGHTS, **(a["w"] if isinstance(a["w"], dict) else {})})) if a["w"] else None
    st = lib.status("rz_decode_layer_paged", *a.values())
    assert st == status and lib.last_error(), (st, lib.last_error())


def test_sizes(lib):
    L = lib.load()
    assert L.rz_kv_q4_page_bytes(16, 1, 128) == 16 * 128 * 9 // 8
    assert L.rz_kv_q4_page_bytes(64, 8, 96) == 8 * 4 * 18 * 96
    for bad in ((15, 1, 128), (16, 0, 128), (16, 1, 100), (16, 1, 0)):
        assert L.rz_kv_q4_page_bytes(*bad) == 0 and lib.last_error()
    assert L.rz_attention_paged_q4_workspace_bytes(4, 3, 64) == 0
    assert L.rz_attention_paged_q4_workspace_bytes(4, 2, 60) == 0


@pytest.fixture
def binding(monkeypatch):
    torch = pytest.importorskip("torch")
    import quantized_q4_q8_gb300 as rz
    from quantized_q4_q8_gb300.build import build
    build()
    if not torch.cuda.is_available():
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return rz


def test_binding_checks_tensors(binding):
    import torch
    rz = binding
    t = torch.zeros(2, 4, 8, dtype=torch.uint8)
    with pytest.raises(TypeError, match="CUDA tensor"):
        rz.PagedKVQ4(t, 16, 64)
    with pytest.raises(ValueError, match="page_size"):
        rz.kv_q4_page_bytes(17, 2, 64)
    with pytest.raises(TypeError, match="block_table"):
        i = torch.zeros(2, dtype=torch.int32)
        rz.paged_plan(i, i, i.view(1, 2), i, i, i[:1], 16, rz.PagedPlan(1, 4, "cpu"))
    with pytest.raises(TypeError, match="q must"):
        rz.qk_norm_rope(torch.zeros(1, 64), torch.zeros(1, 64), None, torch.zeros(1, dtype=torch.int32), 1, 1, 64, 1e4, 0)


# ------------------------------------------------------------------ the reference itself
@pytest.mark.parametrize("nb", range(1, 9))
def test_every_byte_of_a_record_has_one_place(nb):
    k = {R.k_place(nb, t, b, i) for t in range(16) for b in range(nb) for i in range(16)}
    v = {R.v_place(nb, t, b, i) for t in range(16) for b in range(nb) for i in range(16)}
    hd = 32 * nb
    assert k == set(range(8 * hd)) and v == set(range(9 * hd, 17 * hd))


def test_pack_and_store_agree():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 64, 3, 96))
    flat, kv_, vv = R.pack(k, v, 32)
    one = np.zeros_like(flat)
    for s in range(64):
        for h in range(3):
            R.store(one, 32, 3, 96, s, h, R.quantise(k[s, h])[:2], R.quantise(v[s, h])[:2])
    assert np.array_equal(flat, one)
    # a Q4_0 block is off by at most half a step, but for the end that has no code 16
    d = np.abs(k).reshape(64, 3, 3, 32).max(-1).repeat(32, -1).reshape(k.shape) / 8
    assert (np.abs(kv_ - k) <= d * 1.01).all() and (np.abs(kv_ - k) <= d * 0.51).mean() > 0.95


def test_quantise_edges():
    x = np.zeros(32)
    d, c, v = R.quantise(x)
    assert d[0] == 0 and not np.signbit(d[0]) and (c == 8).all() and not v.any()
    x[3], x[7] = 4.0, -4.0            # two peaks of one size: the positive one
    d, c, v = R.quantise(x)
    assert d[0] == -0.5 and c[0, 3] == 0 and c[0, 7] == 15 and v[3] == 4.0 and v[7] == -3.5
    x[0] = np.inf
    d, c, v = R.quantise(x)
    assert np.isnan(d[0]) and (c == 8).all() and np.isnan(v).all()
    x = np.full(32, 1e9)
    d, c, v = R.quantise(x)
    assert d[0] == -65504 and (c == 0).all()
