"""The paged 4-bit KV cache on the GPU at its edges: values of no size beside small ones, numbers that are none in one
block of a head, scales that underflow, state carried from step to step on the device."""
import numpy as np
import pytest

import paged_reference as R
from gpu_common import check_no_device_error, to_dev
from test_gpu_paged import Setup, device_error, ints, no_error_left, run_plan, rz, want_heads  # noqa: F401

pytestmark = pytest.mark.gpu


def with_cache(s, k=None, v=None):
    """The setup over other keys and values ([slots, K, hd]; the format's own rounding applies to them)."""
    import quantized_q4_q8_gb300 as rz
    with np.errstate(all="ignore"):
        flat, s.kval, s.vval = R.pack(s.kval.astype(np.float64) if k is None else k, s.vval.astype(np.float64) if v is None else v, s.page)
    s.kd, s.vd = (np.abs(x.reshape(-1, s.K, s.hd // 32, 32)).max(-1) / 7 for x in (s.kval, s.vval))
    s.kv = rz.PagedKVQ4(to_dev(flat.reshape(s.kv.pages.shape)), s.page, s.hd)
    return s


# ------------------------------------------------------------------ values of no size
@pytest.mark.parametrize("size", [1e-2, 1e-4, 3e-6])
@pytest.mark.parametrize("hd,H,K,reqs", [
    (128, 32, 8, [(1000, 1000)]),          # whole items within a CTA's share
    (128, 4, 2, [(2900, 300)]),            # items in parts of a tile or two
    (64, 8, 1, [(897, 130), (300, 1)]),
    (64, 14, 2, [(700, 20), (650, 1)]),
])
@pytest.mark.parametrize("zero", ["first", "middle", "last", "all"])
def test_attention_tiles_of_zero_values(rz, size, hd, H, K, reqs, zero):
    """Tokens whose values are all zeros say nothing, so they may not set what the others' weights are measured by.
    (The bound is that of Setup.check: relative to the sums of |d| that the row sees, and 1e-5 of all outputs.)"""
    s = Setup(hd + H, H, K, hd, 64, reqs)
    v = s.vval.astype(np.float64) * size
    for (n, _), slots in zip(reqs, s.slots):
        last = (n - 1) // 128 * 128
        tiles = {"first": [(0, 128)], "middle": [(256, 384), (512, 640)], "last": [(last, n)], "all": [(0, n)]}[zero]
        for a, b in tiles:
            v[slots[a:min(b, n)]] = 0.0
    with_cache(s, v=v)
    out = s.run(rz).cpu().numpy()
    s.check(out)
    assert zero != "all" or not out.any()


@pytest.mark.parametrize("hd,H,K,reqs", [(128, 8, 2, [(1000, 1), (33, 3)]), (64, 14, 2, [(900, 5)]), (128, 8, 2, [(1500, 200)]), (64, 8, 1, [(700, 100)])])
@pytest.mark.parametrize("small", [2.0 ** -9, 2.0 ** -16])
def test_attention_blocks_of_different_sizes(rz, hd, H, K, reqs, small):
    """A head whose last block of values is much smaller than its first, and every fifth token small throughout: on top of
    Setup.check's bound a weight is off by up to 2^-31 of the row's largest p |d| (|d| the largest of 128 tokens here),
    for each token, times codes of up to 8."""
    s = Setup(71 + hd, H, K, hd, 32, reqs)
    v = s.vval.astype(np.float64)
    v[..., -32:] *= small
    v[::5] *= small
    with_cache(s, v=v)
    got, G, sc = s.run(rz).cpu().numpy().astype(np.float64), H // K, hd ** -0.5
    for i, (n, m) in enumerate(reqs):
        slots = s.slots[i]
        for h in range(K):
            q = s.q[s.cu[i]:s.cu[i] + m].reshape(m, H, hd)[:, h * G:(h + 1) * G].astype(np.float64).reshape(m * G, hd)
            k, vv = s.kval[slots, h].astype(np.float64), s.vval[slots, h].astype(np.float64)
            want, p = R.attention(q, k, vv, np.repeat(n - m + np.arange(m) + 1, G), sc)
            out = got[s.cu[i]:s.cu[i] + m].reshape(m, H, hd)[:, h * G:(h + 1) * G].reshape(m * G, hd)
            qb = np.abs(q).reshape(m * G, -1, 32).sum(-1) + 2.0 ** -2 * np.abs(q).max(-1, keepdims=True)
            delta = (sc * 2.0 ** -20 * 23 * (qb @ s.kd[slots, h].T)).max(-1)
            top = np.abs(q @ k.T * sc).max(-1)
            rel = 2 * (delta + 2.0 ** -24 * (top * 1.45 + 40)) + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -23 * (n / 16 + 40)
            tile = np.pad(s.vd[slots, h].max(-1), (0, -n % 128)).reshape(-1, 128).max(-1).repeat(128)[:n]
            floor = n * 8 * 2.0 ** -31 * (p * tile).max(-1, keepdims=True)
            err = np.abs(out - want)
            assert (err <= rel[:, None] * 23 * np.repeat(p @ s.vd[slots, h], 32, axis=-1) + floor).all(), (i, h)
            # the small block by itself: 1e-5 of it, and what the floor of independent roundings comes to
            e, w = err[:, -32:], want[:, -32:]
            assert np.sqrt((e ** 2).mean()) <= 1e-5 * np.sqrt((w ** 2).mean()) + floor.max() / np.sqrt(n)


# ------------------------------------------------------------------ no number in one block
@pytest.mark.parametrize("hd,H,K,reqs", [(128, 4, 2, [(500, 200), (60, 1)]), (64, 4, 2, [(500, 200), (60, 1)]),
                                         (128, 32, 8, [(900, 900)]), (128, 4, 2, [(500, 3), (60, 1)]), (96, 4, 2, [(500, 60)])])
def test_attention_no_number_in_one_block_of_a_value(rz, hd, H, K, reqs):
    """A block of 32 values whose scale is NaN reaches those 32 values of the rows that see it, and no others."""
    import torch
    s = Setup(17 + hd, H, K, hd, 16, reqs)
    good = s.run(rz).clone()
    n, m = reqs[0]
    G, nb = H // K, hd // 32
    seen = torch.zeros_like(good, dtype=torch.bool)
    for token, head, block in ((n - m // 2, 1, nb - 1), (n - 1, 0, 0), (n - m + 1, K - 1, 1)):
        at = R.record_of(16, K, hd, int(s.slots[0][token]), head) + 17 * hd + (token % 16) * 2 * nb + 2 * block
        s.kv.pages.view(-1)[at:at + 2] = torch.tensor([0, 0x7e], dtype=torch.uint8, device="cuda")
        for h in range(head * G, (head + 1) * G):
            seen[token - (n - m):m, h * hd + 32 * block:h * hd + 32 * block + 32] = True
    out = s.run(rz)
    assert torch.equal(out[~seen], good[~seen])
    assert torch.isnan(out[seen]).all()


# ------------------------------------------------------------------ scales that underflow
@pytest.mark.parametrize("hd,H,K", [(64, 4, 2), (128, 4, 1), (96, 4, 2)])
@pytest.mark.parametrize("scale", [1e-44, 1e-38])
def test_attention_scale_of_next_to_nothing(rz, hd, H, K, scale):
    """All tokens that a row sees count alike, those that it does not see for nothing."""
    s = Setup(21, H, K, hd, 16, [(77, 5), (200, 100), (9, 1), (3, 6)])
    s.check(s.run(rz, scale=scale).cpu().numpy(), scale=scale)


@pytest.mark.parametrize("hd,H,K", [(64, 4, 2), (128, 4, 1)])
def test_attention_queries_and_keys_of_next_to_nothing(rz, hd, H, K):
    s = Setup(22, H, K, hd, 16, [(77, 5), (200, 100), (9, 1)], sharp=1e-6)
    s.q = (s.q * np.float32(1e-39)).astype(np.float32)
    s.qd = to_dev(s.q)
    s.check(s.run(rz).cpu().numpy())


# ------------------------------------------------------------------ bad lengths
@pytest.mark.parametrize("m", [1, 3, 60])
@pytest.mark.parametrize("length", [-1, -(2 ** 31)])
def test_attention_negative_length_is_reported(rz, m, length):
    """It counts as empty, as one beyond the table does; the others by the usual bound."""
    import torch
    s = Setup(15, 4, 2, 64, 16, [(50, 1), (80, m), (70, 2)])
    s.lend[1] = length
    out = torch.full((s.T, 256), 2.5, device="cuda")
    s.run(rz, out=out)
    assert device_error(rz) == 0x203
    assert not out[1:1 + m].any()
    s.reqs[1] = (0, m)
    s.check(out.cpu().numpy())


# ------------------------------------------------------------------ launches that overlap
def test_steps_one_after_another_read_what_the_last_wrote(rz):
    """Norm + rotation into the same rows of q, then attention, many times without a wait, a long request among the
    requests (a launch becomes resident while the ones before still run): each step's outputs as with every launch
    waiting for the whole one before."""
    import torch
    H, K, hd, page, steps = 8, 2, 128, 64, 24
    s = Setup(33, H, K, hd, page, [(30000, 1), (70, 2), (900, 60), (10, 1)])
    rng = np.random.default_rng(1)
    x = to_dev(rng.standard_normal((steps, s.T, (H + K) * hd)).astype(np.float32))
    pos = ints(rng.integers(0, 4096, s.T))
    q_out = torch.zeros(s.T, H * hd, device="cuda")

    def run():
        outs = []
        for i in range(steps):
            rz.qk_norm_rope(x[i, :, :H * hd], x[i, :, H * hd:], None, pos, H, K, hd, 1e4, 1, q_out=q_out)
            outs.append(rz.attention_paged_q4(q_out, s.kv, s.td, s.cud, s.lend, H, ws=s.ws))
        return torch.stack(outs)

    got = [run() for _ in range(4)]
    rz.set_pdl(False)
    try:
        want = run()
    finally:
        rz.set_pdl(True)
    for g in got:
        assert torch.equal(g, want)


# ------------------------------------------------------------------ lengths carried on the device
def test_state_carried_on_the_device_over_a_refused_step(rz):
    """One captured graph of plan -> norm, rotation, append -> attention -> next lengths, run until the pool is empty
    and on when there are pages again: the refused request keeps its tokens and goes on where it was."""
    import torch
    rng = np.random.default_rng(3)
    n, H, K, hd, page, max_rows, n_pages = 3, 4, 2, 64, 16, 32, 5
    kv = rz.PagedKVQ4(torch.zeros((n_pages, K, page * hd * 9 // 8), dtype=torch.uint8, device="cuda"), page, hd)
    table = torch.full((n, 4), -1, dtype=torch.int32, device="cuda")
    owned, count = torch.zeros(n, dtype=torch.int32, device="cuda"), ints([n_pages])
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    cached, fresh = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    plan = rz.PagedPlan(n, max_rows)
    qkv = torch.zeros(max_rows, (H + 2 * K) * hd, device="cuda")
    q_out, att = torch.zeros(max_rows, H * hd, device="cuda"), torch.zeros(max_rows, H * hd, device="cuda")
    ws = rz.workspace(rz.attention_paged_q4_workspace_bytes(H, K, hd), "cuda")

    def step():
        rz.paged_plan(cached, fresh, table, owned, free, count, page, plan)
        rz.qk_norm_rope(qkv[:, :H * hd], qkv[:, H * hd:(H + K) * hd], qkv[:, (H + K) * hd:], plan.positions, H, K, hd, 1e4, 1,
                        kv=kv, slots=plan.slots, q_out=q_out)
        rz.attention_paged_q4(q_out, kv, table, plan.cu_rows, plan.kv_len, H, out=att, ws=ws)
        plan.next_cached(cached, fresh, out=cached)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    held, lens = [(np.zeros((0, K, hd)), np.zeros((0, K, hd)))] * n, [0] * n
    # 16 + 16 + 23 tokens take 4 pages; then request 0 takes the last page and 1 is refused, twice; 2 ends; 1 goes on
    for news, refused in (([16, 1, 7], []), ([0, 15, 16], []), ([1, 2, 9], [1]), ([1, 3, 0], [1]), ([1, 0, -1], []), ([1, 2, 5], []), ([2, 1, 1], [])):
        x = rng.standard_normal((max_rows, (H + 2 * K) * hd)).astype(np.float32)
        with torch.cuda.stream(stream):
            fresh.copy_(ints(news))
            qkv.copy_(to_dev(x))
            graph.replay()
        stream.synchronize()
        assert device_error(rz) == (0x204 if refused else 0)
        out, at = att.cpu().numpy().astype(np.float64), 0
        for r, m in enumerate(news):
            if m < 0:
                held[r], lens[r] = (np.zeros((0, K, hd)), np.zeros((0, K, hd))), 0
            if m <= 0:
                continue
            if r in refused:
                assert not out[at:at + m].any() and (plan.positions[at:at + m] == -1).all()
                at += m
                continue
            pos = lens[r] + np.arange(m)
            wq, wk, wv = want_heads(x[at:at + m], H, K, hd, pos, 1e4, 1, None, None)
            held[r] = k, v = tuple(np.concatenate([old, R.quantise(new)[2]]) for old, new in zip(held[r], (wk, wv)))
            for h in range(H):
                want, _ = R.attention(wq[:, h], k[:, h // 2], v[:, h // 2], pos + 1, hd ** -0.5)
                # as in test_step_after_step_matches_dense_attention: 2^-20 of q over scores of up to |q| |k| ... 8
                assert np.abs(out[at:at + m, h * hd:(h + 1) * hd] - want).max() <= 2.0 ** -16 * np.abs(v).max()
            lens[r] += m
            at += m
        assert list(cached.cpu().numpy()) == lens


# ------------------------------------------------------------------ bad pages in a plan
@pytest.mark.parametrize("where", ["table", "pool"])
def test_plan_reports_pages_below_zero(rz, where):
    """The rows on such a page would lose their tokens without a word: a slot below 0 is one that is not written."""
    cached, fresh = np.array([10, 20, 30], np.int32), np.array([1, 3, 5], np.int32)
    table = np.array([[3, -1, -1], [4, 5, -1], [6, 7, -1]], np.int32)
    free = np.array([1, 2, 8, 9, 0, 0, 0, 0, 0, 0], np.int32)
    if where == "table":
        table[1, 1] = -3
    else:
        free[3] = -(2 ** 31)
    args = cached, fresh, np.array([1, 2, 2], np.int32), table, free, 4, 16, 12
    want, got = R.plan(*args), run_plan(rz, *args)
    assert device_error(rz) == 0x206
    want["slots"][want["slots"] < 0] = -1
    for k, v in got.items():
        assert np.array_equal(v, want[k]), k
    lost = [1, 2, 3] if where == "table" else [6, 7, 8]  # request 2's first two new tokens go into the page that it has
    assert (got["slots"][lost] == -1).all() and (got["slots"][:9] >= 0).sum() == 6 and (got["positions"][:9] >= 0).all()


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("hd,H,K,reqs", [
    (128, 8, 8, [(20000, 1)]),             # items in parts of many CTAs
    (64, 4, 2, [(700, 1)] * 200),          # many whole items for a CTA
    (256, 8, 2, [(30000, 5), (900, 1)]),
    (64, 14, 2, [(3000, 5)] * 24),
    (128, 8, 2, [(6000, 700)]),            # the tcgen05 kernel, parts of items
    (64, 32, 8, [(1500, 1500)]),           # its whole items, several for a CTA
    (128, 16, 16, [(5000, 1)] * 8 + [(2000, 300)]),  # both kernels
])
def test_attention_whose_copies_do_not_come_ends_in_an_error(rz, hd, H, K, reqs):
    """CTA 0 (whose share of the work is longer than the start of an item here) waits for tokens that are never copied: the call ends with a timeout's code, and with a workspace of
    zeros the next one is right."""
    import torch
    s = Setup(51, H, K, hd, 64, reqs)
    good = s.run(rz).clone()
    rz.rz_debug_stall_next_paged(1 << 14)
    s.run(rz)
    st, code = rz.check_device_error()  # synchronises: the kernels ended
    assert st == 5 and code == 0x110, (st, hex(code))
    s.ws.zero_()
    for _ in range(2):
        assert torch.equal(s.run(rz), good)
    assert not s.ws[:1024].any()


def test_stall_of_the_paged_attention_is_checked_on_the_host(rz):
    from quantized_q4_q8_gb300 import _lib
    assert _lib.status("rz_debug_stall_next_paged", 10) == 1
    assert _lib.status("rz_debug_stall_next_paged", 1 << 30) == 1


# ------------------------------------------------------------------ capacity for more requests than have rows
@pytest.mark.parametrize("hd,H,K", [(128, 8, 2), (64, 14, 2), (64, 4, 4)])
@pytest.mark.parametrize("spare_rows", [0, 700])
def test_attention_one_prompt_among_idle_requests(rz, hd, H, K, spare_rows):
    """Room for a thousand requests, of which one has a prompt and a few a token: more requests than rows, or spare rows
    for all of them (which kernel works the prompt depends on that, what it gives does not)."""
    import torch
    reqs = [(0, 0)] * 1000
    reqs[3], reqs[500], reqs[777], reqs[999] = (900, 1), (1200, 300), (40, 0), (17, 2)
    s = Setup(61, H, K, hd, 16, reqs, extra_rows=spare_rows)
    s.check(s.run(rz, out=torch.zeros(s.T, H * hd, device="cuda")).cpu().numpy())


# ------------------------------------------------------------------ the layer
def layer_of(rz, sh, tag, bias, fused):
    import torch

    import rz_synth as S
    L = S.layer(sh, tag)
    w = {k: to_dev(v) for k, v in L.w.items()} | {"attn_gamma": to_dev(L.attn_gamma), "ffn_gamma": to_dev(L.ffn_gamma)}
    biases = [to_dev(S.uniform(f"{tag}.b{i}", n, -0.5, 0.5)) if bias else None for i, n in enumerate((sh.q_dim, sh.kv_dim, sh.kv_dim))]
    own = dict(w)
    if fused:
        own["wq"] = torch.cat([own.pop("wq"), own.pop("wk"), own.pop("wv")])
    if bias:
        own |= {"bq": torch.cat(biases)} if fused else dict(zip(("bq", "bk", "bv"), biases))
    layer = rz.DeviceLayer(own, sh.hidden, sh.hidden_pad, sh.n_heads, sh.n_kv_heads, sh.head_dim, sh.inter, sh.eps, sh.rope_theta, sh.rope_mode)
    return layer, w, biases if bias else None


def layer_steps(rz, sh, w, biases, x, kv, table, plan):
    """rz_decode_layer_paged from its public calls, for the rows of x."""
    import torch
    H, K, hd, m = sh.n_heads, sh.n_kv_heads, sh.head_dim, x.shape[0]
    rows = [H * hd, K * hd, K * hd]
    if m <= 3:
        qkv = rz.rmsnorm_q4k_gemv(x, w["attn_gamma"], sh.hidden, sh.eps, [w["wq"], w["wk"], w["wv"]], rows, sh.hidden_pad, biases=biases)
    else:
        x8 = rz.rmsnorm(x, w["attn_gamma"], sh.hidden, sh.hidden_pad, sh.eps, want_y=False)[1]
        qkv = rz.q4k_q8_gemv_multi(x8, [w["wq"], w["wk"], w["wv"]], rows, m, sh.hidden_pad, biases=biases)
    q, _, _ = rz.qk_norm_rope(qkv[:, :H * hd], qkv[:, H * hd:(H + K) * hd], qkv[:, (H + K) * hd:], plan.positions, H, K, hd, sh.rope_theta,
                              sh.rope_mode, eps=sh.eps, kv=kv, slots=plan.slots)
    a8 = torch.zeros(rz.q8_1_size(m, sh.q_pad), dtype=torch.uint8, device="cuda")
    rz.attention_paged_q4(q, kv, table, plan.cu_rows, plan.kv_len, H, att_q8=a8)
    res = torch.zeros(m, sh.hidden_pad, device="cuda")
    rz.q4k_q8_gemv_ex(w["wo"], a8, m, sh.hidden, sh.q_pad, residual=x, out=res, ld=sh.hidden_pad)
    res[:, sh.hidden:] = 0
    return rz.swiglu_ffn(res, w["ffn_gamma"], w["wgate"], w["wup"], w["wdown"], sh.hidden, sh.hidden_pad, sh.inter, sh.eps)


@pytest.mark.parametrize("dims,bias,fused", [
    ((896, 4864, 14, 2, 64, 1e6, 1), True, False), ((896, 4864, 14, 2, 64, 1e6, 1), True, True),
    ((512, 512, 4, 4, 128, 1e4, 0), False, True), ((576, 768, 6, 2, 96, 1e4, 0), True, False), ((512, 512, 2, 1, 256, 1e4, 1), False, False)])
def test_decode_layer_paged_with_spare_rows_and_a_refused_request(rz, dims, bias, fused):
    """The rows of the requests that the plan serves are those of the public calls, bit for bit, whatever stands in the
    rows of a refused request and in those of none."""
    import torch

    import rz_synth as S
    sh = S.LayerShape(*dims)
    layer, w, biases = layer_of(rz, sh, f"edges.{dims}", bias, fused)
    page, n, n_pages = 16, 4, 5
    kvs = [rz.PagedKVQ4(torch.zeros((n_pages, sh.n_kv_heads, page * sh.head_dim * 9 // 8), dtype=torch.uint8, device="cuda"), page, sh.head_dim)
           for _ in range(2)]
    table = torch.full((n, 4), -1, dtype=torch.int32, device="cuda")
    owned, count, free = torch.zeros(n, dtype=torch.int32, device="cuda"), ints([n_pages]), torch.arange(n_pages, dtype=torch.int32, device="cuda")
    cached = torch.zeros(n, dtype=torch.int32, device="cuda")
    for step, (news, m, refused) in enumerate((([9, 3, 1, 0], 16, None), ([1, 14, 0, 1], 16, None), ([7, 2, 1, 2], 14, 0), ([1, 0, 1, 0], 3, None), ([1, 0, 0, 0], 1, None))):
        fresh = ints(news)
        plan = rz.PagedPlan(n, m)
        rz.paged_plan(cached, fresh, table, owned, free, count, page, plan)
        assert device_error(rz) == (0 if refused is None else 0x204)
        rows = sum(news)
        live = [r for r, i in enumerate(np.repeat(np.arange(n), news)) if i != refused]
        x = to_dev(S.hidden_input(f"edges.x{step}", m, sh.hidden, sh.hidden_pad))
        dead = [r for r in range(m) if r not in live]
        x[dead, :sh.hidden] = float("nan")
        out = rz.decode_layer_paged(x, layer, kvs[0], table, plan)
        x[dead, :sh.hidden] = 3.0
        want = layer_steps(rz, sh, w, biases, x, kvs[1], table, plan)
        assert torch.isfinite(want[live]).all() and torch.equal(out[live], want[live]), (step, rows)
        assert torch.equal(kvs[0].pages, kvs[1].pages)
        plan.next_cached(cached, fresh, out=cached)


# ------------------------------------------------------------------ offsets beyond 32 bits
@pytest.mark.parametrize("hd,H,K,reqs", [(128, 16, 8, [(700, 1), (300, 4)]), (64, 16, 16, [(500, 3)]), (128, 16, 8, [(400, 90)])])
def test_pages_beyond_four_gigabytes(rz, hd, H, K, reqs):
    """The same pages, the same rows appended to them and the same attention over them at the end of a cache of some 5 GB."""
    import torch
    s = Setup(81, H, K, hd, 64, reqs)
    small, first = s.kv.pages, 5 * 2 ** 30 // (s.kv.pages[0].numel())
    big = torch.empty((first + small.shape[0], *small.shape[1:]), dtype=torch.uint8, device="cuda")
    big[first:] = small
    far = rz.PagedKVQ4(big, 64, hd)
    T = 9
    slots = ints(s.slots[0][-T:], np.int64)  # new keys and values for tokens that the first request holds
    x = to_dev(np.random.default_rng(2).standard_normal((T, (H + 2 * K) * hd)).astype(np.float32))
    want_q = None
    for kv, off in ((s.kv, 0), (far, first)):
        q, _, _ = rz.qk_norm_rope(x[:, :H * hd], x[:, H * hd:(H + K) * hd], x[:, (H + K) * hd:], ints(np.arange(T)), H, K, hd, 1e4, 1, kv=kv,
                                  slots=slots + off * 64)
        table = torch.where(s.td < small.shape[0], s.td + off, s.td)
        out = rz.attention_paged_q4(s.qd, kv, table, s.cud, s.lend, H, ws=s.ws)
        if want_q is None:
            want_q, want = q, out
    assert torch.equal(q, want_q) and torch.equal(out, want) and torch.equal(big[first:], small)
    # a plan hands such pages out as any others
    n = first + small.shape[0]
    free, plan = torch.arange(n, dtype=torch.int32, device="cuda"), rz.PagedPlan(1, 4)
    rz.paged_plan(ints([0]), ints([3]), ints(np.full((1, 4), -1)), ints([0]), free, ints([n]), 64, plan)
    assert list(plan.slots.cpu().numpy()) == [(n - 1) * 64 + i for i in range(3)] + [-1]
