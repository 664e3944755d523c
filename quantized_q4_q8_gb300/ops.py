"""torch-facing helpers over the librz C ABI (marshalling and output allocation only)."""
from __future__ import annotations

import ctypes as C

from ._lib import call, load, status

__all__ = [
    "q8_1_size", "q4k_bytes", "q4_0_bytes",
    "rz_q8_1_quantize", "rz_q4k_q8_gemv", "rz_q4k_q8_subblock_dots", "rz_q4_0_gemv",
    "rz_q4k_q8_gemv_ex", "rz_rmsnorm_q4k_gemv", "q4k_q8_gemv_ex", "rmsnorm_q4k_gemv",
    "rz_q4k_q8_gemv_multi", "q4k_q8_gemv_multi",
    "rz_q4k_f32_gemv", "q4k_f32_gemv",
    "rz_q4k_q8_gemm", "q4k_q8_gemm_workspace_bytes", "q4k_q8_gemm",
    "rz_rmsnorm", "rz_residual_add", "rz_check_device_error", "rz_set_pdl", "rz_debug_stall_next_gemv", "rz_debug_stall_next_paged",
    "rz_debug_stall_next_moe",
    "q8_1_quantize", "q4k_q8_gemv", "q4k_q8_subblock_dots", "q4_0_gemv",
    "rmsnorm", "residual_add", "check_device_error", "set_pdl", "version",
    "DeviceLayer", "DeviceKV", "DeviceStack", "workspace", "swiglu_ffn_workspace_bytes",
    "swiglu_ffn", "rz_swiglu_ffn_static", "attention_workspace_bytes", "attention_decode",
    "decode_layer_workspace_bytes", "decode_layer", "rz_decode_stack", "decode_stack",
    "rz_decode_layers", "decode_layers", "DeviceLayerQ40", "decode_layer_q4_0",
    "kv_q4_page_bytes", "PagedKVQ4", "PagedPlan", "rz_paged_plan", "paged_plan", "rz_qk_norm_rope", "qk_norm_rope",
    "rz_attention_paged_q4", "attention_paged_q4_workspace_bytes", "attention_paged_q4",
    "decode_layer_paged_workspace_bytes", "decode_layer_paged",
    "rz_residual_rmsnorm", "residual_rmsnorm", "MoePlan", "moe_route_workspace_bytes", "rz_moe_route", "moe_route",
    "moe_swiglu_workspace_bytes", "rz_moe_swiglu", "moe_swiglu", "moe_down_workspace_bytes", "rz_moe_down", "moe_down",
    "moe_ffn_workspace_bytes", "rz_moe_ffn", "moe_ffn",
]


def q8_1_size(m: int, n: int) -> int:
    """Bytes of a Q8_1 buffer of m rows of n values (int8 q | f32 d | f32 s)."""
    return m * n + 8 * m * (n // 32)


def q4k_bytes(out_dim: int, in_dim: int) -> int:
    return out_dim * (in_dim // 256) * 144


def q4_0_bytes(out_dim: int, in_dim: int) -> int:
    return out_dim * (in_dim // 32) * 18


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# ------------------------------------------------------------------ raw entry points
def rz_q8_1_quantize(x, q8, m, n, stream=None):
    return call("rz_q8_1_quantize", _ptr(x), _ptr(q8), m, n, _stream(stream))


def rz_q4k_q8_gemv(w, q8, y, m, out_dim, in_dim, stream=None):
    return call("rz_q4k_q8_gemv", _ptr(w), _ptr(q8), _ptr(y), m, out_dim, in_dim, _stream(stream))


def rz_q4k_q8_subblock_dots(w, q8, I, out_dim, in_dim, stream=None):
    return call("rz_q4k_q8_subblock_dots", _ptr(w), _ptr(q8), _ptr(I), out_dim, in_dim,
                _stream(stream))


def rz_q4k_q8_gemv_ex(w, q8, bias, residual, y, ld, m, out_dim, in_dim, stream=None):
    return call("rz_q4k_q8_gemv_ex", _ptr(w), _ptr(q8), _ptr(bias), _ptr(residual), _ptr(y), ld, m,
                out_dim, in_dim, _stream(stream))


def rz_rmsnorm_q4k_gemv(x, ldx, gamma, n, eps, ws, rows, biases, y, ldy, m, in_dim, stream=None):
    """ws, rows, biases: sequences of equal length (1..3); biases may be None."""
    k = len(ws)
    wp = (C.c_void_p * k)(*[_ptr(t) for t in ws])
    rp = (C.c_int64 * k)(*rows)
    bp = None if biases is None else (C.c_void_p * k)(*[_ptr(b) for b in biases])
    return call("rz_rmsnorm_q4k_gemv", _ptr(x), ldx, _ptr(gamma), n, eps, k, wp, rp, bp, _ptr(y), ldy,
                m, in_dim, _stream(stream))


def rz_q4k_q8_gemv_multi(q8, ws, rows, biases, y, ldy, m, in_dim, stream=None):
    """ws, rows, biases: sequences of equal length (1..3); biases may be None."""
    k = len(ws)
    wp = (C.c_void_p * k)(*[_ptr(t) for t in ws])
    rp = (C.c_int64 * k)(*rows)
    bp = None if biases is None else (C.c_void_p * k)(*[_ptr(b) for b in biases])
    return call("rz_q4k_q8_gemv_multi", _ptr(q8), k, wp, rp, bp, _ptr(y), ldy, m, in_dim, _stream(stream))


def q4k_q8_gemv_multi(q8, ws, rows, m, in_dim, biases=None, out=None, stream=None):
    """GEMVs of 1..3 matrices against one Q8_1 activation; returns f32 [m, sum(rows)]."""
    import torch
    if out is None:
        out = torch.empty((m, sum(rows)), dtype=torch.float32, device=q8.device)
    rz_q4k_q8_gemv_multi(q8, ws, rows, biases, out, out.shape[-1], m, in_dim, stream)
    return out


def rz_q4k_f32_gemv(w, x, bias, y, m, out_dim, in_dim, stream=None):
    return call("rz_q4k_f32_gemv", _ptr(w), _ptr(x), _ptr(bias), _ptr(y), m, out_dim, in_dim, _stream(stream))


def q4k_f32_gemv(w, x, out_dim, in_dim, bias=None, out=None, stream=None):
    """Q4_K weights times f32 activations x [m, in_dim] (no Q8_1) -> f32 [m, out_dim]."""
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    if out is None:
        out = torch.empty((m, out_dim), dtype=torch.float32, device=w.device)
    rz_q4k_f32_gemv(w, x, bias, out, m, out_dim, in_dim, stream)
    return out


def rz_q4_0_gemv(w, x, y, m, out_dim, in_dim, stream=None):
    return call("rz_q4_0_gemv", _ptr(w), _ptr(x), _ptr(y), m, out_dim, in_dim, _stream(stream))


def rz_rmsnorm(x, gamma, y, q8, m, n, n_pad, eps, stream=None):
    return call("rz_rmsnorm", _ptr(x), _ptr(gamma), _ptr(y), _ptr(q8), m, n, n_pad, eps,
                _stream(stream))


def rz_residual_add(a, b, out, n, stream=None):
    return call("rz_residual_add", _ptr(a), _ptr(b), _ptr(out), n, _stream(stream))


def rz_check_device_error(stream=None):
    """Returns (status, code); status 0 when the device error word was clear."""
    code = C.c_uint32(0)
    st = status("rz_check_device_error", _stream(stream), C.byref(code))
    return st, code.value


def rz_set_pdl(enable: bool):
    return call("rz_set_pdl", 1 if enable else 0)


def rz_debug_stall_next_gemv(wait_limit: int):
    """Test aid: the next Q4_K GEMV launch runs out of a bounded wait (see rz.h)."""
    return call("rz_debug_stall_next_gemv", int(wait_limit))


def rz_debug_stall_next_paged(wait_limit: int):
    """Test aid: the next paged attention runs out of a bounded wait (see rz.h)."""
    return call("rz_debug_stall_next_paged", int(wait_limit))


def rz_debug_stall_next_moe(wait_limit: int):
    """Test aid: the next grouped product on the tensor cores runs out of a bounded wait (see rz.h)."""
    return call("rz_debug_stall_next_moe", int(wait_limit))


# ------------------------------------------------------------------ tensor helpers
def _cuda_contig(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def q8_1_quantize(x, out=None, stream=None):
    """x: f32 CUDA [m, n] -> uint8 CUDA [q8_1_size(m, n)]."""
    import torch
    _cuda_contig(x, torch.float32, "x")
    m, n = (1, x.shape[0]) if x.dim() == 1 else x.shape
    if out is None:
        out = torch.empty(q8_1_size(m, n), dtype=torch.uint8, device=x.device)
    rz_q8_1_quantize(x, out, m, n, stream)
    return out


def q4k_q8_gemv(w, q8, m, out_dim, in_dim, out=None, stream=None):
    import torch
    _cuda_contig(w, torch.uint8, "w")
    _cuda_contig(q8, torch.uint8, "q8")
    if out is None:
        out = torch.empty((m, out_dim), dtype=torch.float32, device=w.device)
    rz_q4k_q8_gemv(w, q8, out, m, out_dim, in_dim, stream)
    return out


def rz_q4k_q8_gemm(w, q8, y, ldy, m, out_dim, in_dim, ws, ws_bytes, stream=None):
    return call("rz_q4k_q8_gemm", _ptr(w), _ptr(q8), _ptr(y), ldy, m, out_dim, in_dim, _ptr(ws), ws_bytes,
                _stream(stream))


def q4k_q8_gemm_workspace_bytes(m: int, in_dim: int) -> int:
    return int(load().rz_q4k_q8_gemm_workspace_bytes(m, in_dim))


def q4k_q8_gemm(w, q8, m, out_dim, in_dim, out=None, ws=None, stream=None):
    """y = W x_t for m tokens on the tensor cores (any m >= 1); y f32 [m, out_dim]."""
    import torch
    _cuda_contig(w, torch.uint8, "w")
    _cuda_contig(q8, torch.uint8, "q8")
    if out is None:
        out = torch.empty((m, out_dim), dtype=torch.float32, device=w.device)
    need = q4k_q8_gemm_workspace_bytes(m, in_dim)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=w.device)
    rz_q4k_q8_gemm(w, q8, out, out.shape[-1], m, out_dim, in_dim, ws, ws.numel(), stream)
    return out


def q4k_q8_gemv_ex(w, q8, m, out_dim, in_dim, bias=None, residual=None, out=None, ld=0,
                   stream=None):
    """y = W x (+ bias | + residual); y f32 [m, ld or out_dim]."""
    import torch
    if out is None:
        out = torch.empty((m, ld or out_dim), dtype=torch.float32, device=w.device)
    rz_q4k_q8_gemv_ex(w, q8, bias, residual, out, ld, m, out_dim, in_dim, stream)
    return out


def rmsnorm_q4k_gemv(x, gamma, n, eps, ws, rows, in_dim, biases=None, out=None, stream=None):
    """RMSNorm -> Q8_1 -> GEMVs of 1..3 matrices; returns f32 [m, sum(rows)]."""
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    ldx = x.shape[-1]
    if out is None:
        out = torch.empty((m, sum(rows)), dtype=torch.float32, device=x.device)
    rz_rmsnorm_q4k_gemv(x, ldx, gamma, n, eps, ws, rows, biases, out, out.shape[-1], m, in_dim, stream)
    return out


def q4k_q8_subblock_dots(w, q8, out_dim, in_dim, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((out_dim, in_dim // 32), dtype=torch.int32, device=w.device)
    rz_q4k_q8_subblock_dots(w, q8, out, out_dim, in_dim, stream)
    return out


def q4_0_gemv(w, x, out_dim, in_dim, out=None, bias=None, stream=None):
    import torch
    _cuda_contig(w, torch.uint8, "w")
    _cuda_contig(x, torch.float32, "x")
    m = 1 if x.dim() == 1 else x.shape[0]
    if out is None:
        out = torch.empty((m, out_dim), dtype=torch.float32, device=w.device)
    if bias is None:
        rz_q4_0_gemv(w, x, out, m, out_dim, in_dim, stream)
    else:
        call("rz_q4_0_gemv_bias", _ptr(w), _ptr(x), _ptr(bias), _ptr(out), m, out_dim, in_dim, _stream(stream))
    return out


def rmsnorm(x, gamma, n, n_pad, eps, want_y=True, want_q8=True, stream=None):
    """x: f32 [m, n_pad] -> (y f32 [m, n_pad] or None, q8 uint8 or None)."""
    import torch
    _cuda_contig(x, torch.float32, "x")
    m = 1 if x.dim() == 1 else x.shape[0]
    y = torch.empty((m, n_pad), dtype=torch.float32, device=x.device) if want_y else None
    q8 = torch.empty(q8_1_size(m, n_pad), dtype=torch.uint8, device=x.device) if want_q8 else None
    rz_rmsnorm(x, gamma, y, q8, m, n, n_pad, eps, stream)
    return y, q8


def residual_add(a, b, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty_like(a)
    rz_residual_add(a, b, out, a.numel(), stream)
    return out


def check_device_error(stream=None):
    return rz_check_device_error(stream)


def set_pdl(enable: bool):
    rz_set_pdl(enable)


def version() -> str:
    return load().rz_version().decode()


# ------------------------------------------------------------------ layer-level helpers
class DeviceLayer:
    """One Q4_K decode layer resident on the GPU (torch tensors) and its C descriptor.

    weights: dict with uint8 CUDA tensors wq, wk, wv, wo, wgate, wup, wdown and f32
    CUDA tensors attn_gamma, ffn_gamma; optional f32 CUDA tensors bq, bk, bv (QKV
    bias).  The fused Q|K|V layout leaves wk and wv out (or None) and holds the one
    [q_dim + 2 kv_dim][hidden_pad] matrix in wq.  Shapes follow include/rz.h."""

    def __init__(self, weights: dict, hidden: int, hidden_pad: int, n_heads: int,
                 n_kv_heads: int, head_dim: int, inter: int, eps: float, rope_theta: float,
                 rope_mode: int):
        from ._lib import LayerWeightsStruct
        self.t = weights
        self.hidden, self.hidden_pad, self.n_heads = hidden, hidden_pad, n_heads
        self.n_kv_heads, self.head_dim, self.inter = n_kv_heads, head_dim, inter
        self.eps, self.rope_theta, self.rope_mode = eps, rope_theta, rope_mode

        def p(k):
            t = weights.get(k)
            return None if t is None else t.data_ptr()

        self.struct = LayerWeightsStruct(
            *[p(k) for k in ("wq", "wk", "wv", "wo", "wgate", "wup", "wdown", "attn_gamma", "ffn_gamma")],
            hidden, hidden_pad, n_heads, n_kv_heads, head_dim, inter, eps, rope_theta, rope_mode,
            p("bq"), p("bk"), p("bv"))

    @property
    def kv_dim(self):
        return self.n_kv_heads * self.head_dim


class DeviceKV:
    """f32 K and V caches [m][max_seq][kv_dim] of one layer and their C descriptor."""

    def __init__(self, k, v):
        from ._lib import KvCacheStruct
        import torch
        assert k.dtype == torch.float32 and k.is_cuda and k.is_contiguous() and k.dim() == 3
        self.k, self.v = k, v
        m, max_seq, kv_dim = k.shape
        self.max_seq = max_seq
        self.struct = KvCacheStruct(k.data_ptr(), v.data_ptr(), max_seq * kv_dim, max_seq)


def workspace(nbytes: int, device):
    """Zero-filled device workspace (the attention counters start at zero)."""
    import torch
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def swiglu_ffn_workspace_bytes(m, hidden_pad, inter):
    return load().rz_swiglu_ffn_workspace_bytes(m, hidden_pad, inter)


def swiglu_ffn(x, gamma, w_gate, w_up, w_down, hidden, hidden_pad, inter, eps, out=None,
               ws=None, stream=None):
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    if out is None:
        out = torch.empty((m, hidden_pad), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(swiglu_ffn_workspace_bytes(m, hidden_pad, inter), x.device)
    call("rz_swiglu_ffn", _ptr(x), _ptr(gamma), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(out),
         m, hidden, hidden_pad, inter, eps, _ptr(ws), ws.numel(), _stream(stream))
    return out


def rz_swiglu_ffn_static(x, gamma, w_gate, w_up, w_down, out, m, hidden, hidden_pad, inter, eps,
                         stream=None):
    """The SwiGLU FFN with the library's static scratch (no workspace argument)."""
    return call("rz_swiglu_ffn_static", _ptr(x), _ptr(gamma), _ptr(w_gate), _ptr(w_up),
                _ptr(w_down), _ptr(out), m, hidden, hidden_pad, inter, eps, _stream(stream))


def attention_workspace_bytes(m, n_heads, n_kv_heads, head_dim, max_seq):
    return load().rz_attention_workspace_bytes(m, n_heads, n_kv_heads, head_dim, max_seq)


def attention_decode(q, k, v, ld_qkv, kv: "DeviceKV", n_heads, n_kv_heads, head_dim,
                     rope_theta, rope_mode, position=0, positions=None, want_att=True,
                     want_q8=True, ws=None, stream=None):
    import ctypes as C
    import torch
    m = kv.k.shape[0]
    q_dim = n_heads * head_dim
    q_pad = (q_dim + 255) // 256 * 256
    att = torch.empty((m, q_dim), dtype=torch.float32, device=q.device) if want_att else None
    a8 = torch.empty(q8_1_size(m, q_pad), dtype=torch.uint8, device=q.device) if want_q8 else None
    if ws is None:
        ws = workspace(attention_workspace_bytes(m, n_heads, n_kv_heads, head_dim, kv.max_seq),
                       q.device)
    call("rz_attention_decode", _ptr(q), _ptr(k), _ptr(v), ld_qkv, C.byref(kv.struct),
         _ptr(positions), position, m, n_heads, n_kv_heads, head_dim, rope_theta, rope_mode,
         _ptr(att), _ptr(a8), _ptr(ws), ws.numel(), _stream(stream))
    return att, a8


def decode_layer_workspace_bytes(layer: "DeviceLayer", m, max_seq):
    import ctypes as C
    return load().rz_decode_layer_workspace_bytes(C.byref(layer.struct), m, max_seq)


def decode_layer(x, layer: "DeviceLayer", kv: "DeviceKV", position=0, positions=None, out=None,
                 ws=None, stream=None):
    import ctypes as C
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    if out is None:
        out = torch.empty((m, layer.hidden_pad), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(decode_layer_workspace_bytes(layer, m, kv.max_seq), x.device)
    call("rz_decode_layer", _ptr(x), C.byref(layer.struct), C.byref(kv.struct), _ptr(positions),
         position, m, _ptr(out), _ptr(ws), ws.numel(), _stream(stream))
    return out


class DeviceStack:
    """Layers + per-layer KV caches + output norm + Q4_0 LM head, with the host
    descriptor arrays the C ABI takes."""

    def __init__(self, layers, kvs, out_gamma, lm_head, vocab, lm_bias=None):
        from ._lib import KvCacheStruct, LayerWeightsStruct
        self.layers, self.kvs = layers, kvs
        self.out_gamma, self.lm_head, self.vocab, self.lm_bias = out_gamma, lm_head, vocab, lm_bias
        n = len(layers)
        self.lw = (LayerWeightsStruct * n)(*[l.struct for l in layers])
        self.kv = (KvCacheStruct * n)(*[k.struct for k in kvs])

    def workspace_bytes(self, m):
        return load().rz_decode_stack_workspace_bytes(self.lw, len(self.layers), m,
                                                      self.kvs[0].max_seq)

    def launches(self, m, with_head=True):
        """librz kernels one rz_decode_stack (or rz_decode_layers) call launches."""
        return load().rz_decode_stack_launches(self.lw, len(self.layers), m, self.kvs[0].max_seq,
                                               1 if with_head else 0, self.vocab)


def rz_decode_stack(x, stack: "DeviceStack", positions, position, m, hidden_out, logits, ws,
                    stream=None):
    return call("rz_decode_stack", _ptr(x), stack.lw, stack.kv, len(stack.layers),
                _ptr(positions), position, m, _ptr(stack.out_gamma), _ptr(stack.lm_head),
                _ptr(stack.lm_bias), stack.vocab, _ptr(hidden_out), _ptr(logits), _ptr(ws), ws.numel(),
                _stream(stream))


def rz_decode_layers(x, stack: "DeviceStack", positions, position, m, out, ws, stream=None):
    return call("rz_decode_layers", _ptr(x), stack.lw, stack.kv, len(stack.layers), _ptr(positions),
                position, m, _ptr(out), _ptr(ws), ws.numel(), _stream(stream))


def decode_layers(x, stack: "DeviceStack", position=0, positions=None, ws=None, stream=None):
    """The stack's layers without the output norm and LM head; returns the hidden state."""
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    out = torch.empty((m, stack.layers[0].hidden_pad), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(stack.workspace_bytes(m), x.device)
    rz_decode_layers(x, stack, positions, position, m, out, ws, stream)
    return out


def decode_stack(x, stack: "DeviceStack", position=0, positions=None, ws=None, stream=None,
                 want_hidden=True):
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    hp = stack.layers[0].hidden_pad
    hid = torch.empty((m, hp), dtype=torch.float32, device=x.device) if want_hidden else None
    logits = torch.empty((m, stack.vocab), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(stack.workspace_bytes(m), x.device)
    rz_decode_stack(x, stack, positions, position, m, hid, logits, ws, stream)
    return hid, logits


# ------------------------------------------------------------------ Q4_0 whole-model layer
class DeviceLayerQ40:
    """One Q4_0 layer on the GPU: uint8 CUDA tensors wqkv, wo, wup, wdown (and wgate
    for SwiGLU, absent for the GELU FFN), f32 attn_gamma, ffn_gamma."""

    def __init__(self, weights: dict, hidden: int, n_heads: int, n_kv_heads: int, head_dim: int, inter: int,
                 eps: float, rope_theta: float, rope_mode: int):
        from ._lib import LayerWeightsQ40Struct
        self.t = weights
        self.hidden, self.n_heads, self.n_kv_heads, self.head_dim, self.inter = hidden, n_heads, n_kv_heads, head_dim, inter

        def p(k):
            t = weights.get(k)
            return None if t is None else t.data_ptr()

        self.struct = LayerWeightsQ40Struct(
            *[p(k) for k in ("wqkv", "wo", "wgate", "wup", "wdown", "attn_gamma", "ffn_gamma")],
            hidden, n_heads, n_kv_heads, head_dim, inter, eps, rope_theta, rope_mode)


def decode_layer_q4_0(x, layer: DeviceLayerQ40, kv: "DeviceKV", position=0, positions=None, out=None, ws=None,
                      stream=None):
    import ctypes as C
    import torch
    m = 1 if x.dim() == 1 else x.shape[0]
    if out is None:
        out = torch.empty((m, layer.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(load().rz_decode_layer_q4_0_workspace_bytes(C.byref(layer.struct), m, kv.max_seq), x.device)
    call("rz_decode_layer_q4_0", _ptr(x), C.byref(layer.struct), C.byref(kv.struct), _ptr(positions), position, m,
         _ptr(out), _ptr(ws), ws.numel(), _stream(stream))
    return out


# ------------------------------------------------------------------ paged 4-bit KV cache
def kv_q4_page_bytes(page_size: int, n_kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the 4-bit cache."""
    n = int(load().rz_kv_q4_page_bytes(page_size, n_kv_heads, head_dim))
    if n == 0:
        raise ValueError(load().rz_last_error().decode())
    return n


def _on_device(t, dtype, dim, dev, name):
    """A CUDA tensor of device `dev`, of this type and number of dimensions."""
    at = t.get_device() if hasattr(t, "get_device") else -1
    if at < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if at != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimension{'s' if dim > 1 else ''}, got {t.dim()}")
    return t


def _vector(t, dtype, n, dev, name, more=False):
    """The address of n contiguous values (or, with more, at least n)."""
    _on_device(t, dtype, 1, dev, name)
    have = t.shape[0]
    if (have < n if more else have != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values")
    return t.data_ptr()


def _row_ld(t, cols, name):
    """Row stride of a 2-D tensor of `cols` contiguous columns."""
    if t.shape[1] != cols or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must have {cols} contiguous columns")
    return max(t.stride(0), cols) if t.shape[0] == 1 else t.stride(0)


def _new(shape, dtype, dev, stream):
    """An output allocated for the stream that the call runs on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _stream_on(stream, dev):
    """The raw stream of a call on device `dev` (its current one unless given)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


class PagedKVQ4:
    """The 4-bit K and V cache of one layer: a uint8 CUDA tensor of pages
    [n_pages, n_kv_heads, page_size * head_dim * 9 / 8] and its C descriptor."""

    def __init__(self, pages, page_size: int, head_dim: int):
        import torch
        from ._lib import KvQ4Struct
        _on_device(pages, torch.uint8, 3, torch.cuda.current_device(), "pages")
        n_pages, n_kv_heads, size = pages.shape
        if not pages.is_contiguous() or n_pages < 1 or size * n_kv_heads != kv_q4_page_bytes(page_size, n_kv_heads, head_dim):
            raise ValueError("pages must be contiguous [n_pages, n_kv_heads, page_size * head_dim * 9 / 8]")
        self.pages, self.page_size, self.n_kv_heads, self.head_dim = pages, page_size, n_kv_heads, head_dim
        self.dev = pages.get_device()
        self.struct = KvQ4Struct(pages.data_ptr(), n_pages, page_size, n_kv_heads, head_dim)
        self.ref = C.byref(self.struct)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda"):
        import torch
        size = kv_q4_page_bytes(page_size, n_kv_heads, head_dim) // n_kv_heads
        return cls(torch.empty((n_pages, n_kv_heads, size), dtype=torch.uint8, device=device), page_size, head_dim)


class PagedPlan:
    """The outputs of paged_plan for n_seqs requests and up to max_rows new tokens: cu_rows,
    kv_len, row_seq, positions (int32) and slots (int64), kept from step to step."""

    def __init__(self, n_seqs: int, max_rows: int, device="cuda"):
        import torch
        self.n_seqs, self.max_rows = n_seqs, max_rows
        self.cu_rows = torch.zeros(n_seqs + 1, dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(n_seqs, dtype=torch.int32, device=device)
        self.row_seq = torch.full((max_rows,), -1, dtype=torch.int32, device=device)
        self.positions = torch.full((max_rows,), -1, dtype=torch.int32, device=device)
        self.slots = torch.full((max_rows,), -1, dtype=torch.int64, device=device)

    def next_cached(self, cached, fresh, out=None):
        """The tokens that each request holds after the step whose plan this is, from the step's cached and
        fresh: the next step's cached.  kv_len for served requests; a refused one keeps its cached tokens (its
        kv_len is 0, so that attention passes over it), an ended one has none.  Into `out` (which may be
        cached) if given; on the current stream."""
        import torch
        new = torch.where(self.kv_len > 0, self.kv_len, cached).masked_fill_(fresh < 0, 0)
        return new if out is None else out.copy_(new)


def rz_paged_plan(cached, fresh, n_seqs, owned, owned_out, free_count, free_count_out, free_pages, n_pages, block_table,
                  ld_table, max_blocks, page_size, max_rows, cu_rows, kv_len, row_seq, positions, slots, stream=None):
    return call("rz_paged_plan", _ptr(cached), _ptr(fresh), n_seqs, _ptr(owned), _ptr(owned_out), _ptr(free_count),
                _ptr(free_count_out), _ptr(free_pages), n_pages, _ptr(block_table), ld_table, max_blocks, page_size,
                max_rows, _ptr(cu_rows), _ptr(kv_len), _ptr(row_seq), _ptr(positions), _ptr(slots), _stream(stream))


def paged_plan(cached, fresh, block_table, owned, free_pages, free_count, page_size: int, out: PagedPlan, owned_out=None,
               free_count_out=None, stream=None) -> PagedPlan:
    """Pages, slots, positions and row offsets of one step (see rz.h), into `out`.

    cached, fresh, owned int32 [n]; block_table int32 [n, max_blocks]; free_pages int32
    [n_pages] and free_count int32 [1]: the pool.  owned and free_count are updated in
    place unless owned_out / free_count_out take the new state."""
    import torch
    i32, dev, n = torch.int32, torch.cuda.current_device(), out.n_seqs
    _on_device(block_table, i32, 2, dev, "block_table")
    rows, max_blocks = block_table.shape
    if rows != n:
        raise ValueError(f"block_table must have {n} rows")
    _on_device(out.slots, torch.int64, 1, dev, "out")
    _on_device(free_pages, i32, 1, dev, "free_pages")
    n_pages = free_pages.shape[0]
    owned_at, count_at = _vector(owned, i32, n, dev, "owned"), _vector(free_count, i32, 1, dev, "free_count")
    call("rz_paged_plan", _vector(cached, i32, n, dev, "cached"), _vector(fresh, i32, n, dev, "fresh"), n, owned_at,
         owned_at if owned_out is None else _vector(owned_out, i32, n, dev, "owned_out"), count_at,
         count_at if free_count_out is None else _vector(free_count_out, i32, 1, dev, "free_count_out"),
         _vector(free_pages, i32, n_pages, dev, "free_pages"), n_pages, block_table.data_ptr(),
         _row_ld(block_table, max_blocks, "block_table"), max_blocks, page_size, out.max_rows, out.cu_rows.data_ptr(),
         out.kv_len.data_ptr(), out.row_seq.data_ptr(), out.positions.data_ptr(), out.slots.data_ptr(),
         _stream_on(stream, dev))
    return out


def rz_qk_norm_rope(q, ld_q, k, ld_k, v, ld_v, q_gamma, k_gamma, eps, positions, slots, kv, n_rows, n_heads, n_kv_heads,
                    head_dim, rope_theta, rope_mode, q_out, ld_qo, k_out, v_out, stream=None):
    return call("rz_qk_norm_rope", _ptr(q), ld_q, _ptr(k), ld_k, _ptr(v), ld_v, _ptr(q_gamma), _ptr(k_gamma), eps,
                _ptr(positions), _ptr(slots), None if kv is None else kv.ref, n_rows, n_heads, n_kv_heads, head_dim,
                rope_theta, rope_mode, _ptr(q_out), ld_qo, _ptr(k_out), _ptr(v_out), _stream(stream))


def qk_norm_rope(q, k, v, positions, n_heads: int, n_kv_heads: int, head_dim: int, rope_theta: float, rope_mode: int,
                 q_gamma=None, k_gamma=None, eps: float = 1e-6, kv: PagedKVQ4 = None, slots=None, q_out=None,
                 want_k: bool = False, want_v: bool = False, stream=None):
    """Norm each head of q and k (f32 [n, heads * head_dim], rows may be strided), rotate them,
    and append k and v to the cache `kv` at `slots` (see rz.h).  Returns (q, k, v): k and
    v as the cache holds them when asked for (else None); without a cache k is the rotated k."""
    import torch
    f32, dev = torch.float32, torch.cuda.current_device()
    n = _on_device(q, f32, 2, dev, "q").shape[0]
    if _on_device(k, f32, 2, dev, "k").shape[0] != n:
        raise ValueError("k must have a row for each of q")
    q_dim, kv_dim = n_heads * head_dim, n_kv_heads * head_dim
    ref = v_at = slots_at = None
    ld_v = kv_dim
    if kv is None:
        if want_v or slots is not None:
            raise ValueError("slots and want_v need a cache")
        want_k = True
    else:
        if _on_device(v, f32, 2, dev, "v").shape[0] != n:
            raise ValueError("v must have a row for each of q")
        if kv.dev != dev:
            raise ValueError("the cache is not on the current device")
        ref, v_at, ld_v = kv.ref, v.data_ptr(), _row_ld(v, kv_dim, "v")
        slots_at = _vector(slots, torch.int64, n, dev, "slots", more=True)
    pos_at = _vector(positions, torch.int32, n, dev, "positions", more=True)
    qg_at = None if q_gamma is None else _vector(q_gamma, f32, head_dim, dev, "q_gamma")
    kg_at = None if k_gamma is None else _vector(k_gamma, f32, head_dim, dev, "k_gamma")
    if q_out is None:
        q_out, ld_qo = _new((n, q_dim), f32, dev, stream), q_dim
    else:
        if _on_device(q_out, f32, 2, dev, "q_out").shape[0] != n:
            raise ValueError("q_out must have a row for each of q")
        ld_qo = _row_ld(q_out, q_dim, "q_out")
    k_out = _new((n, kv_dim), f32, dev, stream) if want_k else None
    v_out = _new((n, kv_dim), f32, dev, stream) if want_v else None
    call("rz_qk_norm_rope", q.data_ptr(), _row_ld(q, q_dim, "q"), k.data_ptr(), _row_ld(k, kv_dim, "k"), v_at, ld_v, qg_at,
         kg_at, eps, pos_at, slots_at, ref, n, n_heads, n_kv_heads, head_dim, rope_theta, rope_mode, q_out.data_ptr(), ld_qo,
         None if k_out is None else k_out.data_ptr(), None if v_out is None else v_out.data_ptr(), _stream_on(stream, dev))
    return q_out, k_out, v_out


def rz_attention_paged_q4(q, ld_q, n_rows, kv, block_table, ld_table, max_blocks, cu_rows, kv_len, n_seqs, n_heads, scale,
                          att, att_q8, ws, ws_bytes, stream=None):
    return call("rz_attention_paged_q4", _ptr(q), ld_q, n_rows, kv.ref, _ptr(block_table), ld_table, max_blocks,
                _ptr(cu_rows), _ptr(kv_len), n_seqs, n_heads, scale, _ptr(att), _ptr(att_q8), _ptr(ws), ws_bytes,
                _stream(stream))


def attention_paged_q4_workspace_bytes(n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(load().rz_attention_paged_q4_workspace_bytes(n_heads, n_kv_heads, head_dim))


def attention_paged_q4(q, kv: PagedKVQ4, block_table, cu_rows, kv_len, n_heads: int, scale: float = 0.0, out=None, ws=None,
                       att_q8=None, stream=None):
    """Attention of each request's new rows of q (f32 [n_rows, n_heads * head_dim]) over its
    pages (see rz.h); returns f32 [n_rows, n_heads * head_dim] (rows behind the last request's as
    they were in `out`).  att_q8: a uint8 tensor of q8_1_size(n_rows, q_pad) for the Q8_1 form."""
    import torch
    i32, dev = torch.int32, torch.cuda.current_device()
    n_rows = _on_device(q, torch.float32, 2, dev, "q").shape[0]
    q_dim = n_heads * kv.head_dim
    if kv.dev != dev:
        raise ValueError("the cache is not on the current device")
    n, max_blocks = _on_device(block_table, i32, 2, dev, "block_table").shape
    if out is None:
        out = _new((n_rows, q_dim), torch.float32, dev, stream)
    elif _on_device(out, torch.float32, 2, dev, "out").shape != (n_rows, q_dim) or not out.is_contiguous():
        raise ValueError("out must be contiguous, with the shape of q")
    q8_at = None
    if att_q8 is not None:
        q8_at = _vector(att_q8, torch.uint8, q8_1_size(n_rows, -(-q_dim // 256) * 256), dev, "att_q8", more=True)
    if ws is None:
        size = max(attention_paged_q4_workspace_bytes(n_heads, kv.n_kv_heads, kv.head_dim), 16)
        ws = _new((size,), torch.uint8, dev, stream)
        with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                               torch.cuda.ExternalStream(_stream_on(stream, dev))):
            ws.zero_()
    call("rz_attention_paged_q4", q.data_ptr(), _row_ld(q, q_dim, "q"), n_rows, kv.ref, block_table.data_ptr(),
         _row_ld(block_table, max_blocks, "block_table"), max_blocks, _vector(cu_rows, i32, n + 1, dev, "cu_rows"),
         _vector(kv_len, i32, n, dev, "kv_len"), n, n_heads, scale, out.data_ptr(), q8_at,
         _vector(ws, torch.uint8, 0, dev, "ws", more=True), ws.shape[0], _stream_on(stream, dev))
    return out


def decode_layer_paged_workspace_bytes(layer: DeviceLayer, m: int) -> int:
    return int(load().rz_decode_layer_paged_workspace_bytes(C.byref(layer.struct), m))


def decode_layer_paged(x, layer: DeviceLayer, kv: PagedKVQ4, block_table, plan: PagedPlan, q_gamma=None, k_gamma=None,
                       out=None, ws=None, stream=None):
    """One decode step of one layer over the paged 4-bit cache, for the rows of `plan` (see
    rz.h).  x f32 [m, hidden_pad], m up to 16 and to plan.max_rows; the plan serves every layer of the step."""
    import torch
    i32, dev = torch.int32, torch.cuda.current_device()
    m, width = _on_device(x, torch.float32, 2, dev, "x").shape
    if width != layer.hidden_pad or not x.is_contiguous():
        raise ValueError("x must be contiguous [m, hidden_pad]")
    if m > plan.max_rows or kv.dev != dev:
        raise ValueError("the plan has fewer rows than x, or the cache is on another device")
    n, max_blocks = _on_device(block_table, i32, 2, dev, "block_table").shape
    if n != plan.n_seqs:
        raise ValueError("block_table must have a row for each request of the plan")
    gammas = [None if t is None else _vector(t, torch.float32, layer.head_dim, dev, name)
              for name, t in (("q_gamma", q_gamma), ("k_gamma", k_gamma))]
    if out is None:
        out = _new((m, width), torch.float32, dev, stream)
    elif _on_device(out, torch.float32, 2, dev, "out").shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, with the shape of x")
    if ws is None:
        ws = _new((max(decode_layer_paged_workspace_bytes(layer, m), 16),), torch.uint8, dev, stream)
        with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                               torch.cuda.ExternalStream(_stream_on(stream, dev))):
            ws.zero_()
    call("rz_decode_layer_paged", x.data_ptr(), C.byref(layer.struct), *gammas, kv.ref,
         _on_device(plan.positions, i32, 1, dev, "plan").data_ptr(), plan.slots.data_ptr(), block_table.data_ptr(),
         _row_ld(block_table, max_blocks, "block_table"), max_blocks, plan.cu_rows.data_ptr(), plan.kv_len.data_ptr(), n, m,
         out.data_ptr(), _vector(ws, torch.uint8, 0, dev, "ws", more=True), ws.shape[0], _stream_on(stream, dev))
    return out


# ------------------------------------------------------------------ an FFN of experts
def rz_residual_rmsnorm(x, delta, gamma, sum, y, q8, m, n, n_pad, eps, stream=None):
    return call("rz_residual_rmsnorm", _ptr(x), _ptr(delta), _ptr(gamma), _ptr(sum), _ptr(y), _ptr(q8), m, n, n_pad, eps,
                _stream(stream))


def _matrix(t, dtype, rows, cols, dev, name):
    """The address of a contiguous tensor [rows, cols]."""
    try:
        if t.get_device() == dev and t.dtype == dtype and t.shape == (rows, cols) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _on_device(t, dtype, 2, dev, name)
    raise ValueError(f"{name} must be contiguous [{rows}, {cols}], got {list(t.shape)}")


def _values(t, dtype, n, dev, name):
    """The address of a contiguous tensor of n values."""
    try:
        if t.get_device() == dev and t.dtype == dtype and t.shape == (n,) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _vector(t, dtype, n, dev, name)


def residual_rmsnorm(x, delta, gamma, n: int, n_pad: int, eps: float, want_y: bool = True, want_q8: bool = True, sum_out=None,
                     stream=None):
    """x + delta (f32 [m, n_pad] each; delta may be None), its RMSNorm and the Q8_1 form of that (see rz.h), in
    one pass.  Returns (sum, y, q8), y and q8 None where not wanted; sum_out may be x or delta."""
    import torch
    f32, dev = torch.float32, torch.cuda.current_device()
    m = _on_device(x, f32, 2, dev, "x").shape[0]
    x_at = _matrix(x, f32, m, n_pad, dev, "x")
    delta_at = None if delta is None else _matrix(delta, f32, m, n_pad, dev, "delta")
    gamma_at = _values(gamma, f32, n, dev, "gamma")
    if sum_out is None:
        sum_out = _new((m, n_pad), f32, dev, stream)
        sum_at = sum_out.data_ptr()
    else:
        sum_at = _matrix(sum_out, f32, m, n_pad, dev, "sum_out")
    y = _new((m, n_pad), f32, dev, stream) if want_y else None
    q8 = _new((q8_1_size(m, n_pad),), torch.uint8, dev, stream) if want_q8 else None
    call("rz_residual_rmsnorm", x_at, delta_at, gamma_at, sum_at, None if y is None else y.data_ptr(), None if q8 is None else q8.data_ptr(), m,
         n, n_pad, eps, _stream_on(stream, dev))
    return sum_out, y, q8


class MoePlan:
    """Which experts the tokens of a batch go to (rz_moe_plan): experts, weights [n_tokens, top_k], offsets
    [n_experts + 1], rows and places [n_tokens * top_k]; moe_route fills it, and it is kept from step
    to step.  Tensors given by name are taken as they are."""

    def __init__(self, n_tokens: int, n_experts: int, top_k: int, device="cuda", **given):
        import torch
        from ._lib import MoePlanStruct
        i32, pairs = torch.int32, n_tokens * top_k
        shapes = {"experts": ((n_tokens, top_k), i32), "weights": ((n_tokens, top_k), torch.float32), "offsets": ((n_experts + 1,), i32),
                  "rows": ((pairs,), i32), "places": ((pairs,), i32)}
        if not set(given) <= set(shapes):
            raise TypeError(f"unknown tensors {sorted(set(given) - set(shapes))}")
        self.n_tokens, self.n_experts, self.top_k = n_tokens, n_experts, top_k
        for name, (shape, dtype) in shapes.items():
            t = given.get(name)
            if t is None:
                t = torch.zeros(shape, dtype=dtype, device=device)
            elif _on_device(t, dtype, len(shape), t.get_device(), name).shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {list(shape)}")
            setattr(self, name, t)
        self.dev = self.experts.get_device()
        if any(getattr(self, name).get_device() != self.dev for name in shapes):
            raise ValueError("the tensors of a plan must be on one device")
        self.struct = MoePlanStruct(*[getattr(self, name).data_ptr() for name in shapes], n_tokens, n_experts, top_k)
        self.ref = C.byref(self.struct)


def _plan_on(plan, dev):
    if plan.dev != dev:
        raise ValueError("the plan is not on the current device")
    return plan.ref


def moe_route_workspace_bytes(n_tokens: int, n_experts: int) -> int:
    return int(load().rz_moe_route_workspace_bytes(n_tokens, n_experts))


def rz_moe_route(logits, ld, row_seq, plan, renormalise, scale, ws, ws_bytes, stream=None):
    return call("rz_moe_route", _ptr(logits), ld, _ptr(row_seq), plan.ref, renormalise, scale, _ptr(ws), ws_bytes, _stream(stream))


def _scratch(ws, need, dev, stream):
    """(address, bytes, tensor) of the workspace given, or of a new one of need() bytes."""
    import torch
    if ws is None:
        size = need()
        if size == 0:
            return None, 0, None
        ws = _new((size,), torch.uint8, dev, stream)
    return _vector(ws, torch.uint8, 0, dev, "ws", more=True), ws.shape[0], ws


def moe_route(logits, plan: MoePlan, renormalise: bool = True, scale: float = 1.0, row_seq=None, ws=None, stream=None) -> MoePlan:
    """The top_k experts of each token by its logits (f32 [n_tokens, n_experts], rows may be strided), their softmax
    weights, and the rows by expert (see rz.h), into `plan`.  row_seq int32 [n_tokens]: negative for tokens without
    a request."""
    import torch
    dev = torch.cuda.current_device()
    if _on_device(logits, torch.float32, 2, dev, "logits").shape[0] != plan.n_tokens:
        raise ValueError("logits must have a row for each token of the plan")
    at, size, ws = _scratch(ws, lambda: moe_route_workspace_bytes(plan.n_tokens, plan.n_experts), dev, stream)
    call("rz_moe_route", logits.data_ptr(), _row_ld(logits, plan.n_experts, "logits"),
         None if row_seq is None else _vector(row_seq, torch.int32, plan.n_tokens, dev, "row_seq", more=True), _plan_on(plan, dev),
         1 if renormalise else 0, scale, at, size, _stream_on(stream, dev))
    return plan


def _expert_weights(w, n_experts, out_dim, in_dim, dev, name):
    """The address of Q4_K weights [n_experts][out_dim][in_dim]: a contiguous uint8 tensor of any shape."""
    import torch
    try:
        if w.get_device() == dev and w.dtype == torch.uint8 and w.is_contiguous() and w.numel() == n_experts * out_dim * (in_dim // 256) * 144:
            return w.data_ptr()
    except AttributeError:
        pass
    _on_device(w, torch.uint8, w.dim() if hasattr(w, "dim") else 0, dev, name)
    raise ValueError(f"{name} must hold {n_experts} x {out_dim} x {in_dim} Q4_K weights, contiguous")


def moe_swiglu_workspace_bytes(n_tokens: int, n_experts: int, top_k: int, in_dim: int) -> int:
    return int(load().rz_moe_swiglu_workspace_bytes(n_tokens, n_experts, top_k, in_dim))


def rz_moe_swiglu(w_gate, w_up, x_q8, plan, inter, in_dim, h, h_q8, ws, ws_bytes, stream=None):
    return call("rz_moe_swiglu", _ptr(w_gate), _ptr(w_up), _ptr(x_q8), plan.ref, inter, in_dim, _ptr(h), _ptr(h_q8), _ptr(ws), ws_bytes,
                _stream(stream))


def moe_swiglu(w_gate, w_up, x_q8, plan: MoePlan, inter: int, in_dim: int, out=None, out_q8=None, want_h: bool = True, ws=None,
               stream=None):
    """silu(gate) * up of each row of the plan with its expert (see rz.h): f32 [n_tokens * top_k, inter] in the plan's
    order (None with want_h False), and its Q8_1 form into out_q8 where that is given."""
    import torch
    u8, dev, pairs = torch.uint8, torch.cuda.current_device(), plan.n_tokens * plan.top_k
    if out is None and want_h:
        out = _new((pairs, inter), torch.float32, dev, stream)
    at, size, ws = _scratch(ws, lambda: moe_swiglu_workspace_bytes(plan.n_tokens, plan.n_experts, plan.top_k, in_dim), dev, stream)
    call("rz_moe_swiglu", _expert_weights(w_gate, plan.n_experts, inter, in_dim, dev, "w_gate"),
         _expert_weights(w_up, plan.n_experts, inter, in_dim, dev, "w_up"),
         _values(x_q8, u8, q8_1_size(plan.n_tokens, in_dim), dev, "x_q8"), _plan_on(plan, dev), inter, in_dim,
         None if out is None else _matrix(out, torch.float32, pairs, inter, dev, "out"),
         None if out_q8 is None else _values(out_q8, u8, q8_1_size(pairs, inter), dev, "out_q8"), at, size, _stream_on(stream, dev))
    return out


def moe_down_workspace_bytes(n_tokens: int, n_experts: int, top_k: int, out_dim: int, in_dim: int) -> int:
    return int(load().rz_moe_down_workspace_bytes(n_tokens, n_experts, top_k, out_dim, in_dim))


def rz_moe_down(w_down, h_q8, plan, residual, y, out_dim, out_pad, in_dim, ws, ws_bytes, stream=None):
    return call("rz_moe_down", _ptr(w_down), _ptr(h_q8), plan.ref, _ptr(residual), _ptr(y), out_dim, out_pad, in_dim, _ptr(ws), ws_bytes,
                _stream(stream))


def moe_down(w_down, h_q8, plan: MoePlan, out_dim: int, in_dim: int, residual=None, out=None, out_pad: int = 0, ws=None, stream=None):
    """The product back of each row of the plan, the weighted sum of a token's rows and the residual (see rz.h):
    f32 [n_tokens, out_pad or out_dim].  out may be residual."""
    import torch
    f32, dev, out_pad = torch.float32, torch.cuda.current_device(), out_pad or out_dim
    if out is None:
        out = _new((plan.n_tokens, out_pad), f32, dev, stream)
        out_at = out.data_ptr()
    else:
        out_at = _matrix(out, f32, plan.n_tokens, out_pad, dev, "out")
    at, size, ws = _scratch(ws, lambda: moe_down_workspace_bytes(plan.n_tokens, plan.n_experts, plan.top_k, out_dim, in_dim), dev, stream)
    call("rz_moe_down", _expert_weights(w_down, plan.n_experts, out_dim, in_dim, dev, "w_down"),
         _values(h_q8, torch.uint8, q8_1_size(plan.n_tokens * plan.top_k, in_dim), dev, "h_q8"), _plan_on(plan, dev),
         None if residual is None else _matrix(residual, f32, plan.n_tokens, out_pad, dev, "residual"),
         out_at, out_dim, out_pad, in_dim, at, size, _stream_on(stream, dev))
    return out


def moe_ffn_workspace_bytes(n_tokens: int, n_experts: int, top_k: int, hidden: int, hidden_pad: int, inter: int) -> int:
    return int(load().rz_moe_ffn_workspace_bytes(n_tokens, n_experts, top_k, hidden, hidden_pad, inter))


def rz_moe_ffn(logits, ld, row_seq, x_q8, w_gate, w_up, w_down, residual, out, plan, renormalise, scale, hidden, hidden_pad, inter, ws,
               ws_bytes, stream=None):
    return call("rz_moe_ffn", _ptr(logits), ld, _ptr(row_seq), _ptr(x_q8), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(residual), _ptr(out),
                plan.ref, renormalise, scale, hidden, hidden_pad, inter, _ptr(ws), ws_bytes, _stream(stream))


def moe_ffn(logits, x_q8, w_gate, w_up, w_down, plan: MoePlan, hidden: int, hidden_pad: int, inter: int, renormalise: bool = True,
            scale: float = 1.0, row_seq=None, residual=None, out=None, ws=None, stream=None):
    """moe_route, moe_swiglu and moe_down in one call (see rz.h): f32 [n_tokens, hidden_pad].  out may be residual."""
    import torch
    f32, dev, T, E = torch.float32, torch.cuda.current_device(), plan.n_tokens, plan.n_experts
    if _on_device(logits, f32, 2, dev, "logits").shape[0] != T:
        raise ValueError("logits must have a row for each token of the plan")
    if out is None:
        out = _new((T, hidden_pad), f32, dev, stream)
    at, size, ws = _scratch(ws, lambda: moe_ffn_workspace_bytes(T, E, plan.top_k, hidden, hidden_pad, inter), dev, stream)
    call("rz_moe_ffn", logits.data_ptr(), _row_ld(logits, E, "logits"),
         None if row_seq is None else _vector(row_seq, torch.int32, T, dev, "row_seq", more=True),
         _values(x_q8, torch.uint8, q8_1_size(T, hidden_pad), dev, "x_q8"), _expert_weights(w_gate, E, inter, hidden_pad, dev, "w_gate"),
         _expert_weights(w_up, E, inter, hidden_pad, dev, "w_up"), _expert_weights(w_down, E, hidden, inter, dev, "w_down"),
         None if residual is None else _matrix(residual, f32, T, hidden_pad, dev, "residual"), _matrix(out, f32, T, hidden_pad, dev, "out"),
         _plan_on(plan, dev), 1 if renormalise else 0, scale, hidden, hidden_pad, inter, at, size, _stream_on(stream, dev))
    return out
