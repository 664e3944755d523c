// abi_moe.cu -- the extern "C" boundary of an FFN of experts: argument checks of its
// entry points (see abi.cu for the conventions).  Every check runs on the host before any
// launch.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/rz.h"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
rz_status record_error(rz_status st, const char *msg);
rz_status ensure_device();
}  // namespace rz

using namespace rz;

namespace {

rz_status fail(rz_status st, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return record_error(st, buf);
}

#define RZ_TRY(expr)                  \
    do {                              \
        rz_status _st = (expr);       \
        if (_st != RZ_OK) return _st; \
    } while (0)

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

rz_status launched(const char *fn, cudaError_t e)
{
    if (e == cudaSuccess) return RZ_OK;
    return fail(RZ_ERR_CUDA, "%s launch: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr int64_t kMaxDim = int64_t(1) << 20;  // of a row, in values

rz_status check_counts(const char *fn, int64_t n_tokens, int32_t n_experts, int32_t top_k)
{
    if (n_experts < 1 || n_experts > kMoeMaxExperts)
        return fail(RZ_ERR_SHAPE, "%s: n_experts=%d outside [1, %d]", fn, n_experts, kMoeMaxExperts);
    if (top_k < 1 || top_k > kMoeMaxTopK || top_k > n_experts)
        return fail(RZ_ERR_SHAPE, "%s: top_k=%d with %d experts (at most %d)", fn, top_k, n_experts, kMoeMaxTopK);
    if (n_tokens < 1) return fail(RZ_ERR_INVALID_ARG, "%s: n_tokens=%lld", fn, (long long)n_tokens);
    if (n_tokens > kMoeMaxPairs / top_k)
        return fail(RZ_ERR_SHAPE, "%s: n_tokens=%lld times top_k=%d is more than %lld rows", fn, (long long)n_tokens, top_k, (long long)kMoeMaxPairs);
    return RZ_OK;
}

rz_status check_plan(const char *fn, const rz_moe_plan *p)
{
    if (!p) return fail(RZ_ERR_INVALID_ARG, "%s: null plan", fn);
    const void *words[] = {p->experts, p->weights, p->offsets, p->rows, p->places};
    for (const void *w : words)
        if (!w) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer in the plan", fn);
    for (const void *w : words)
        if (!aligned(w, 4)) return fail(RZ_ERR_ALIGN, "%s: the plan's buffers must be 4-byte aligned", fn);
    return check_counts(fn, p->n_tokens, p->n_experts, p->top_k);
}

rz_status check_in_dim(const char *fn, int64_t in_dim)
{
    if (in_dim < 256 || in_dim % 256 || in_dim > kMaxDim)
        return fail(RZ_ERR_SHAPE, "%s: in_dim=%lld is not a multiple of 256 up to %lld", fn, (long long)in_dim, (long long)kMaxDim);
    return RZ_OK;
}

rz_status check_out_dim(const char *fn, const char *name, int64_t out_dim)
{
    if (out_dim < 1 || out_dim > kMaxDim) return fail(RZ_ERR_SHAPE, "%s: %s=%lld", fn, name, (long long)out_dim);
    return RZ_OK;
}

struct Q8 {
    const int8_t *q;
    const float *d, *s;
};
Q8 q8_parts(const void *p, int64_t m, int64_t n)
{
    const int8_t *q = static_cast<const int8_t *>(p);
    const float *d = reinterpret_cast<const float *>(q + m * n);
    return {q, d, d + m * (n / 32)};
}

void fill(MoeGemvArgs &a, const rz_moe_plan *p, int64_t out_dim, int64_t in_dim)
{
    a.offsets = p->offsets;
    a.out_dim = out_dim;
    a.in_dim = static_cast<int>(in_dim);
    a.n_experts = p->n_experts;
    a.top_k = p->top_k;
    a.n_pairs = static_cast<int>(p->n_tokens * p->top_k);
    a.err = dev_error_word();
}

void swiglu_args(MoeGemvArgs &a, const void *w_gate, const void *w_up, const void *x_q8, const rz_moe_plan *p, int64_t inter,
                 int64_t in_dim, float *h, void *h_q8)
{
    fill(a, p, inter, in_dim);
    const Q8 x = q8_parts(x_q8, p->n_tokens, in_dim), o = q8_parts(h_q8, a.n_pairs, inter);
    a.w1 = static_cast<const uint8_t *>(w_gate);
    a.w2 = static_cast<const uint8_t *>(w_up);
    a.xq = x.q;
    a.xd = x.d;
    a.xs = x.s;
    a.rows = p->rows;
    a.y = h;
    a.yq = h_q8 ? const_cast<int8_t *>(o.q) : nullptr;
    a.yd = const_cast<float *>(o.d);
    a.ys = const_cast<float *>(o.s);
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// the activations as the tensor-core kernel takes them, if that can be the one; the integer kernel needs nothing
int64_t swiglu_pack_bytes(int64_t n_pairs, int n_experts, int64_t in_dim)
{
    return moe_pack_bytes(moe_tiles(n_pairs, n_experts, true), n_pairs, n_experts, in_dim);
}

// the rows' products, in how many parts, then B
int64_t down_products_bytes(int64_t pairs, int parts, int64_t out_dim) { return align256(parts * pairs * out_dim * 4) + (parts > 1 ? 256 : 0); }

int64_t down_workspace_bytes(int64_t n_tokens, int n_experts, int top_k, int64_t out_dim, int64_t in_dim)
{
    const int64_t pairs = n_tokens * top_k;
    const int columns = moe_columns(pairs, n_experts, top_k, out_dim, in_dim, false);
    if (columns == 0) return 0;
    return down_products_bytes(pairs, moe_max_parts(columns, pairs, out_dim, in_dim), out_dim) + moe_pack_bytes(columns, pairs, n_experts, in_dim);
}

cudaError_t run_swiglu(const MoeGemvArgs &a, void *workspace, cudaStream_t s)
{
    const int columns = moe_columns(a.n_pairs, a.n_experts, a.top_k, a.out_dim, a.in_dim, true);
    return columns ? launch_moe_gemm_tc(a, columns, workspace, s) : launch_moe_swiglu(a, s);
}

cudaError_t run_down(const void *w_down, const void *h_q8, const rz_moe_plan *p, const float *residual, float *y, int64_t out_dim,
                     int64_t out_pad, int64_t in_dim, void *workspace, cudaStream_t s)
{
    MoeGemvArgs a{};
    fill(a, p, out_dim, in_dim);
    const Q8 h = q8_parts(h_q8, a.n_pairs, in_dim);
    a.w1 = static_cast<const uint8_t *>(w_down);
    a.xq = h.q;
    a.xd = h.d;
    a.xs = h.s;
    a.y = static_cast<float *>(workspace);
    MoeCombineArgs c{};
    c.o = a.y;
    c.experts = p->experts;
    c.places = p->places;
    c.offsets = p->offsets;
    c.weights = p->weights;
    c.residual = residual;
    c.y = y;
    c.out_dim = static_cast<int>(out_dim);
    c.out_pad = static_cast<int>(out_pad);
    c.n_experts = p->n_experts;
    c.top_k = p->top_k;
    c.n_pairs = a.n_pairs;
    c.err = a.err;
    const int columns = moe_columns(a.n_pairs, a.n_experts, a.top_k, out_dim, in_dim, false);
    if (columns == 0) return launch_moe_down_tokens(a, c, p->n_tokens, s);
    a.max_parts = moe_max_parts(columns, a.n_pairs, out_dim, in_dim);
    uint8_t *pack = static_cast<uint8_t *>(workspace) + down_products_bytes(a.n_pairs, a.max_parts, out_dim);
    if (a.max_parts > 1) c.parts = a.parts = reinterpret_cast<int32_t *>(pack - 256);
    const cudaError_t e = launch_moe_gemm_tc(a, columns, pack, s);
    return e != cudaSuccess ? e : launch_moe_combine(c, p->n_tokens, s);
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

rz_status check_workspace(const char *fn, const void *ws, size_t have, size_t need)
{
    if (need == 0) return RZ_OK;
    if (!ws) return fail(RZ_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (!aligned(ws, 16)) return fail(RZ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    if (have < need) return fail(RZ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, have, need);
    return RZ_OK;
}

rz_status check_route(const char *fn, const float *logits, int64_t ld, const int32_t *row_seq, const rz_moe_plan *p, float scale)
{
    if (!logits) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    RZ_TRY(check_plan(fn, p));
    if (!aligned(logits, 4) || !aligned(row_seq, 4)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 4-byte aligned", fn);
    if (ld < p->n_experts) return fail(RZ_ERR_SHAPE, "%s: ld=%lld < %d experts", fn, (long long)ld, p->n_experts);
    if (!std::isfinite(scale)) return fail(RZ_ERR_INVALID_ARG, "%s: scale", fn);
    return RZ_OK;
}

cudaError_t run_route(const float *logits, int64_t ld, const int32_t *row_seq, const rz_moe_plan *p, int32_t renormalise, float scale,
                      void *workspace, cudaStream_t s)
{
    MoeRouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.row_seq = row_seq;
    a.n_tokens = p->n_tokens;
    a.n_experts = p->n_experts;
    a.top_k = p->top_k;
    a.renormalise = renormalise;
    a.scale = scale;
    a.experts = p->experts;
    a.weights = p->weights;
    a.offsets = p->offsets;
    a.rows = p->rows;
    a.places = p->places;
    a.hist = static_cast<int32_t *>(workspace);
    return launch_moe_route(a, s);
}

rz_status check_down(const char *fn, const void *w_down, const float *residual, const float *y, int64_t out_dim, int64_t out_pad,
                     int64_t in_dim)
{
    if (!w_down || !y) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    RZ_TRY(check_out_dim(fn, "out_dim", out_dim));
    if (out_pad < out_dim || out_pad > kMaxDim) return fail(RZ_ERR_SHAPE, "%s: out_pad=%lld", fn, (long long)out_pad);
    RZ_TRY(check_in_dim(fn, in_dim));
    if (!aligned(w_down, 16) || !aligned(residual, 16) || !aligned(y, 16))
        return fail(RZ_ERR_ALIGN, "%s: buffers must be 16-byte aligned", fn);
    return RZ_OK;
}

}  // namespace

extern "C" {

rz_status rz_residual_rmsnorm(const float *x, const float *delta, const float *gamma, float *sum, float *y, void *q8, int64_t m,
                              int64_t n, int64_t n_pad, float eps, rz_stream stream)
{
    const char *fn = "rz_residual_rmsnorm";
    record_error(RZ_OK, "");
    if (!x || !gamma || (!y && !q8)) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (m < 1 || n < 1 || n_pad < n) return fail(RZ_ERR_INVALID_ARG, "%s: m=%lld n=%lld n_pad=%lld", fn, (long long)m, (long long)n, (long long)n_pad);
    if (m > (1 << 30)) return fail(RZ_ERR_SHAPE, "%s: m=%lld", fn, (long long)m);
    if (n_pad > 16384) return fail(RZ_ERR_UNSUPPORTED, "%s: rows longer than 16384 values", fn);
    if (n_pad % 32) return fail(RZ_ERR_SHAPE, "%s: n_pad=%lld is not a multiple of 32", fn, (long long)n_pad);
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(RZ_ERR_INVALID_ARG, "%s: eps", fn);
    if (y && y == sum) return fail(RZ_ERR_INVALID_ARG, "%s: y and sum are one buffer", fn);
    const void *bufs[] = {x, delta, gamma, sum, y, q8};
    for (const void *p : bufs)
        if (!aligned(p, 16)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 16-byte aligned", fn);
    RZ_TRY(ensure_device());
    return launched(fn, launch_residual_rmsnorm(x, delta, gamma, sum, y, q8, m, n, n_pad, eps, static_cast<cudaStream_t>(stream)));
}

size_t rz_moe_route_workspace_bytes(int64_t n_tokens, int32_t n_experts)
{
    const char *fn = "rz_moe_route_workspace_bytes";
    record_error(RZ_OK, "");
    if (check_counts(fn, n_tokens, n_experts, 1) != RZ_OK) return 0;
    return align16(moe_route_workspace_bytes(n_tokens, n_experts));
}

rz_status rz_moe_route(const float *logits, int64_t ld, const int32_t *row_seq, const rz_moe_plan *plan, int32_t renormalise, float scale,
                       void *workspace, size_t ws_bytes, rz_stream stream)
{
    const char *fn = "rz_moe_route";
    record_error(RZ_OK, "");
    RZ_TRY(check_route(fn, logits, ld, row_seq, plan, scale));
    RZ_TRY(check_workspace(fn, workspace, ws_bytes, moe_route_workspace_bytes(plan->n_tokens, plan->n_experts)));
    RZ_TRY(ensure_device());
    return launched(fn, run_route(logits, ld, row_seq, plan, renormalise != 0, scale, workspace, static_cast<cudaStream_t>(stream)));
}

size_t rz_moe_swiglu_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t top_k, int64_t in_dim)
{
    const char *fn = "rz_moe_swiglu_workspace_bytes";
    record_error(RZ_OK, "");
    if (check_counts(fn, n_tokens, n_experts, top_k) != RZ_OK || check_in_dim(fn, in_dim) != RZ_OK) return 0;
    return swiglu_pack_bytes(n_tokens * top_k, n_experts, in_dim);
}

rz_status rz_moe_swiglu(const void *w_gate, const void *w_up, const void *x_q8, const rz_moe_plan *plan, int64_t inter, int64_t in_dim,
                        float *h, void *h_q8, void *workspace, size_t ws_bytes, rz_stream stream)
{
    const char *fn = "rz_moe_swiglu";
    record_error(RZ_OK, "");
    if (!w_gate || !w_up || !x_q8 || (!h && !h_q8)) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    RZ_TRY(check_plan(fn, plan));
    RZ_TRY(check_out_dim(fn, "inter", inter));
    if (h_q8 && inter % 32) return fail(RZ_ERR_SHAPE, "%s: inter=%lld is not a multiple of 32, with a Q8_1 output", fn, (long long)inter);
    RZ_TRY(check_in_dim(fn, in_dim));
    const void *bufs[] = {w_gate, w_up, x_q8, h, h_q8};
    for (const void *p : bufs)
        if (!aligned(p, 16)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 16-byte aligned", fn);
    RZ_TRY(check_workspace(fn, workspace, ws_bytes, swiglu_pack_bytes(plan->n_tokens * plan->top_k, plan->n_experts, in_dim)));
    RZ_TRY(ensure_device());
    MoeGemvArgs a{};
    swiglu_args(a, w_gate, w_up, x_q8, plan, inter, in_dim, h, h_q8);
    return launched(fn, run_swiglu(a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t rz_moe_down_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t top_k, int64_t out_dim, int64_t in_dim)
{
    const char *fn = "rz_moe_down_workspace_bytes";
    record_error(RZ_OK, "");
    if (check_counts(fn, n_tokens, n_experts, top_k) != RZ_OK || check_out_dim(fn, "out_dim", out_dim) != RZ_OK || check_in_dim(fn, in_dim) != RZ_OK)
        return 0;
    return down_workspace_bytes(n_tokens, n_experts, top_k, out_dim, in_dim);
}

rz_status rz_moe_down(const void *w_down, const void *h_q8, const rz_moe_plan *plan, const float *residual, float *y, int64_t out_dim,
                      int64_t out_pad, int64_t in_dim, void *workspace, size_t ws_bytes, rz_stream stream)
{
    const char *fn = "rz_moe_down";
    record_error(RZ_OK, "");
    if (!h_q8) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    RZ_TRY(check_plan(fn, plan));
    RZ_TRY(check_down(fn, w_down, residual, y, out_dim, out_pad, in_dim));
    if (!aligned(h_q8, 16)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 16-byte aligned", fn);
    RZ_TRY(check_workspace(fn, workspace, ws_bytes, down_workspace_bytes(plan->n_tokens, plan->n_experts, plan->top_k, out_dim, in_dim)));
    RZ_TRY(ensure_device());
    return launched(fn, run_down(w_down, h_q8, plan, residual, y, out_dim, out_pad, in_dim, workspace, static_cast<cudaStream_t>(stream)));
}

// Q8_1 of h, then what routing and the products need, one after another
static size_t ffn_h_bytes(int64_t n_tokens, int top_k, int64_t inter) { return align256(RZ_Q8_1_BYTES(n_tokens * top_k, inter)); }
static size_t ffn_workspace_bytes(int64_t n_tokens, int n_experts, int top_k, int64_t hidden, int64_t hidden_pad, int64_t inter)
{
    const int64_t parts[] = {moe_route_workspace_bytes(n_tokens, n_experts), swiglu_pack_bytes(n_tokens * top_k, n_experts, hidden_pad),
                             down_workspace_bytes(n_tokens, n_experts, top_k, hidden, inter)};
    return ffn_h_bytes(n_tokens, top_k, inter) + align256(std::max({parts[0], parts[1], parts[2]}));
}

static rz_status check_ffn_dims(const char *fn, int64_t hidden, int64_t hidden_pad, int64_t inter)
{
    RZ_TRY(check_out_dim(fn, "hidden", hidden));
    RZ_TRY(check_in_dim(fn, hidden_pad));
    if (hidden_pad < hidden) return fail(RZ_ERR_SHAPE, "%s: hidden_pad=%lld < hidden=%lld", fn, (long long)hidden_pad, (long long)hidden);
    return check_in_dim(fn, inter);
}

size_t rz_moe_ffn_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t top_k, int64_t hidden, int64_t hidden_pad, int64_t inter)
{
    const char *fn = "rz_moe_ffn_workspace_bytes";
    record_error(RZ_OK, "");
    if (check_counts(fn, n_tokens, n_experts, top_k) != RZ_OK || check_ffn_dims(fn, hidden, hidden_pad, inter) != RZ_OK) return 0;
    return ffn_workspace_bytes(n_tokens, n_experts, top_k, hidden, hidden_pad, inter);
}

rz_status rz_moe_ffn(const float *logits, int64_t ld, const int32_t *row_seq, const void *x_q8, const void *w_gate, const void *w_up,
                     const void *w_down, const float *residual, float *out, const rz_moe_plan *plan, int32_t renormalise, float scale,
                     int64_t hidden, int64_t hidden_pad, int64_t inter, void *workspace, size_t ws_bytes, rz_stream stream)
{
    const char *fn = "rz_moe_ffn";
    record_error(RZ_OK, "");
    RZ_TRY(check_route(fn, logits, ld, row_seq, plan, scale));
    if (!x_q8 || !w_gate || !w_up) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    RZ_TRY(check_ffn_dims(fn, hidden, hidden_pad, inter));
    RZ_TRY(check_down(fn, w_down, residual, out, hidden, hidden_pad, inter));
    const void *bufs[] = {x_q8, w_gate, w_up};
    for (const void *p : bufs)
        if (!aligned(p, 16)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 16-byte aligned", fn);
    RZ_TRY(check_workspace(fn, workspace, ws_bytes, ffn_workspace_bytes(plan->n_tokens, plan->n_experts, plan->top_k, hidden, hidden_pad, inter)));
    RZ_TRY(ensure_device());
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *rest = static_cast<uint8_t *>(workspace) + ffn_h_bytes(plan->n_tokens, plan->top_k, inter);
    RZ_TRY(launched(fn, run_route(logits, ld, row_seq, plan, renormalise != 0, scale, rest, s)));
    MoeGemvArgs a{};
    swiglu_args(a, w_gate, w_up, x_q8, plan, inter, hidden_pad, nullptr, workspace);
    RZ_TRY(launched(fn, run_swiglu(a, rest, s)));
    return launched(fn, run_down(w_down, workspace, plan, residual, out, hidden, hidden_pad, inter, rest, s));
}

}  // extern "C"
