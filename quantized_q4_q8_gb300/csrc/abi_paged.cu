// abi_paged.cu -- the extern "C" boundary of the paged 4-bit KV cache: argument checks
// of its entry points (see abi.cu for the conventions).  Every check runs on the host
// before any launch.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/rz.h"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
rz_status record_error(rz_status st, const char *msg);
rz_status ensure_device();
rz_status check_layer_weights(const rz_layer_weights *w, const char *fn, int64_t m, LayerDesc *out);
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

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // of one request
constexpr int64_t kMaxInt = 2147483647;
constexpr int kMaxHeads = 65536;  // a row's values are counted in 32 bits

int page_log(int page_size)
{
    switch (page_size) {
        case 16: return 0;
        case 32: return 1;
        case 64: return 2;
        case 128: return 3;
        default: return -1;
    }
}

rz_status check_page_size(const char *fn, int page_size)
{
    if (page_log(page_size) < 0)
        return fail(RZ_ERR_SHAPE, "%s: page_size=%d is not 16, 32, 64 or 128", fn, page_size);
    return RZ_OK;
}

rz_status check_blocks(const char *fn, int max_blocks, int64_t ld_table, int page_size)
{
    if (max_blocks < 1 || (int64_t)max_blocks * page_size > kMaxTokens)
        return fail(RZ_ERR_SHAPE, "%s: max_blocks=%d with page_size=%d", fn, max_blocks, page_size);
    if (ld_table < max_blocks) return fail(RZ_ERR_SHAPE, "%s: ld_table=%lld < max_blocks", fn, (long long)ld_table);
    return RZ_OK;
}

rz_status check_head_dim(const char *fn, int head_dim)
{
    if (head_dim < 32 || head_dim > 256 || head_dim % 32) return fail(RZ_ERR_SHAPE, "%s: head_dim=%d", fn, head_dim);
    return RZ_OK;
}

rz_status check_kv_q4(const char *fn, const rz_kv_q4 *kv, PagedKv *out)
{
    if (!kv || !kv->pages) return fail(RZ_ERR_INVALID_ARG, "%s: null cache", fn);
    if (!aligned(kv->pages, 16)) return fail(RZ_ERR_ALIGN, "%s: the cache must be 16-byte aligned", fn);
    RZ_TRY(check_page_size(fn, kv->page_size));
    RZ_TRY(check_head_dim(fn, kv->head_dim));
    if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024) return fail(RZ_ERR_SHAPE, "%s: n_kv_heads=%d", fn, kv->n_kv_heads);
    if (kv->n_pages < 1 || kv->n_pages > kMaxInt) return fail(RZ_ERR_SHAPE, "%s: n_pages=%lld", fn, (long long)kv->n_pages);
    *out = PagedKv{static_cast<uint8_t *>(kv->pages), kv->n_pages, page_log(kv->page_size), kv->n_kv_heads, kv->head_dim};
    return RZ_OK;
}

}  // namespace

extern "C" {

size_t rz_kv_q4_page_bytes(int32_t page_size, int32_t n_kv_heads, int32_t head_dim)
{
    const char *fn = "rz_kv_q4_page_bytes";
    record_error(RZ_OK, "");
    if (check_page_size(fn, page_size) != RZ_OK || check_head_dim(fn, head_dim) != RZ_OK) return 0;
    if (n_kv_heads < 1 || n_kv_heads > 1024) {
        fail(RZ_ERR_SHAPE, "%s: n_kv_heads=%d", fn, n_kv_heads);
        return 0;
    }
    return (size_t)n_kv_heads * (page_size / 16) * q4_record_bytes(head_dim);
}

rz_status rz_paged_plan(const int32_t *cached, const int32_t *fresh, int32_t n_seqs, const int32_t *owned,
                        int32_t *owned_out, const int32_t *free_count, int32_t *free_count_out, int32_t *free_pages,
                        int64_t n_pages, int32_t *block_table, int64_t ld_table, int32_t max_blocks, int32_t page_size,
                        int64_t max_rows, int32_t *cu_rows, int32_t *kv_len, int32_t *row_seq, int32_t *positions,
                        int64_t *slots, rz_stream stream)
{
    const char *fn = "rz_paged_plan";
    record_error(RZ_OK, "");
    const void *words[] = {cached, fresh, owned, owned_out, free_count, free_count_out, free_pages, block_table,
                           cu_rows, kv_len, row_seq, positions};
    for (const void *p : words)
        if (!p) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!slots) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void *p : words)
        if (!aligned(p, 4)) return fail(RZ_ERR_ALIGN, "%s: int32 buffers must be 4-byte aligned", fn);
    if (!aligned(slots, 8)) return fail(RZ_ERR_ALIGN, "%s: slots must be 8-byte aligned", fn);
    if (n_seqs < 1 || n_seqs > kPlanMaxSeqs) return fail(RZ_ERR_SHAPE, "%s: n_seqs=%d outside [1, %d]", fn, n_seqs, kPlanMaxSeqs);
    RZ_TRY(check_page_size(fn, page_size));
    RZ_TRY(check_blocks(fn, max_blocks, ld_table, page_size));
    if (n_pages < 1 || n_pages > kMaxInt) return fail(RZ_ERR_SHAPE, "%s: n_pages=%lld", fn, (long long)n_pages);
    if (max_rows < 1 || max_rows > kMaxInt) return fail(RZ_ERR_SHAPE, "%s: max_rows=%lld", fn, (long long)max_rows);
    if (kv_len == cached || kv_len == fresh)
        return fail(RZ_ERR_INVALID_ARG, "%s: kv_len may not be cached or fresh (a refused request's length is 0 in it)", fn);
    RZ_TRY(ensure_device());
    PlanArgs a{};
    a.cached = cached;
    a.fresh = fresh;
    a.owned = owned;
    a.free_count = free_count;
    a.owned_out = owned_out;
    a.free_count_out = free_count_out;
    a.free_pages = free_pages;
    a.table = block_table;
    a.cu_rows = cu_rows;
    a.kv_len = kv_len;
    a.row_seq = row_seq;
    a.positions = positions;
    a.slots = slots;
    a.table_ld = ld_table;
    a.n_pages = n_pages;
    a.max_rows = max_rows;
    a.n_seqs = n_seqs;
    a.max_blocks = max_blocks;
    a.page_size = page_size;
    a.err = dev_error_word();
    return launched(fn, launch_paged_plan(a, static_cast<cudaStream_t>(stream)));
}

rz_status rz_qk_norm_rope(const float *q, int64_t ld_q, const float *k, int64_t ld_k, const float *v, int64_t ld_v,
                          const float *q_gamma, const float *k_gamma, float eps, const int32_t *positions,
                          const int64_t *slots, const rz_kv_q4 *kv, int64_t n_rows, int32_t n_heads, int32_t n_kv_heads,
                          int32_t head_dim, float rope_theta, int32_t rope_mode, float *q_out, int64_t ld_qo,
                          float *k_out, float *v_out, rz_stream stream)
{
    const char *fn = "rz_qk_norm_rope";
    record_error(RZ_OK, "");
    if (!q || !k || !positions || !q_out) return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (kv && (!v || !slots)) return fail(RZ_ERR_INVALID_ARG, "%s: a cache needs v and slots", fn);
    if (!kv && (v_out || !k_out)) return fail(RZ_ERR_INVALID_ARG, "%s: without a cache, k_out and no v_out", fn);
    const void *words[] = {q, k, v, q_gamma, k_gamma, positions, q_out, k_out, v_out};
    for (const void *p : words)
        if (!aligned(p, 4)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 4-byte aligned", fn);
    if (!aligned(slots, 8)) return fail(RZ_ERR_ALIGN, "%s: slots must be 8-byte aligned", fn);
    if (n_rows < 1 || n_rows > kMaxInt) return fail(RZ_ERR_INVALID_ARG, "%s: n_rows=%lld", fn, (long long)n_rows);
    RZ_TRY(check_head_dim(fn, head_dim));
    if (n_heads < 1 || n_kv_heads < 1 || n_kv_heads > 1024 || n_heads > kMaxHeads)
        return fail(RZ_ERR_SHAPE, "%s: n_heads=%d n_kv_heads=%d", fn, n_heads, n_kv_heads);
    if (rope_mode != 0 && rope_mode != 1) return fail(RZ_ERR_INVALID_ARG, "%s: rope_mode", fn);
    if (!(rope_theta > 0.0f) || std::isinf(rope_theta)) return fail(RZ_ERR_INVALID_ARG, "%s: rope_theta", fn);
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(RZ_ERR_INVALID_ARG, "%s: eps", fn);
    const int64_t q_dim = (int64_t)n_heads * head_dim, kv_dim = (int64_t)n_kv_heads * head_dim;
    if (ld_q < q_dim || ld_qo < q_dim || ld_k < kv_dim || (v && ld_v < kv_dim))
        return fail(RZ_ERR_SHAPE, "%s: a row stride is smaller than its row", fn);
    if (q_out == q && ld_qo != ld_q && n_rows > 1)
        return fail(RZ_ERR_SHAPE, "%s: q_out is q, but ld_qo=%lld is not ld_q=%lld", fn, (long long)ld_qo, (long long)ld_q);
    PagedKv pk{};
    if (kv) {
        RZ_TRY(check_kv_q4(fn, kv, &pk));
        if (pk.n_kv_heads != n_kv_heads || pk.head_dim != head_dim)
            return fail(RZ_ERR_SHAPE, "%s: the cache holds %d heads of %d", fn, pk.n_kv_heads, pk.head_dim);
    }
    RZ_TRY(ensure_device());
    HeadsArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.q_gamma = q_gamma;
    a.k_gamma = k_gamma;
    a.positions = positions;
    a.slots = slots;
    a.kv = pk;
    a.q_out = q_out;
    a.k_out = k_out;
    a.v_out = v_out;
    a.ld_qo = ld_qo;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.rope_mode = rope_mode;
    a.eps = eps;
    a.err = dev_error_word();
    return launched(fn, launch_qk_norm_rope(a, n_rows, head_dim, rope_theta, static_cast<cudaStream_t>(stream)));
}

size_t rz_attention_paged_q4_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim)
{
    const char *fn = "rz_attention_paged_q4_workspace_bytes";
    record_error(RZ_OK, "");
    if (check_head_dim(fn, head_dim) != RZ_OK) return 0;
    if (n_heads < 1 || n_heads > kMaxHeads || n_kv_heads < 1 || n_kv_heads > 1024 || n_heads % n_kv_heads) {
        fail(RZ_ERR_SHAPE, "%s: n_heads=%d n_kv_heads=%d", fn, n_heads, n_kv_heads);
        return 0;
    }
    if (ensure_device() != RZ_OK) return 0;
    return paged_attention_workspace_bytes(head_dim);
}

rz_status rz_attention_paged_q4(const float *q, int64_t ld_q, int64_t n_rows, const rz_kv_q4 *kv,
                                const int32_t *block_table, int64_t ld_table, int32_t max_blocks,
                                const int32_t *cu_rows, const int32_t *kv_len, int32_t n_seqs, int32_t n_heads,
                                float scale, float *att, void *att_q8, void *workspace, size_t ws_bytes, rz_stream stream)
{
    const char *fn = "rz_attention_paged_q4";
    record_error(RZ_OK, "");
    if (!q || !block_table || !cu_rows || !kv_len || (!att && !att_q8))
        return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    PagedKv pk{};
    RZ_TRY(check_kv_q4(fn, kv, &pk));
    RZ_TRY(check_blocks(fn, max_blocks, ld_table, kv->page_size));
    if (n_seqs < 1 || n_seqs > kPagedMaxSeqs) return fail(RZ_ERR_SHAPE, "%s: n_seqs=%d outside [1, %d]", fn, n_seqs, kPagedMaxSeqs);
    if (n_heads < 1 || n_heads > kMaxHeads || n_heads % pk.n_kv_heads)
        return fail(RZ_ERR_SHAPE, "%s: n_heads=%d with n_kv_heads=%d", fn, n_heads, pk.n_kv_heads);
    if (n_rows < 1) return fail(RZ_ERR_INVALID_ARG, "%s: n_rows=%lld", fn, (long long)n_rows);
    if (n_rows > kMaxInt || n_rows * (n_heads / pk.n_kv_heads) > kMaxTokens)
        return fail(RZ_ERR_SHAPE, "%s: n_rows=%lld with %d heads for each kv head", fn, (long long)n_rows, n_heads / pk.n_kv_heads);
    const int64_t q_dim = (int64_t)n_heads * pk.head_dim;
    if (ld_q < q_dim || ld_q % 4) return fail(RZ_ERR_SHAPE, "%s: ld_q=%lld (at least %lld, a multiple of 4)", fn, (long long)ld_q, (long long)q_dim);
    if (!(scale >= 0.0f) || std::isinf(scale)) return fail(RZ_ERR_INVALID_ARG, "%s: scale", fn);
    if (!aligned(q, 16) || !aligned(att, 16) || !aligned(att_q8, 16))
        return fail(RZ_ERR_ALIGN, "%s: q and the outputs must be 16-byte aligned", fn);
    const void *words[] = {block_table, cu_rows, kv_len};
    for (const void *p : words)
        if (!aligned(p, 4)) return fail(RZ_ERR_ALIGN, "%s: int32 buffers must be 4-byte aligned", fn);
    if (!workspace) return fail(RZ_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (!aligned(workspace, 16)) return fail(RZ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    RZ_TRY(ensure_device());
    const size_t need = paged_attention_workspace_bytes(pk.head_dim);
    if (ws_bytes < need) return fail(RZ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    PagedAttnArgs a{};
    a.q = q;
    a.ld_q = ld_q;
    a.n_rows = n_rows;
    a.kv = pk;
    a.table = block_table;
    a.table_ld = ld_table;
    a.max_blocks = max_blocks;
    a.cu_rows = cu_rows;
    a.kv_len = kv_len;
    a.n_seqs = n_seqs;
    a.n_heads = n_heads;
    a.scale = scale > 0.0f ? scale : 1.0f / std::sqrt((float)pk.head_dim);
    a.att = att;
    a.att_q8 = att_q8;
    a.err = dev_error_word();
    return launched(fn, launch_paged_attention(a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t rz_decode_layer_paged_workspace_bytes(const rz_layer_weights *w, int64_t m)
{
    record_error(RZ_OK, "");
    LayerDesc L;
    if (check_layer_weights(w, "rz_decode_layer_paged_workspace_bytes", m, &L) != RZ_OK) return 0;
    return layer_paged_workspace_bytes(L, m);
}

rz_status rz_decode_layer_paged(const float *input, const rz_layer_weights *w, const float *q_gamma, const float *k_gamma,
                                const rz_kv_q4 *kv, const int32_t *positions, const int64_t *slots,
                                const int32_t *block_table, int64_t ld_table, int32_t max_blocks, const int32_t *cu_rows,
                                const int32_t *kv_len, int32_t n_seqs, int64_t m, float *output, void *workspace,
                                size_t ws_bytes, rz_stream stream)
{
    const char *fn = "rz_decode_layer_paged";
    record_error(RZ_OK, "");
    if (!input || !output || !positions || !slots || !block_table || !cu_rows || !kv_len)
        return fail(RZ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(input, 16) || !aligned(output, 16)) return fail(RZ_ERR_ALIGN, "%s: input/output alignment", fn);
    const void *words[] = {q_gamma, k_gamma, positions, block_table, cu_rows, kv_len};
    for (const void *p : words)
        if (!aligned(p, 4)) return fail(RZ_ERR_ALIGN, "%s: buffers must be 4-byte aligned", fn);
    if (!aligned(slots, 8)) return fail(RZ_ERR_ALIGN, "%s: slots must be 8-byte aligned", fn);
    if (n_seqs < 1 || n_seqs > kPagedMaxSeqs) return fail(RZ_ERR_SHAPE, "%s: n_seqs=%d outside [1, %d]", fn, n_seqs, kPagedMaxSeqs);
    PagedKv pk{};
    RZ_TRY(check_kv_q4(fn, kv, &pk));
    RZ_TRY(check_blocks(fn, max_blocks, ld_table, kv->page_size));
    if (w && (pk.n_kv_heads != w->n_kv_heads || pk.head_dim != w->head_dim))
        return fail(RZ_ERR_SHAPE, "%s: the cache holds %d heads of %d", fn, pk.n_kv_heads, pk.head_dim);
    LayerDesc L;
    RZ_TRY(check_layer_weights(w, fn, m, &L));
    if (!workspace) return fail(RZ_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (!aligned(workspace, 16)) return fail(RZ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    const size_t need = layer_paged_workspace_bytes(L, m);
    if (ws_bytes < need) return fail(RZ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    HeadsArgs h{};
    h.q_gamma = q_gamma;
    h.k_gamma = k_gamma;
    h.positions = positions;
    h.slots = slots;
    h.kv = pk;
    h.err = dev_error_word();
    PagedAttnArgs a{};
    a.kv = pk;
    a.table = block_table;
    a.table_ld = ld_table;
    a.max_blocks = max_blocks;
    a.cu_rows = cu_rows;
    a.kv_len = kv_len;
    a.n_seqs = n_seqs;
    a.scale = 1.0f / std::sqrt((float)pk.head_dim);
    a.err = h.err;
    return launched(fn, launch_decode_layer_paged(input, L, h, a, m, output, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
