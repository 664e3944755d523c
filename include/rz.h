/*
 * rz.h -- C ABI of librz, the GB300 (sm_103a) Q4_K x Q8_1 single-token decode path.
 *
 * The operations follow the dp4a decode layer of realizar 0.8.5
 * src/cuda/executor/cached.rs (transformer_layer_gpu_true_dp4a), the Q4_0 model
 * forward of realizar 0.8.4 src/gpu/adapters/using.rs (GpuModelQ4::forward,
 * q4_0_gemv_into, rms_norm_inplace), the GPU-resident stack of realizar 0.8.5
 * src/cuda/executor/layers/forward_utils.rs (forward_all_layers_gpu_to_logits)
 * and the single-token semantics of realizar 0.8.4
 * src/gguf/cuda/clone_layer_weights.rs (forward_single_full_cuda_with_cache).
 *
 * Conventions for every entry point
 *   - Pointers named w, x, y, q8, gamma, out, input, output, workspace, k, v are
 *     DEVICE pointers owned by the caller.  librz never allocates device memory,
 *     never synchronises the stream and never copies between host and device
 *     (except rz_check_device_error, which reads one word back).
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default stream)
 *     and returns immediately.  Launches are stream-ordered and can be captured
 *     into a CUDA graph.
 *   - Every shape, alignment and range check runs on the host before anything is
 *     launched.  A failed check returns a non-zero rz_status, launches nothing and
 *     sets a message readable with rz_last_error() (thread-local).
 *   - Weights must be 16-byte aligned; f32 and Q8_1 buffers 16-byte aligned.
 *   - Device-side conditions that the host cannot see (a position read from device
 *     memory outside the cache, a bounded wait that ran out) never trap: the kernel
 *     records a code in a device error word and skips the access; the host reads
 *     and clears it with rz_check_device_error().
 *
 * Data formats (GGML convention for the weights; the pages name the types but do
 * not print their layouts):
 *   Q4_K  super-block of 256 weights in 144 bytes: f16 d | f16 dmin | 12 bytes of
 *         eight 6-bit scales and eight 6-bit mins | 128 bytes of 4-bit quants.
 *         weight = d * sc_j * q - dmin * m_j for sub-block j = e / 32; weight e is
 *         nibble (e % 64 < 32 ? low : high) of qs[32 * (e / 64) + e % 32].
 *         A matrix [out_dim][in_dim] is row-major: out_dim rows of in_dim / 256
 *         consecutive super-blocks.
 *   Q4_0  block of 32 weights in 18 bytes: f16 d | 16 bytes of 4-bit quants;
 *         weight i = d * (q_i - 8), q_i the low nibble of byte i (i < 16) or the
 *         high nibble of byte i - 16.  Row-major like Q4_K.
 *   Q8_1  activations quantised in blocks of 32: d = max|x| / 127 (f32 division),
 *         q = round-half-away(x / d) clamped to [-127, 127] (0 when d == 0),
 *         s = d * sum(q).  A buffer for m rows of n values (n % 32 == 0) holds
 *         int8 q[m][n], then f32 d[m][n/32], then f32 s[m][n/32]:
 *         RZ_Q8_1_BYTES(m, n) bytes.  (d and s are f32 so that s stays finite for
 *         block maxima beyond fp16 range / 32.)
 */
#ifndef RZ_H
#define RZ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    RZ_OK = 0,
    RZ_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, bad enum */
    RZ_ERR_SHAPE = 2,       /* dimension not a multiple of the block size, m > RZ_MAX_BATCH, ... */
    RZ_ERR_ALIGN = 3,       /* pointer not 16-byte aligned */
    RZ_ERR_CUDA = 4,        /* a CUDA runtime call failed (message has the CUDA error) */
    RZ_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out (rz_check_device_error) */
    RZ_ERR_UNSUPPORTED = 6, /* no sm_103a device, or a configuration this build does not handle */
    RZ_ERR_DEVICE = 7       /* a device-side range check failed (rz_check_device_error) */
} rz_status;

typedef void *rz_stream; /* cudaStream_t */

#define RZ_Q4K_BLOCK_BYTES 144
#define RZ_Q4K_BLOCK_WEIGHTS 256
#define RZ_Q4_0_BLOCK_BYTES 18
#define RZ_Q4_0_BLOCK_WEIGHTS 32
#define RZ_Q8_1_BLOCK 32
#define RZ_Q8_1_BYTES(m, n) ((m) * (n) + 8 * (m) * ((n) / 32))
#define RZ_MAX_BATCH 16

/* Message of the last failed call on this thread ("" if none). */
const char *rz_last_error(void);
/* Library version string. */
const char *rz_version(void);

/*
 * rz_q8_1_quantize -- Q8_1 quantisation of activations (q8_quantize_async in
 * transformer_layer_gpu_true_dp4a, steps 2 and 5).
 *   x    f32 [m][n], row-major.            q8  RZ_Q8_1_BYTES(m, n) bytes (output).
 *   1 <= m, n % 32 == 0.  Bit-exact with the format definition above.
 */
rz_status rz_q8_1_quantize(const float *x, void *q8, int64_t m, int64_t n, rz_stream stream);

/*
 * rz_q4k_q8_gemv -- y = W x for Q4_K weights and Q8_1 activations, the integer
 * GEMV behind every Q/K/V/O and FFN projection (q4k_q8_gemv_async in
 * transformer_layer_gpu_true_dp4a, steps 3 and 6).
 *   For token t < m and row r:
 *     y[t][r] = sum_b d_b * sum_j sc_bj * d8_tbj * I_tbrj - dmin_b * sum_j m_bj * s_tbj
 *   with I the exact int32 dot of the 32 codes of sub-block j.
 *   w   Q4_K [out_dim][in_dim]     q8  Q8_1 of m rows of in_dim     y  f32 [m][out_dim]
 *   1 <= m <= RZ_MAX_BATCH, in_dim % 256 == 0, out_dim >= 1.  Weights are read once
 *   for all m tokens.  f32 combination order differs from a sequential sum
 *   (deterministic run to run).
 */
rz_status rz_q4k_q8_gemv(const void *w, const void *q8, float *y, int64_t m, int64_t out_dim,
                         int64_t in_dim, rz_stream stream);

/*
 * rz_q4k_q8_subblock_dots -- the integer sub-block dots alone, for exact checks:
 *   I[r][k] = sum_{i<32} q4[r][32k + i] * q8[32k + i]   (one activation row)
 *   I  int32 [out_dim][in_dim/32] (output).  in_dim % 256 == 0.
 */
rz_status rz_q4k_q8_subblock_dots(const void *w, const void *q8, int32_t *I, int64_t out_dim,
                                  int64_t in_dim, rz_stream stream);

/*
 * rz_q4k_q8_gemv_ex -- the same GEMV with an epilogue:
 *     y[t][r] = (W x_t)_r + bias[r]           (bias != NULL; the QKV and head biases
 *                                              of preload_qkv_bias in cached.rs)
 *     y[t][r] = (W x_t)_r + residual[t][r]    (residual != NULL; steps 6-7 and 9-10 of
 *                                              transformer_layer_gpu_true_dp4a)
 *     y[t][r] = (W x_t)_r                     (both NULL)
 *   bias f32 [out_dim] (4-byte aligned); residual, y f32 [m][ld] with row stride ld
 *   (0 = out_dim; ld >= out_dim); y may alias residual.  A bias and a residual in
 *   one call: RZ_ERR_UNSUPPORTED.  Other arguments and checks as rz_q4k_q8_gemv.
 */
rz_status rz_q4k_q8_gemv_ex(const void *w, const void *q8, const float *bias, const float *residual, float *y,
                            int64_t ld, int64_t m, int64_t out_dim, int64_t in_dim, rz_stream stream);

/*
 * rz_q4k_q8_gemm -- the same product for many tokens at once (a prompt's prefill:
 * GpuModelQ4::forward of realizar 0.8.4 src/gpu/adapters/using.rs takes a sequence
 * of token ids), on the tensor cores (tcgen05.mma):
 *     y[t][r] = sum_b d_b * sum_j sc_bj * d8_tbj * I_tbrj - dmin_b * sum_j m_bj * s_tbj
 *   for every token t < m, with the integer sub-block dots I exact, as
 *   rz_q4k_q8_gemv.  Each 128 x 128 tile of (tokens, rows) reads its weights once.
 *   w          Q4_K [out_dim][in_dim]         q8  Q8_1 of m rows of in_dim
 *   y          f32 [m][ldy] (ldy 0 = out_dim; ldy >= out_dim), 4-byte aligned
 *   workspace  device scratch of at least rz_q4k_q8_gemm_workspace_bytes(m, in_dim)
 *              bytes, 16-byte aligned (the activations re-laid out as tensor-core
 *              operands); contents need no initialisation and are not kept.
 *   1 <= m (any; tokens beyond a multiple of 128 are padding inside the kernel),
 *   in_dim % 256 == 0, out_dim >= 1.  Two launches.  f32 combination order
 *   differs from rz_q4k_q8_gemv's (deterministic run to run).  A bounded wait that
 *   runs out records RZ_ERR_TIMEOUT for rz_check_device_error.
 */
size_t rz_q4k_q8_gemm_workspace_bytes(int64_t m, int64_t in_dim);
rz_status rz_q4k_q8_gemm(const void *w, const void *q8, float *y, int64_t ldy, int64_t m, int64_t out_dim,
                         int64_t in_dim, void *workspace, size_t ws_bytes, rz_stream stream);

/*
 * rz_rmsnorm_q4k_gemv -- steps 1-3 of transformer_layer_gpu_true_dp4a in one
 * launch: RMSNorm of x over its first n values with gamma (zero padding after n),
 * Q8_1 quantisation of the normed row (bit-identical to rz_rmsnorm's q8 output),
 * then up to three Q4_K GEMVs against that one Q8_1 activation, their outputs
 * side by side in y (the Q | K | V projections):
 *     y[t][off_k + r] = (W_k q8(norm(x_t)))_r (+ bias[k][r]),  off_k = rows[0] + ... + rows[k-1]
 *   x      f32 [m][ldx], in_dim values per row are read (ldx >= in_dim)
 *   gamma  f32 [n]; n <= in_dim; in_dim % 256 == 0
 *   w      host array of n_mats (1..3) device pointers to Q4_K [rows[k]][in_dim]
 *   bias   host array of n_mats device pointers (each may be NULL), or NULL
 *   y      f32 [m][ldy], ldy >= rows[0] + ... + rows[n_mats-1]
 *   x, gamma, y 16-byte aligned, ldx and ldy multiples of 4.  Every CTA normalises and
 *   quantises the whole row (m * in_dim * 1.25 B of shared memory must fit, else
 *   RZ_ERR_UNSUPPORTED).
 */
rz_status rz_rmsnorm_q4k_gemv(const float *x, int64_t ldx, const float *gamma, int64_t n, float eps, int32_t n_mats,
                              const void *const *w, const int64_t *rows, const float *const *bias, float *y,
                              int64_t ldy, int64_t m, int64_t in_dim, rz_stream stream);

/*
 * rz_q4k_q8_gemv_multi -- up to three Q4_K GEMVs against one Q8_1 activation in one
 * launch (the Q | K | V projections of transformer_layer_gpu_true_dp4a, realizar
 * 0.8.5 src/cuda/executor/cached.rs, with the activation quantised beforehand, as
 * a layer does from four tokens on):
 *     y[t][off_k + r] = (W_k q8_t)_r (+ bias[k][r]),  off_k = rows[0] + ... + rows[k-1]
 *   q8     Q8_1 of m rows of in_dim values (the layout of rz_q8_1_quantize), 16-byte aligned
 *   w      host array of n_mats (1..3) device pointers to Q4_K [rows[k]][in_dim], 16-byte aligned
 *   bias   host array of n_mats device pointers (each may be NULL), or NULL
 *   y      f32 [m][ldy], ldy >= rows[0] + ... + rows[n_mats-1], 4-byte aligned
 *   1 <= m <= RZ_MAX_BATCH, in_dim % 256 == 0.  The same results as one
 *   rz_q4k_q8_gemv_ex per matrix.
 */
rz_status rz_q4k_q8_gemv_multi(const void *q8, int32_t n_mats, const void *const *w, const int64_t *rows,
                               const float *const *bias, float *y, int64_t ldy, int64_t m, int64_t in_dim,
                               rz_stream stream);

/*
 * rz_q4k_f32_gemv -- y = W x (+ bias) for Q4_K weights and f32 activations, with no
 * Q8_1 quantisation of x (q4k_gemv_cached_async in transformer_layer_gpu_cached,
 * realizar 0.8.5 src/cuda/executor/cached.rs):
 *     y[t][r] = sum_e (d * sc_j * q_e - dmin * m_j) x[t][e]   (+ bias[r])
 *   w Q4_K [out_dim][in_dim]   x f32 [m][in_dim]   y f32 [m][out_dim]   bias f32 [out_dim] or NULL
 *   1 <= m <= RZ_MAX_BATCH, in_dim % 256 == 0; w and x 16-byte aligned, y and bias
 *   4-byte aligned.  f32 products and sums (order differs from a sequential sum;
 *   deterministic run to run).
 */
rz_status rz_q4k_f32_gemv(const void *w, const float *x, const float *bias, float *y, int64_t m, int64_t out_dim,
                          int64_t in_dim, rz_stream stream);

/*
 * rz_q4_0_gemv -- y = W x for Q4_0 weights and f32 activations (the LM head of
 * GpuModelQ4::forward, q4_0_gemv_into; step 5 of that function).
 *   w  Q4_0 [out_dim][in_dim]   x  f32 [m][in_dim]   y  f32 [m][out_dim]
 *   in_dim % 32 == 0, 1 <= m <= RZ_MAX_BATCH.  Only w needs 16-byte alignment of
 *   its base; rows of 18-byte blocks may start anywhere.  When in_dim % 256 == 0
 *   and x is 16-byte aligned the products run on the tensor cores with x split
 *   into two f16 pieces (x to about 2^-22 relative; |x| must stay below 65504);
 *   otherwise in f32 FMAs.  f32 accumulation either way (order differs from a
 *   sequential sum; deterministic run to run).
 */
rz_status rz_q4_0_gemv(const void *w, const float *x, float *y, int64_t m, int64_t out_dim,
                       int64_t in_dim, rz_stream stream);

/*
 * rz_q4_0_gemv_bias -- rz_q4_0_gemv plus a bias added to every token's output:
 * y[t][r] = (W x_t)_r + bias[r] (the LM-head bias of preload_lm_head_bias,
 * realizar 0.8.5 src/cuda/executor/cached.rs).  bias f32 [out_dim], 4-byte
 * aligned; other arguments as rz_q4_0_gemv.
 */
rz_status rz_q4_0_gemv_bias(const void *w, const float *x, const float *bias, float *y, int64_t m, int64_t out_dim,
                            int64_t in_dim, rz_stream stream);

/*
 * rz_rmsnorm -- RMSNorm with optional fused Q8_1 quantisation (rms_norm_inplace in
 * using.rs; rmsnorm_gpu + q8_quantize_async in transformer_layer_gpu_true_dp4a):
 *   rms = sqrt(sum_{i<n} x_i^2 / n + eps);  y_i = x_i / rms * gamma_i (i < n),
 *   y_i = 0 for n <= i < n_pad (the zero padding of pad_and_upload_input).
 *   x      f32 [m][n_pad] (only the first n of each row are read)
 *   gamma  f32 [n]
 *   y      f32 [m][n_pad] output, or NULL
 *   q8     Q8_1 of m rows of n_pad (output), or NULL.  When given, it is exactly
 *          the Q8_1 quantisation of the f32 y this call computes.
 *   At least one of y, q8 non-NULL.  n >= 1, n_pad >= n, n_pad % 32 == 0 when q8.
 */
rz_status rz_rmsnorm(const float *x, const float *gamma, float *y, void *q8, int64_t m, int64_t n,
                     int64_t n_pad, float eps, rz_stream stream);

/*
 * rz_residual_add -- out = a + b elementwise in f32 (residual_add_gpu, steps 7 and
 * 10 of transformer_layer_gpu_true_dp4a).  out may alias a or b.  Bit-exact.
 */
rz_status rz_residual_add(const float *a, const float *b, float *out, int64_t n, rz_stream stream);

/*
 * ---------------------------------------------------------------------------
 * Layer-level entry points.  They launch several kernels in stream order and
 * use a caller-provided device workspace (size from the *_workspace_bytes
 * function, base 16-byte aligned).  The workspace holds intermediates only; the
 * attention counters inside it must be zero before the first call (fill the
 * workspace with zeros once after allocating it); every completed call leaves
 * them zero again.  Calls that share a workspace must not overlap on the GPU.
 * ---------------------------------------------------------------------------
 */

/* One Q4_K decode layer (the weights of transformer_layer_gpu_true_dp4a).
 * Matrices (Q4_K, row-major [out][in]):
 *   wq [n_heads*head_dim][hidden_pad]   wk, wv [n_kv_heads*head_dim][hidden_pad]
 *   wo [hidden][q_pad]                  q_pad = n_heads*head_dim rounded up to 256
 *   wgate, wup [inter][hidden_pad]      wdown [hidden][inter]
 * attn_gamma, ffn_gamma: f32 [hidden].  hidden_pad % 256 == 0 (the zero padding of
 * pad_and_upload_input), inter % 256 == 0, head_dim % 32 == 0 and <= 256,
 * n_heads % n_kv_heads == 0 with at most 16 query heads per kv head.
 * rope_mode 0 rotates adjacent pairs (2i, 2i+1), 1 rotates (i, i + head_dim/2);
 * the angle of pair i at position p is p * rope_theta^(-2i/head_dim).
 * Fused Q|K|V layout (OwnedQKVWeights::Fused of realizar 0.8.4
 * clone_layer_weights.rs): wk = wv = NULL and wq holds the one matrix
 * [n_heads*head_dim + 2*n_kv_heads*head_dim][hidden_pad] (Q rows, then K, then V).
 * Biases (the Qwen2 QKV bias of preload_qkv_bias in realizar 0.8.5 cached.rs):
 * bq [n_heads*head_dim], bk, bv [n_kv_heads*head_dim] f32, each NULL for none,
 * added to the projections before RoPE; with the fused layout bq holds the fused
 * bias [q_dim + 2*kv_dim] and bk, bv must be NULL.  Biases need 4-byte alignment. */
typedef struct {
    const void *wq, *wk, *wv, *wo, *wgate, *wup, *wdown;
    const float *attn_gamma, *ffn_gamma;
    int32_t hidden, hidden_pad, n_heads, n_kv_heads, head_dim, inter;
    float eps, rope_theta;
    int32_t rope_mode;
    const float *bq, *bk, *bv;
} rz_layer_weights;

/* f32 KV cache of one layer.  Row p of sequence t (token t of a batch) is at
 * k + t*seq_stride + p*kv_dim (same for v), kv_dim = n_kv_heads*head_dim.
 * seq_stride is ignored when m == 1; otherwise >= max_seq*kv_dim and a multiple of 4
 * (every sequence starts 16-byte aligned).  1 <= max_seq <= 4096. */
typedef struct {
    float *k, *v;
    int64_t seq_stride;
    int32_t max_seq;
} rz_kv_cache;

/*
 * rz_swiglu_ffn -- out = x + W_down q8( silu(W_gate q8(n)) * (W_up q8(n)) ),
 * n = RMSNorm(x; gamma) (steps 8-10 of transformer_layer_gpu_true_dp4a;
 * fused_ffn_swiglu_gpu_true_dp4a; SiLU of the gate times up as in cuda_swiglu_ffn
 * of clone_layer_weights.rs).  x, out f32 [m][hidden_pad] (out may alias x;
 * out[.][hidden..hidden_pad) is written as 0).
 */
size_t rz_swiglu_ffn_workspace_bytes(int64_t m, int64_t hidden_pad, int64_t inter);
rz_status rz_swiglu_ffn(const float *x, const float *gamma, const void *w_gate, const void *w_up,
                        const void *w_down, float *out, int64_t m, int64_t hidden,
                        int64_t hidden_pad, int64_t inter, float eps, void *workspace,
                        size_t ws_bytes, rz_stream stream);

/*
 * rz_attention_decode -- RoPE on q and k at each token's position, append k and v
 * to the cache row `position`, then softmax(q k^T / sqrt(head_dim)) v over cache
 * rows 0..position with the GQA map kv_head = q_head / (n_heads / n_kv_heads)
 * (incremental_attention_async, step 4; first-token and GQA semantics of
 * forward_single_full_cuda_with_cache).
 *   q, k, v   f32 projections, token t at q + t*ld_qkv (same ld for k, v);
 *             q [n_heads*head_dim], k, v [n_kv_heads*head_dim] per token.
 *   positions device int32 [m] (each checked in the kernel against max_seq; a bad
 *             one records RZ_ERR_DEVICE, skips its cache write and yields zeros),
 *             or NULL to use `position` for every token (checked on the host).
 *   att       f32 [m][n_heads*head_dim] output, or NULL.
 *   att_q8    Q8_1 of m rows of q_pad (output, the O projection's input), or NULL.
 */
size_t rz_attention_workspace_bytes(int64_t m, int32_t n_heads, int32_t n_kv_heads,
                                    int32_t head_dim, int32_t max_seq);
rz_status rz_attention_decode(const float *q, const float *k, const float *v, int64_t ld_qkv,
                              const rz_kv_cache *kv, const int32_t *positions, int32_t position,
                              int64_t m, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                              float rope_theta, int32_t rope_mode, float *att, void *att_q8,
                              void *workspace, size_t ws_bytes, rz_stream stream);

/*
 * rz_decode_layer -- one decode step of one layer for m tokens (m sequences),
 * the step order of transformer_layer_gpu_true_dp4a.
 *   input, output f32 [m][hidden_pad] (zero padding kept; output may alias input)
 *   kv            this layer's cache, written at each token's position
 *   positions     device int32 [m] or NULL for the host `position`
 */
size_t rz_decode_layer_workspace_bytes(const rz_layer_weights *w, int64_t m, int32_t max_seq);
rz_status rz_decode_layer(const float *input, const rz_layer_weights *w, const rz_kv_cache *kv,
                          const int32_t *positions, int32_t position, int64_t m, float *output,
                          void *workspace, size_t ws_bytes, rz_stream stream);

/*
 * rz_decode_stack -- n_layers decode layers, then the output RMSNorm and the Q4_0
 * LM head (forward_all_layers_gpu_to_logits; GpuModelQ4::forward steps 4-5).
 *   layers, kvs   host arrays of n_layers descriptors (same hidden, hidden_pad,
 *                 eps and kv max_seq for every layer)
 *   out_gamma     f32 [hidden];  lm_head Q4_0 [vocab][hidden]
 *   lm_bias       f32 [vocab] added to the logits (preload_lm_head_bias in realizar
 *                 0.8.5 cached.rs), or NULL
 *   hidden_out    f32 [m][hidden_pad] final hidden state, or NULL
 *   logits        f32 [m][vocab]
 */
size_t rz_decode_stack_workspace_bytes(const rz_layer_weights *layers, int32_t n_layers, int64_t m,
                                       int32_t max_seq);
rz_status rz_decode_stack(const float *input, const rz_layer_weights *layers, const rz_kv_cache *kvs,
                          int32_t n_layers, const int32_t *positions, int32_t position, int64_t m,
                          const float *out_gamma, const void *lm_head, const float *lm_bias, int64_t vocab,
                          float *hidden_out, float *logits, void *workspace, size_t ws_bytes,
                          rz_stream stream);

/*
 * rz_decode_layers -- the n_layers decode layers of rz_decode_stack without the
 * output RMSNorm and the LM head (a pipeline stage, or a caller with its own
 * head).  output: f32 [m][hidden_pad], the final hidden state (padding zero).
 * Other arguments, checks and the workspace (rz_decode_stack_workspace_bytes)
 * as for rz_decode_stack.
 */
rz_status rz_decode_layers(const float *input, const rz_layer_weights *layers, const rz_kv_cache *kvs,
                           int32_t n_layers, const int32_t *positions, int32_t position, int64_t m, float *output,
                           void *workspace, size_t ws_bytes, rz_stream stream);

/*
 * The Q4_0 whole-model layer (GpuModelQ4::forward_layer of realizar 0.8.4
 * src/gpu/adapters/using.rs): every projection Q4_0 against f32 activations.
 *   wqkv   Q4_0 [n_heads*head_dim + 2*n_kv_heads*head_dim][hidden] (Q rows, then K, then V)
 *   wo     Q4_0 [hidden][n_heads*head_dim]
 *   wgate  Q4_0 [inter][hidden], or NULL for the GELU FFN
 *   wup    Q4_0 [inter][hidden]      wdown  Q4_0 [hidden][inter]
 *   attn_gamma, ffn_gamma f32 [hidden]
 * hidden and inter multiples of 32 (hidden <= 16384), head_dim a multiple of 32 in
 * [32, 256], rope as rz_layer_weights.
 * Step order: RMSNorm -> QKV GEMV -> RoPE q, k at the position, KV append,
 * attention over rows 0..position -> O GEMV -> + input -> RMSNorm -> FFN ->
 * + residual.  FFN: silu(gate) * up then down (ffn_swiglu_gpu) with a gate,
 * else GELU(up) then down (ffn_standard_gpu), GELU in its tanh form
 * 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))).  Intermediates are f32.
 */
typedef struct {
    const void *wqkv, *wo, *wgate, *wup, *wdown;
    const float *attn_gamma, *ffn_gamma;
    int32_t hidden, n_heads, n_kv_heads, head_dim, inter;
    float eps, rope_theta;
    int32_t rope_mode;
} rz_layer_weights_q4_0;

/*
 * rz_decode_layer_q4_0 -- one decode step of one Q4_0 layer for m tokens.
 *   input, output f32 [m][hidden] (output may alias input); kv, positions,
 *   position and the workspace (zero-filled once) as for rz_decode_layer.
 */
size_t rz_decode_layer_q4_0_workspace_bytes(const rz_layer_weights_q4_0 *w, int64_t m, int32_t max_seq);
rz_status rz_decode_layer_q4_0(const float *input, const rz_layer_weights_q4_0 *w, const rz_kv_cache *kv,
                               const int32_t *positions, int32_t position, int64_t m, float *output, void *workspace,
                               size_t ws_bytes, rz_stream stream);

/*
 * rz_decode_stack_launches -- the number of librz kernels one rz_decode_stack call
 * (with_head != 0, an LM head of `vocab` rows) or one rz_decode_layers call
 * (with_head == 0, vocab unused) launches for these layers, batch m and cache
 * length max_seq.  Memset nodes are not kernels and are not counted.
 * Returns 0 for arguments the calls would reject.
 */
int32_t rz_decode_stack_launches(const rz_layer_weights *layers, int32_t n_layers, int64_t m, int32_t max_seq,
                                 int32_t with_head, int64_t vocab);

/*
 * rz_swiglu_ffn_static -- the same computation as rz_swiglu_ffn, for callers that
 * cannot allocate device memory or pass a workspace (the paper has no
 * counterpart: this is a packaging variant of rz_swiglu_ffn).  Its intermediates
 * live in a fixed 512 KiB device array inside the library (every GPU that loads
 * the library holds one until the process exits); shapes whose scratch
 * (rz_swiglu_ffn_workspace_bytes) exceeds 512 KiB are rejected with
 * RZ_ERR_UNSUPPORTED.  It calls no allocator.  The first call on a device looks
 * up the array's device address (a runtime query), so make that first call before
 * any stream capture.  All calls share the array: calls that overlap on the GPU
 * race and must be ordered by the caller.  Arguments as for rz_swiglu_ffn.
 */
rz_status rz_swiglu_ffn_static(const float *x, const float *gamma, const void *w_gate, const void *w_up,
                               const void *w_down, float *out, int64_t m, int64_t hidden,
                               int64_t hidden_pad, int64_t inter, float eps, rz_stream stream);

/*
 * ---------------------------------------------------------------------------
 * The paged KV cache in 4 bits.  Three calls serve requests of ragged lengths, any
 * number of new tokens each (one token, drafted tokens, a prompt chunk):
 *   rz_paged_plan          once a step: pages, slots, positions and row offsets
 *   rz_qk_norm_rope        each layer: norm and rotate q and k, append k and v
 *   rz_attention_paged_q4  each layer: attention over the pages
 * The new tokens of all requests are packed into rows, request after request.  Lengths,
 * positions, slots and tables are read from device memory, so that one captured
 * graph serves every step.
 *
 * K and V are held as Q4_0 blocks of 32 values along the head: d = f16 of the value
 * of largest magnitude (of +a and -a the positive one) divided by -8, clamped to f16's
 * range; code = round-half-even(x / d) + 8 clamped to 0..15; value = d * (code - 8).
 * d == 0 gives codes 8; a block with a NaN or an infinity gets d = NaN (d is never an infinity).  Bytes are laid
 * out for the kernels (csrc/paged_q4.cuh), 16 tokens of one kv head in a record of
 * 18 * head_dim bytes.
 * ---------------------------------------------------------------------------
 */

/* The cache of one layer: pages holds n_pages * rz_kv_q4_page_bytes(...) bytes, 16-byte
 * aligned; page_size 16, 32, 64 or 128 tokens; head_dim a multiple of 32 in [32, 256].
 * Slot = page * page_size + offset names one token's place.  A page needs no
 * initialisation: tokens beyond a request's length are never used. */
typedef struct {
    void *pages;
    int64_t n_pages;
    int32_t page_size, n_kv_heads, head_dim;
} rz_kv_q4;

/* Bytes of one page (0 for arguments outside their range). */
size_t rz_kv_q4_page_bytes(int32_t page_size, int32_t n_kv_heads, int32_t head_dim);

/*
 * rz_paged_plan -- page table, slot map, positions and row offsets of one step from the
 * requests' lengths, in one launch.
 *   cached  int32 [n_seqs] tokens that each request holds in its pages
 *   fresh   int32 [n_seqs] its new tokens of this step (0: none); negative: the request
 *           has ended, and its pages go back to the pool before any are handed out
 *   owned   int32 [n_seqs] pages each request has: block_table[i][0 .. owned[i])
 *   free_pages, free_count  the pool: a stack of n_pages entries, the first *free_count of
 *           them free.  Pages are taken from its top, in order of request and block.
 *   block_table int32 [n_seqs][ld_table], max_blocks entries of a row in use; the new
 *           pages are written behind the owned ones, nothing else is changed
 *   owned_out, free_count_out  the state after the step; each may be its input
 * Outputs:
 *   cu_rows   int32 [n_seqs + 1]  rows of request i: cu_rows[i] .. cu_rows[i + 1]
 *   kv_len    int32 [n_seqs]      cached + fresh; 0 for ended and refused requests (not
 *             the buffer of cached or fresh).  What rz_attention_paged_q4 takes.  The next step's cached
 *             it is for served requests only: a refused one still holds its cached tokens, so a caller that
 *             carries lengths on the device takes fresh < 0 ? 0 : kv_len > 0 ? kv_len : cached.
 *   row_seq, positions int32 [max_rows], slots int64 [max_rows]: the request, position and
 *             cache slot of each row; -1 in the rows behind the last and, but for
 *             row_seq, in those of a refused request
 * Requests are served in order: the first whose new pages the pool does not have is
 * refused, and so is every later one that needs a page; its rows stay in place, its state
 * as it was (RZ_ERR_DEVICE from rz_check_device_error, code 0x204).  Refused with
 * RZ_ERR_DEVICE too: negative lengths, owned outside [0, max_blocks], more tokens
 * cached than its pages hold or in all than max_blocks pages do, and a request whose rows end
 * beyond max_rows (it has none).  A page that an ended request returns beyond n_pages
 * is dropped.  A page below 0 that holds a new row records RZ_ERR_DEVICE (0x206), and the row's slot
 * is -1; one beyond the cache is reported by the calls that use it.
 * 1 <= n_seqs <= 1024, page_size as above, max_blocks * page_size <= 2^30.
 */
rz_status rz_paged_plan(const int32_t *cached, const int32_t *fresh, int32_t n_seqs, const int32_t *owned,
                        int32_t *owned_out, const int32_t *free_count, int32_t *free_count_out, int32_t *free_pages,
                        int64_t n_pages, int32_t *block_table, int64_t ld_table, int32_t max_blocks, int32_t page_size,
                        int64_t max_rows, int32_t *cu_rows, int32_t *kv_len, int32_t *row_seq, int32_t *positions,
                        int64_t *slots, rz_stream stream);

/*
 * rz_qk_norm_rope -- for each row: RMSNorm of every head of q and k (q_gamma, k_gamma f32
 * [head_dim], each NULL for none), rotation by the row's position (angles, theta and
 * rope_mode as rz_layer_weights), and the append of k and v to the cache at the row's slot.
 *   q, k, v    f32 rows of n_heads, n_kv_heads, n_kv_heads heads, row strides ld_*
 *              (parts of one fused Q|K|V output, say); 4-byte aligned; n_heads <= 65536, n_kv_heads <= 1024
 *   positions  int32 [n_rows]; a negative one marks a padding row, whose outputs and
 *              cache stay as they are
 *   slots      int64 [n_rows]; negative: the row is not appended.  A slot beyond the cache
 *              records RZ_ERR_DEVICE and is not written.  Slots of one call are distinct.
 *   kv         the cache, or NULL: q_out and k_out only (v, slots unused, v_out NULL)
 *   q_out      f32, row stride ld_qo; may be q (with ld_qo == ld_q)
 *   k_out, v_out f32 [n_rows][n_kv_heads * head_dim] or NULL: with a cache the values as
 *              it holds them, without one the rotated k
 * The cache's codes and scales are those of the format evaluated in f64 (the kernel
 * carries a key as a sum of two f32; a value may take either of two codes within 2^-40 of the border
 * between them, relative to its pair, or within position * 2^-52 from position 4096 on, the rounding of
 * the angle: 2^-35 at 131072).
 */
rz_status rz_qk_norm_rope(const float *q, int64_t ld_q, const float *k, int64_t ld_k, const float *v, int64_t ld_v,
                          const float *q_gamma, const float *k_gamma, float eps, const int32_t *positions,
                          const int64_t *slots, const rz_kv_q4 *kv, int64_t n_rows, int32_t n_heads, int32_t n_kv_heads,
                          int32_t head_dim, float rope_theta, int32_t rope_mode, float *q_out, int64_t ld_qo,
                          float *k_out, float *v_out, rz_stream stream);

/*
 * rz_attention_paged_q4 -- softmax(scale * q k^T) v of each request's new rows over its
 * pages: row r of request i (r = 0 .. m - 1, m = cu_rows[i + 1] - cu_rows[i]) sees its first
 * kv_len[i] - m + r + 1 tokens (the new ones are in the cache already); a row that sees
 * none comes out as zeros.  Query head h reads kv head h / (n_heads / n_kv_heads); n_heads <= 65536.
 *   q          f32 [n_rows] rows of n_heads * head_dim, stride ld_q (a multiple of 4),
 *              16-byte aligned, |q| < 1e35; rows behind cu_rows[n_seqs] are not read and their outputs not
 *              written
 *   block_table int32 [n_seqs][ld_table], max_blocks entries of a row in use; a page may
 *              stand in several rows (a shared prefix; rz_paged_plan itself gives each page to one request)
 *   scale      0 for 1 / sqrt(head_dim)
 *   att        f32 [n_rows][n_heads * head_dim], or NULL
 *   att_q8     Q8_1 of n_rows rows of q_pad (n_heads * head_dim rounded up to 256; the O
 *              projection's input), or NULL
 *              (the outputs and q may not overlap)
 *   workspace  rz_attention_paged_q4_workspace_bytes bytes, 16-byte aligned, zero-filled
 *              once after allocating it (a completed call leaves its counters zero; after
 *              RZ_ERR_TIMEOUT fill it with zeros again); calls that share it must not overlap on
 *              the GPU, captured ones among them
 * Scores and sums are f32-accurate: q and the weights enter as two f16 pieces each (22 bits), the
 * codes exactly.  A weight p |d| of V does not come closer than 2^-31 of the row's largest p |d|, taking for
 * |d| the largest of the blocks of the token and of up to 3 others near it: where the blocks of a head, or such
 * tokens, differ by more than some 2^9, the small ones have fewer bits than f32.
 * Requests of more than 40 query rows for a kv head, at a head_dim of 64 or 128, are worked 128 tokens at a time, K and V
 * as two f16 pieces each: a value comes to within 2^-30 of the largest |d| of the 128, which stands in the place
 * of the 4 tokens' above.  (Where n_rows - n_seqs + 1 rows would be 40 query rows or fewer, which is what one request
 * can have when every other has a row, they are worked as few rows are: a prompt among more idle requests than
 * there are rows takes about twice as long.)
 * A length, row offset or page outside its range records RZ_ERR_DEVICE:
 * a request of a length below 0 or beyond its table holds no token (zeros), one of bad row offsets has
 * no rows (its outputs stay as they were), and one of a bad page has rows that are undefined.  1 <= n_seqs <= 1024.
 */
size_t rz_attention_paged_q4_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);
rz_status rz_attention_paged_q4(const float *q, int64_t ld_q, int64_t n_rows, const rz_kv_q4 *kv,
                                const int32_t *block_table, int64_t ld_table, int32_t max_blocks,
                                const int32_t *cu_rows, const int32_t *kv_len, int32_t n_seqs, int32_t n_heads,
                                float scale, float *att, void *att_q8, void *workspace, size_t ws_bytes,
                                rz_stream stream);

/*
 * rz_decode_layer_paged -- rz_decode_layer over the paged 4-bit cache: the new tokens of
 * any requests, m rows in all (1 .. RZ_MAX_BATCH), through one layer: the RMSNorm and Q, K, V
 * projections, rz_qk_norm_rope, rz_attention_paged_q4, then the O projection and the FFN.
 *   input, output f32 [m][hidden_pad] (output may alias input)
 *   w             as rz_decode_layer; q_gamma, k_gamma f32 [head_dim] norms of the heads, or NULL
 *   kv            this layer's cache; positions, slots, block_table, cu_rows, kv_len: of one
 *                 rz_paged_plan, for every layer of the step.  Rows without a request (or of
 *                 a refused one) come out undefined.
 *   workspace     rz_decode_layer_paged_workspace_bytes bytes, 16-byte aligned, zero-filled
 *                 once after allocating it; calls that share it must not overlap on the GPU
 */
size_t rz_decode_layer_paged_workspace_bytes(const rz_layer_weights *w, int64_t m);
rz_status rz_decode_layer_paged(const float *input, const rz_layer_weights *w, const float *q_gamma, const float *k_gamma,
                                const rz_kv_q4 *kv, const int32_t *positions, const int64_t *slots,
                                const int32_t *block_table, int64_t ld_table, int32_t max_blocks, const int32_t *cu_rows,
                                const int32_t *kv_len, int32_t n_seqs, int64_t m, float *output, void *workspace,
                                size_t ws_bytes, rz_stream stream);

/*
 * ---------------------------------------------------------------------------
 * An FFN of experts (a mixture of experts) in Q4_K.  A layer calls, in this order:
 *   rz_residual_rmsnorm  the attention's output is added to the hidden state, the sum normed
 *   (the router's product, logits = W_router y, is the caller's: rz_q4_0_gemv, say)
 *   rz_moe_route         the experts of each token, their weights, the rows by expert
 *   rz_moe_swiglu        silu(gate) * up of each (token, choice) row with its expert
 *   rz_moe_down          the product back, the weighted sum of a token's rows, the residual
 * and rz_moe_ffn is the last three in one call.
 *
 * Row r of a plan is one (token, choice): the rows of expert e are offsets[e] .. offsets[e + 1], in
 * the order of their tokens.  All of a plan is in device memory, so that one captured graph serves every
 * step.  A plan may also come from elsewhere.  Offsets outside [0, n_tokens * top_k] or decreasing ones make an expert
 * have no rows.  What is not in the plan's bounds records RZ_ERR_DEVICE: a row outside [0, n_tokens * top_k] reads
 * row 0, a choice whose place is not among the rows of its expert is left out of the token's sum.  Offsets that
 * overlap give undefined values.  Calls that share a workspace or write one plan must not overlap on the GPU,
 * captured ones among them.
 * ---------------------------------------------------------------------------
 */
typedef struct {
    int32_t *experts; /* [n_tokens][top_k] the experts of a token, the largest logit first; -1: none */
    float *weights;   /* [n_tokens][top_k] */
    int32_t *offsets; /* [n_experts + 1] */
    int32_t *rows;    /* [n_tokens * top_k] token * top_k + choice of row r; -1 behind offsets[n_experts] */
    int32_t *places;  /* [n_tokens * top_k] the row of token * top_k + choice; -1: none */
    int64_t n_tokens; /* n_tokens * top_k <= 2^27 */
    int32_t n_experts, top_k; /* 1 <= top_k <= n_experts <= 512, top_k <= 32 */
} rz_moe_plan;

/*
 * rz_residual_rmsnorm -- rz_residual_add, rz_rmsnorm and its Q8_1 form in one pass, for any
 * number of rows:
 *   s = x + delta (f32);  y_i = s_i / sqrt(sum_{i<n} s_i^2 / n + eps) * gamma_i (i < n), 0 for n <= i < n_pad
 *   x, delta  f32 [m][n_pad] (the first n of each row are read); delta may be NULL: s = x
 *   gamma     f32 [n]
 *   sum       f32 [m][n_pad] output: s, 0 behind n; or NULL.  May be x or delta.
 *   y         f32 [m][n_pad] output, or NULL.  May be x or delta (not sum).
 *   q8        Q8_1 of m rows of n_pad, of the y as it is rounded; or NULL.  (One of y, q8 is given.)  Its scales are
 *             max|y| times the f32 nearest to 1/127, at most an ulp from rz_q8_1_quantize's quotient; codes
 *             and sums follow from them as there.  A block with a NaN has d = s = NaN (rz_q8_1_quantize leaves
 *             it out of the largest value), so that what is made of it is NaN too.
 *   n_pad a multiple of 32 up to 16384; all buffers 16-byte aligned.
 * y is the f32 nearest to the formula's value of s but for about one value in 2^20 (sums and products are
 * carried as sums of two f32), so that codes do not depend on the order of a sum.  Squares of s stay in f32's range.
 */
rz_status rz_residual_rmsnorm(const float *x, const float *delta, const float *gamma, float *sum, float *y, void *q8,
                              int64_t m, int64_t n, int64_t n_pad, float eps, rz_stream stream);

/*
 * rz_moe_route -- the top_k experts of each token by its logits, their weights, and the rows
 * grouped by expert, into the buffers of `plan`.
 *   logits    f32 [n_tokens] rows of n_experts, row stride ld, 4-byte aligned
 *   row_seq   int32 [n_tokens], or NULL: a negative entry marks a token without a request
 *             (rz_paged_plan's row_seq): it has no experts and no rows, its logits are not read
 *   renormalise  0: weights are the softmax over all experts, taken at the chosen; else the
 *             softmax over the chosen
 *   scale     times every weight
 * Of equal logits the lowest index comes first.  A logit of -infinity masks its expert for the token: it is
 * never chosen; a choice that is left without an expert has -1 and the weight 0.  A token with a NaN or +infinity among its
 * logits has weights NaN (a NaN is chosen after every number).
 *   workspace rz_moe_route_workspace_bytes bytes, 16-byte aligned; no initialisation; may be
 *             NULL where that is 0 (few tokens: one launch; more: two)
 */
size_t rz_moe_route_workspace_bytes(int64_t n_tokens, int32_t n_experts);
rz_status rz_moe_route(const float *logits, int64_t ld, const int32_t *row_seq, const rz_moe_plan *plan,
                       int32_t renormalise, float scale, void *workspace, size_t ws_bytes, rz_stream stream);

/*
 * rz_moe_swiglu -- h_r = silu(G_e x_t) * (U_e x_t) for every row r of the plan, e its expert, t its
 * token; the product of rz_q4k_q8_gemv.
 *   w_gate, w_up  Q4_K [n_experts][inter][in_dim]     x_q8  Q8_1 of n_tokens rows of in_dim
 *   h         f32 [n_tokens * top_k][inter] output, in the plan's order of rows, or NULL
 *   h_q8      Q8_1 of n_tokens * top_k rows of inter (rz_moe_down's input): exactly the quantisation of
 *             h, but d = s = NaN for a block with a NaN; or NULL (inter % 32 == 0)
 *   workspace rz_moe_swiglu_workspace_bytes bytes; no initialisation; may be NULL where that is 0
 *   in_dim % 256 == 0; all 16-byte aligned.  Rows behind offsets[n_experts] stay as they were.
 * Sums are f32-accurate: exact integer dots for few rows of an expert, else the tensor cores.  There codes enter with
 * every bit (where |dmin| is over 2^37 |d|, off by up to 2^-33 |dmin|), activations with 22 bits of the largest scale
 * among the 256 values that share a super-block: where a block's scale is 2^-k of that, its values are off by up to
 * 2^(k - 24) of its largest.  silu is within 11 half-ulps of the formula's.
 */
size_t rz_moe_swiglu_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t top_k, int64_t in_dim);
rz_status rz_moe_swiglu(const void *w_gate, const void *w_up, const void *x_q8, const rz_moe_plan *plan, int64_t inter,
                        int64_t in_dim, float *h, void *h_q8, void *workspace, size_t ws_bytes, rz_stream stream);

/*
 * rz_moe_down -- y_t = residual_t + sum_j weights[t][j] D_e h_r, r = places[t][j], e its expert, the
 * choices in order.
 *   w_down    Q4_K [n_experts][out_dim][in_dim]       h_q8  Q8_1 of n_tokens * top_k rows of in_dim
 *   residual  f32 [n_tokens][out_pad], or NULL: 0
 *   y         f32 [n_tokens][out_pad] output; may be residual; 0 in the columns out_dim .. out_pad.  A token
 *             without experts gets its residual.
 *   workspace rz_moe_down_workspace_bytes bytes, 16-byte aligned; no initialisation; may be NULL where that is 0
 * Sums as in rz_moe_swiglu.
 */
size_t rz_moe_down_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t top_k, int64_t out_dim, int64_t in_dim);
rz_status rz_moe_down(const void *w_down, const void *h_q8, const rz_moe_plan *plan, const float *residual, float *y,
                      int64_t out_dim, int64_t out_pad, int64_t in_dim, void *workspace, size_t ws_bytes,
                      rz_stream stream);

/*
 * rz_moe_ffn -- rz_moe_route, rz_moe_swiglu (its Q8_1 output) and rz_moe_down in one call, the
 * same results:  out = residual + the experts' FFNs of x, weighted.
 *   x_q8      Q8_1 of n_tokens rows of hidden_pad (rz_residual_rmsnorm's)
 *   w_gate, w_up Q4_K [n_experts][inter][hidden_pad]   w_down Q4_K [n_experts][hidden][inter]
 *   residual, out f32 [n_tokens][hidden_pad]; residual may be NULL or out; the padding of out is 0
 *   plan      receives the routing; hidden_pad and inter multiples of 256
 *   workspace rz_moe_ffn_workspace_bytes bytes, 16-byte aligned; no initialisation
 */
size_t rz_moe_ffn_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t top_k, int64_t hidden, int64_t hidden_pad,
                                  int64_t inter);
rz_status rz_moe_ffn(const float *logits, int64_t ld, const int32_t *row_seq, const void *x_q8, const void *w_gate,
                     const void *w_up, const void *w_down, const float *residual, float *out, const rz_moe_plan *plan,
                     int32_t renormalise, float scale, int64_t hidden, int64_t hidden_pad, int64_t inter, void *workspace,
                     size_t ws_bytes, rz_stream stream);

/*
 * rz_check_device_error -- synchronise `stream`, read the device error word of the
 * current device and clear it.  *code_out (nullable) receives the raw code (0 = none).
 * Returns RZ_OK, RZ_ERR_TIMEOUT (a bounded wait ran out) or RZ_ERR_DEVICE (a
 * device-side range check failed and the access was skipped).
 */
rz_status rz_check_device_error(rz_stream stream, uint32_t *code_out);

/*
 * rz_set_pdl -- enable (default) or disable programmatic dependent launch between
 * consecutive librz kernels in a stream.  With it a GEMV starts streaming its
 * weights while the previous kernel finishes; results are identical either way.
 */
rz_status rz_set_pdl(int enable);

/*
 * rz_debug_stall_next_gemv -- test aid for the bounded-wait error path (off by
 * default).  The next Q4_K GEMV launch of this process leaves the first weight
 * stage of its CTA 0 unissued and bounds every wait of that CTA by wait_limit
 * polls (1024 <= wait_limit <= 2^22, else RZ_ERR_INVALID_ARG).  Its consumer warps
 * then run out of their wait, record code 0x101 in the device error word and
 * stop; the CTA still waits for every copy it did issue before it exits, so no
 * copy outlives the kernel.  rz_check_device_error then returns RZ_ERR_TIMEOUT,
 * and the output rows of CTA 0 of that launch are undefined.  One shot: the
 * setting clears itself at that launch.  The pages return errors instead of
 * panicking (GpuError in realizar 0.8.5 forward_utils.rs); this checks that a
 * wait that cannot complete ends in such an error and not in a hung GPU.
 */
rz_status rz_debug_stall_next_gemv(uint32_t wait_limit);

/*
 * rz_debug_stall_next_paged -- the same for the next rz_attention_paged_q4 (or
 * rz_decode_layer_paged) of this process: CTA 0 leaves its first tokens uncopied, in each
 * kernel of the call in which it has any.  Code 0x110, RZ_ERR_TIMEOUT; the rows of the
 * items that CTA 0 works are undefined, and the workspace is to be filled with zeros again.
 */
rz_status rz_debug_stall_next_paged(uint32_t wait_limit);

/*
 * rz_debug_stall_next_moe -- the same for the next product of rz_moe_swiglu, rz_moe_down or
 * rz_moe_ffn that runs on the tensor cores: CTA 0 leaves its first weights uncopied.  Code 0x120,
 * RZ_ERR_TIMEOUT; the outputs of CTA 0 are undefined.
 */
rz_status rz_debug_stall_next_moe(uint32_t wait_limit);


#ifdef __cplusplus
}
#endif
#endif /* RZ_H */
