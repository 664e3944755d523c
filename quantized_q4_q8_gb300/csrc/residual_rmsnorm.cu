// residual_rmsnorm.cu -- residual addition, RMSNorm of the sum and its Q8_1 form in one
// pass (steps 7-8 and 10-1 of transformer_layer_gpu_true_dp4a in realizar 0.8.5
// src/cuda/executor/cached.rs make them three; rms_norm_inplace in realizar 0.8.4
// src/gpu/adapters/using.rs is the norm):
//   s = x + delta (f32);  y = s / sqrt(sum_{i<n} s_i^2 / n + eps) * gamma;  Q8_1 of y
//
// Precision.  A code is decided by y / d, so y has to be the f32 nearest to the formula's value
// for the codes to be those of the formula, whatever the order of the sum: an error of one
// ulp of y moves one code in some 10^5.  The sum of squares, the scale and the products are
// therefore carried as sums of two f32 (about 2^-45 of the value; f64 would take as long as
// the copies do at this GPU's rate) and rounded once, when y is stored.
//
// Bound: bytes, 8 read and 9.25 written for each value.  A CTA has a row and holds it in
// registers between the sum and the outputs, a float4 of each 4 * kThreads values for a thread;
// eight threads hold a Q8_1 block.  4095 rows of 4096: 47.7 us, 6.07 TB/s, 89% of a copy's rate (issue slots 77%: the sums
// of two f32).  Few rows are a launch and a row's latency: 33 of 2048 2.8 us, 1 of 896 2.0 us.
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

// hi + lo, |lo| <= ulp(hi) / 2 up to the last additions
struct Two {
    float hi, lo;
};

__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two two_prod(float a, float b)
{
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two two_add(Two a, Two b)
{
    const Two s = two_sum(a.hi, b.hi);
    const float l = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s.hi, l);
    return {hi, __fsub_rn(l, __fsub_rn(hi, s.hi))};
}
__device__ __forceinline__ Two two_shfl(Two a, int mask)
{
    return {__shfl_xor_sync(0xffffffffu, a.hi, mask), __shfl_xor_sync(0xffffffffu, a.lo, mask)};
}

// 1 / sqrt(sum / n + eps): the quotient with its remainder, then a Newton step from the
// f32 square root, its residual 1 - v r^2 exact to 2^-45
__device__ __forceinline__ Two inverse_rms(Two sum, float n, float eps)
{
    const float q = __fdiv_rn(sum.hi, n);
    const float rest = __fadd_rn(__fmaf_rn(-q, n, sum.hi), sum.lo);
    const Two v = two_add({q, __fdiv_rn(rest, n)}, {eps, 0.0f});
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(v.hi));
    const Two rr = two_prod(r, r);
    const Two p = two_prod(rr.hi, v.hi);
    const float res = __fsub_rn(__fsub_rn(1.0f, p.hi), __fadd_rn(p.lo, __fmaf_rn(rr.hi, v.lo, __fmul_rn(rr.lo, v.hi))));
    return {r, __fmul_rn(0.5f * r, res)};
}

// The larger, NaN if one is: a block with a NaN has the scale NaN.
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

template <int kThreads, int kVec>
__global__ void __launch_bounds__(kThreads) residual_rmsnorm_kernel(const float *x, const float *delta, const float *__restrict__ gamma,
                                                                    float *sum, float *y, int8_t *__restrict__ q, float *__restrict__ qd,
                                                                    float *__restrict__ qs, int n, int n_pad, float eps)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ Two part[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x, at = row * n_pad;
    pdl_launch_dependents();
    pdl_wait();
    float s[kVec][4];
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
        const int i = 4 * (tid + k * kThreads);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (i < n) {
            a = *reinterpret_cast<const float4 *>(x + at + i);
            if (delta) b = *reinterpret_cast<const float4 *>(delta + at + i);
        }
        const float va[4] = {a.x, a.y, a.z, a.w}, vb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) s[k][e] = i + e < n ? (delta ? __fadd_rn(va[e], vb[e]) : va[e]) : 0.0f;
    }
    Two acc = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kVec; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Two p = two_prod(s[k][e], s[k][e]);
            const Two t = two_sum(acc.hi, p.hi);
            acc = {t.hi, __fadd_rn(acc.lo, __fadd_rn(t.lo, p.lo))};
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc = two_add(acc, two_shfl(acc, o));
    if (lane == 0) part[warp] = acc;
    __syncthreads();
    acc = lane < kWarps ? part[lane] : Two{0.0f, 0.0f};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) acc = two_add(acc, two_shfl(acc, o));
    acc = {__shfl_sync(0xffffffffu, acc.hi, 0), __shfl_sync(0xffffffffu, acc.lo, 0)};
    const Two r = inverse_rms(acc, static_cast<float>(n), eps);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
        const int i = 4 * (tid + k * kThreads);
        if (i - 4 * lane >= n_pad) break;  // the same for a warp; n_pad is a multiple of 32
        const bool in = i < n_pad;
        float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v[4];
        if (i + 3 < n) {
            const float4 t = __ldg(reinterpret_cast<const float4 *>(gamma + i));
            g[0] = t.x, g[1] = t.y, g[2] = t.z, g[3] = t.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) g[e] = __ldg(gamma + i + e);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float p = __fmul_rn(s[k][e], r.hi);
            const float pl = __fmaf_rn(s[k][e], r.lo, __fmaf_rn(s[k][e], r.hi, -p));
            const float w = __fmul_rn(p, g[e]);
            v[e] = i + e < n ? __fadd_rn(w, __fmaf_rn(pl, g[e], __fmaf_rn(p, g[e], -w))) : 0.0f;
        }
        if (in && sum) *reinterpret_cast<float4 *>(sum + at + i) = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
        if (in && y) *reinterpret_cast<float4 *>(y + at + i) = make_float4(v[0], v[1], v[2], v[3]);
        if (q) {
            float top = max_or_nan(max_or_nan(fabsf(v[0]), fabsf(v[1])), max_or_nan(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float d = __fmul_rn(top, 1.0f / 127.0f);  // within an ulp of the division that rz_q8_1_quantize makes
            const Q8Scale qsc = q8_scale(d);
            uint32_t word = 0;
            int total = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = q8_code(v[e], qsc);
                total += c;
                word |= (static_cast<uint32_t>(c) & 0xffu) << (8 * e);
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (in) {
                *reinterpret_cast<uint32_t *>(q + at + i) = word;
                if ((lane & 7) == 0) {
                    const int64_t b = (at + i) / 32;
                    qd[b] = d;
                    qs[b] = __fmul_rn(d, static_cast<float>(total));
                }
            }
        }
    }
}

template <int kThreads, int kVec>
cudaError_t launch(const float *x, const float *delta, const float *gamma, float *sum, float *y, void *q8, int64_t m, int n, int n_pad,
                   float eps, cudaStream_t s)
{
    int8_t *q = static_cast<int8_t *>(q8);
    float *qd = q ? reinterpret_cast<float *>(q + m * n_pad) : nullptr;
    float *qs = q ? qd + m * (n_pad / 32) : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(m));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, residual_rmsnorm_kernel<kThreads, kVec>, x, delta, gamma, sum, y, q, qd, qs, n, n_pad, eps);
}

}  // namespace

cudaError_t launch_residual_rmsnorm(const float *x, const float *delta, const float *gamma, float *sum, float *y, void *q8, int64_t m,
                                    int64_t n, int64_t n_pad, float eps, cudaStream_t s)
{
    const int ni = static_cast<int>(n), np = static_cast<int>(n_pad);
    if (np <= 1024) return launch<256, 1>(x, delta, gamma, sum, y, q8, m, ni, np, eps, s);
    if (np <= 2048) return launch<256, 2>(x, delta, gamma, sum, y, q8, m, ni, np, eps, s);
    if (np <= 4096) return launch<256, 4>(x, delta, gamma, sum, y, q8, m, ni, np, eps, s);
    if (np <= 8192) return launch<512, 4>(x, delta, gamma, sum, y, q8, m, ni, np, eps, s);
    return launch<512, 8>(x, delta, gamma, sum, y, q8, m, ni, np, eps, s);
}

}  // namespace rz
