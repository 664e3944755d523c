// qk_norm_rope.cu -- the norms of queries and keys for each head, their rotation,
// and the append of the new keys and values to the 4-bit paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma          (each head of q and k; optional)
//   z = y rotated by position * theta^(-2i/head_dim) in pair i
//   K, V of the cache: blocks of 32 values, s the value of largest magnitude (of +a
//   and -a the positive one), d = f16(clamp(s / -8, +-65504)), code = clamp(
//   round-half-even(x / d) + 8, 0, 15); d == 0 gives codes 8; a block with a NaN or an
//   infinity gets d = NaN, so that what reads it sees it.
//
// A warp works one head of one token; lane l holds value 32 e + l of it in register
// e, so that a Q4_0 block is one register across the warp.  A CTA works the heads of
// one token (several CTAs share a token's heads when there are few tokens) and forms
// the token's cosines and sines once: the angle as a fraction of a turn is
// position * F_i mod 2^64 with F_i = 2^64 theta^(-2i/head_dim) / (2 pi), a product of
// integers, which drops whole turns exactly at any position and needs no f64.
//
// Codes of the definition: V is f32 and its codes are decided exactly (the sign of
// |x| - h |d| at the border h is exact in one fused multiply-add, since h |d| has 16
// significant bits).  K comes out of the norm and the rotation with an error below
// 2^-20 (|y0| + |y1|) of its pair: (head_dim / 32 + 5) / 2 <= 6.5 roundings of the sum
// of squares, 5 of the square root, quotient and products with gamma, 3.2 of a cosine
// or sine near 1 with its argument, 1.5 of the rotation, each 2^-24.  A warp that finds a
// value closer than that to the border of two codes, a scale as close to the border of
// two f16 numbers, or two largest values as close to each other works the head again
// in f64 (about one head in a hundred).  So the cache holds what the definition in 64
// bits says, whatever the order of the sums.
#include <math.h>

#include <algorithm>

#include "paged_q4.cuh"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kKeyError = 0x1p-20f;
constexpr double kTwoPiHi = 6.283185307179586476925286766559;
constexpr double kTwoPiLo = 2.449293598294706e-16;  // 2 pi - kTwoPiHi
constexpr double kInvTwoPi = 0.15915494309189533576888376337251;

// NaN wins in both
__device__ __forceinline__ float redux_max(float v)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float redux_min(float v)
{
    float r;
    asm volatile("redux.sync.min.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ double warp_sum_f64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_max_f64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// One pair's turn, as the lane that holds x (the other value of the pair is o) sees it.
template <typename T>
__device__ __forceinline__ T turned(T x, T o, T cs, T sn, bool first)
{
    return first ? x * cs - o * sn : o * sn + x * cs;
}

// Rotates a head held as x[e] = value 32 e + lane; pair(i, cs, sn) gives pair i's cosine
// and sine, mag[e] receives |x| + |o| of the value's pair.
template <int NB, typename T, typename F>
__device__ __forceinline__ void rotate(T (&x)[NB], T (&mag)[NB], int mode, int lane, F pair)
{
    constexpr int half = 16 * NB;
    T cs, sn;
    if (mode == 0) {  // pairs (2i, 2i + 1): the neighbouring lane
#pragma unroll
        for (int e = 0; e < NB; ++e) {
            const T o = __shfl_xor_sync(0xffffffffu, x[e], 1);
            pair(16 * e + (lane >> 1), cs, sn);
            mag[e] = fabs(x[e]) + fabs(o);
            x[e] = turned(x[e], o, cs, sn, (lane & 1) == 0);
        }
    } else if (NB % 2 == 0) {  // pairs (i, i + half): another register of the lane
#pragma unroll
        for (int e = 0; e < NB / 2; ++e) {
            const T a = x[e], b = x[e + NB / 2];
            pair(32 * e + lane, cs, sn);
            mag[e] = mag[e + NB / 2] = fabs(a) + fabs(b);
            x[e] = turned(a, b, cs, sn, true);
            x[e + NB / 2] = turned(b, a, cs, sn, false);
        }
    } else {
        // half is an odd multiple of 16: the partner of value 32 e + l lies in lane l ^ 16, at
        // register e + h or e - h - 1 (lanes below 16) or e + h + 1 or e - h (the others)
        constexpr int h = NB / 2;
        T r[NB];
#pragma unroll
        for (int e = 0; e < NB; ++e) r[e] = __shfl_xor_sync(0xffffffffu, x[e], 16);
        const bool low = lane < 16;
#pragma unroll
        for (int e = 0; e < NB; ++e) {
            const T ol = r[e + h < NB ? e + h : e - h - 1], oh = r[e + h + 1 < NB ? e + h + 1 : e - h];
            const T o = low ? ol : oh;
            const bool first = low ? e + h < NB : e + h + 1 < NB;
            const int d = 32 * e + lane;
            pair(first ? d : d - half, cs, sn);
            mag[e] = fabs(x[e]) + fabs(o);
            x[e] = turned(x[e], o, cs, sn, first);
        }
    }
}

struct Block {
    uint16_t d;  // f16 bits of the scale
    int code;    // this lane's code
    float value; // and what it stands for
};

__device__ __forceinline__ uint16_t scale_bits(float s8)
{
    const uint16_t b = __half_as_ushort(__float2half_rn(fminf(fmaxf(s8, -65504.0f), 65504.0f)));
    return (b & 0x7fffu) ? b : uint16_t(0);
}

__device__ __forceinline__ int signed_code(float mag, bool negative)
{
    const int m = static_cast<int>(mag);
    return min(max(negative ? 8 - m : 8 + m, 0), 15);
}

// The block of 32 values z, one in each lane, with |z - true z| <= err.  Returns true
// where the codes or the scale of the true values may be others.
template <bool kExact>
__device__ __forceinline__ bool quantise(float z, float err, Block &o)
{
    const float mx = redux_max(z), mn = redux_min(z);
    if (!(mx < INFINITY && mn > -INFINITY)) {  // the same in every lane
        o = Block{0x7e00, 8, __int_as_float(0x7fffffff)};
        return !kExact;
    }
    const float s = mx >= -mn ? mx : mn;
    o.d = scale_bits(s * -0.125f);
    bool unsure = false;
    if (!kExact) {
        const float eb = redux_max(err);
        unsure = fabsf(mx + mn) < 2.0f * eb || scale_bits((s - eb) * -0.125f) != scale_bits((s + eb) * -0.125f);
    }
    const float d = h2f(o.d), ad = fabsf(d), az = fabsf(z);
    if (ad == 0.0f) {
        o.code = 8;
        o.value = 0.0f;
        return unsure;
    }
    const float k = floorf(fminf(az * rcp_approx(ad), 64.0f));
    const float t = __fmaf_rn(-(k + 0.5f), ad, az);
    if (!kExact) unsure = unsure || fabsf(t) < err;
    const bool up = t > 0.0f || (t == 0.0f && (static_cast<int>(k) & 1));
    o.code = signed_code(up ? k + 1.0f : k, (z < 0.0f) != (d < 0.0f));
    o.value = static_cast<float>(o.code - 8) * d;
    return unsure;
}

// The same for values in f64, as the definition has them.
__device__ __forceinline__ void quantise_f64(double z, Block &o)
{
    const bool fine = __all_sync(0xffffffffu, fabs(z) < (double)INFINITY);
    if (!fine) {
        o = Block{0x7e00, 8, __int_as_float(0x7fffffff)};
        return;
    }
    const double mx = warp_max_f64(z), mn = -warp_max_f64(-z);
    o.d = scale_bits(static_cast<float>((mx >= -mn ? mx : mn) * -0.125));
    const float d = h2f(o.d);
    if (d == 0.0f) {
        o.code = 8;
        o.value = 0.0f;
        return;
    }
    const double m = fmin(rint(fabs(z) / fabs(static_cast<double>(d))), 64.0);
    o.code = signed_code(static_cast<float>(m), (z < 0.0) != (d < 0.0f));
    o.value = static_cast<float>(o.code - 8) * d;
}

// A head normed and rotated in f64.
template <int NB>
__device__ __noinline__ void head_f64(const float *src, const float *gamma, float eps, int pos, const double *freq,
                                      int mode, int lane, double (&z)[NB])
{
    double ss = 0.0, mag[NB];
#pragma unroll
    for (int e = 0; e < NB; ++e) {
        z[e] = src[32 * e + lane];
        ss = fma(z[e], z[e], ss);
    }
    if (gamma) {
        const double inv = 1.0 / sqrt(warp_sum_f64(ss) / (32 * NB) + eps);
#pragma unroll
        for (int e = 0; e < NB; ++e) z[e] = z[e] * inv * gamma[32 * e + lane];
    }
    rotate<NB, double>(z, mag, mode, lane, [&](int i, double &cs, double &sn) {
        const double ang = pos * freq[i], n = rint(ang * kInvTwoPi);
        sincos(fma(-n, kTwoPiLo, fma(-n, kTwoPiHi, ang)), &sn, &cs);
    });
}

// grid (tokens, splits): CTA (t, y) works heads y * per .. of token t's n_heads + 2
// n_kv_heads rows, a warp at a time, the next row's values on their way meanwhile.
template <int NB>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ HeadsArgs a)
{
    constexpr int hd = 32 * NB;
    __shared__ float2 tab[hd / 2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int pos = a.positions[t];
    if (pos < 0) return;  // the same for the whole CTA: a padding row
    for (int i = tid; i < hd / 2; i += kThreads) {
        const int turn = static_cast<int>(static_cast<uint64_t>(pos) * a.turn[i] >> 32);
        float2 cs;
        sincospif(static_cast<float>(turn) * 0x1p-31f, &cs.y, &cs.x);
        tab[i] = cs;
    }
    const int H = a.n_heads, K = a.n_kv_heads;
    const int rows = a.kv.pages ? H + 2 * K : H + K;
    const int per = (rows + gridDim.y - 1) / gridDim.y;
    const int r0 = blockIdx.y * per, r1 = min(rows, r0 + per);

    // where the token lies in the cache
    uint8_t *rec = nullptr;
    int tok = 0;
    if (a.kv.pages && a.slots) {
        const int64_t slot = a.slots[t];
        const int lg = a.kv.page_log + 4;
        if (slot >= 0 && (slot >> lg) < a.kv.n_pages) {
            const int in_page = static_cast<int>(slot & ((1 << lg) - 1));
            tok = in_page & 15;
            rec = a.kv.pages + ((((slot >> lg) * K) << a.kv.page_log) + (in_page >> 4)) * (int64_t)q4_record_bytes(hd);
        } else if (slot >= 0 && tid == 0) {
            set_error(a.err, DEV_BAD_SLOT);
        }
    }

    auto row_ptr = [&](int r) {
        return r < H ? a.q + t * a.ld_q + (int64_t)r * hd
                     : r < H + K ? a.k + t * a.ld_k + (int64_t)(r - H) * hd : a.v + t * a.ld_v + (int64_t)(r - H - K) * hd;
    };
    float nx[NB];
    if (r0 + warp < r1) {
        const float *p = row_ptr(r0 + warp);
#pragma unroll
        for (int e = 0; e < NB; ++e) nx[e] = p[32 * e + lane];
    }
    __syncthreads();
    for (int r = r0 + warp; r < r1; r += kWarps) {
        float x[NB], mag[NB];
#pragma unroll
        for (int e = 0; e < NB; ++e) x[e] = nx[e];
        if (r + kWarps < r1) {
            const float *p = row_ptr(r + kWarps);
#pragma unroll
            for (int e = 0; e < NB; ++e) nx[e] = p[32 * e + lane];
        }
        const bool is_v = r >= H + K, is_q = r < H;
        Block blk[NB];
        if (!is_v) {
            const float *gamma = is_q ? a.q_gamma : a.k_gamma;
            bool far = false;  // squares whose sum leaves f32's range
            if (gamma) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < NB; ++e) ss = fmaf(x[e], x[e], ss);
                ss = warp_sum(ss);
                if (!(ss > 1e-30f && ss < 1e37f)) {
                    bool any = false;
#pragma unroll
                    for (int e = 0; e < NB; ++e) any |= x[e] != 0.0f;
                    far = __any_sync(0xffffffffu, any);
                }
                const float inv = rms_scale(ss, hd, a.eps);
#pragma unroll
                for (int e = 0; e < NB; ++e) x[e] = x[e] * inv * __ldg(gamma + 32 * e + lane);
            }
            rotate<NB, float>(x, mag, a.rope_mode, lane, [&](int i, float &cs, float &sn) {
                const float2 c = tab[i];
                cs = c.x;
                sn = c.y;
            });
            bool again = far;
            if (!is_q && a.kv.pages) {
                bool unsure = false;
#pragma unroll
                for (int e = 0; e < NB; ++e) unsure |= quantise<false>(x[e], kKeyError * mag[e], blk[e]);
                again = __any_sync(0xffffffffu, unsure) || far;
            }
            if (again) {
                double z[NB];
                head_f64<NB>(row_ptr(r), gamma, a.eps, pos, a.freq, a.rope_mode, lane, z);
#pragma unroll
                for (int e = 0; e < NB; ++e) {
                    x[e] = static_cast<float>(z[e]);
                    if (!is_q && a.kv.pages) quantise_f64(z[e], blk[e]);
                }
            }
            if (is_q || !a.kv.pages) {
                float *o = is_q ? a.q_out + t * a.ld_qo + (int64_t)r * hd
                                : a.k_out ? a.k_out + (t * K + (r - H)) * (int64_t)hd : nullptr;
                if (o) {
#pragma unroll
                    for (int e = 0; e < NB; ++e) o[32 * e + lane] = x[e];
                }
                continue;
            }
        } else {
#pragma unroll
            for (int e = 0; e < NB; ++e) quantise<true>(x[e], 0.0f, blk[e]);
        }
        // a key or value of the cache
        const int h = is_v ? r - H - K : r - H;
        float *o = is_v ? a.v_out : a.k_out;
        if (o) {
            o += (t * K + h) * (int64_t)hd;
#pragma unroll
            for (int e = 0; e < NB; ++e) o[32 * e + lane] = blk[e].value;
        }
        if (rec) {
            uint8_t *base = rec + ((int64_t)h << a.kv.page_log) * q4_record_bytes(hd);
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const int high = __shfl_down_sync(0xffffffffu, blk[e].code, 16);
                if (lane < 16)
                    base[is_v ? q4_v_byte(NB, tok, e, lane) : q4_k_byte(NB, tok, e, lane)] =
                        static_cast<uint8_t>(blk[e].code | (high << 4));
                if (lane == e)
                    reinterpret_cast<uint16_t *>(base + (is_v ? q4_v_scale(NB, tok) : q4_k_scale(NB, tok)))[e] =
                        blk[e].d;
            }
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(HeadsArgs &a, int64_t rows, int head_dim, float rope_theta, cudaStream_t s)
{
    for (int i = 0; i < head_dim / 2; ++i) {
        a.freq[i] = pow((double)rope_theta, -2.0 * i / head_dim);
        const double turns = a.freq[i] * kInvTwoPi;
        a.turn[i] = static_cast<uint64_t>(static_cast<int64_t>((turns - floor(turns)) * 0x1p62)) << 2;
    }
    const int per_token = a.n_heads + (a.kv.pages ? 2 : 1) * a.n_kv_heads;
    // CTAs for each token: up to one row for each warp, so that a few tokens spread over
    // the SMs, and one for each token once the tokens alone fill them twice
    const int64_t want = 2 * (int64_t)dev_info().sm_count;
    const int64_t split = std::min<int64_t>((per_token + kWarps - 1) / kWarps, std::max<int64_t>(1, want / rows));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows, (unsigned)split);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    switch (head_dim / 32) {
        case 1: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<1>, a);
        case 2: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<2>, a);
        case 3: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<3>, a);
        case 4: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<4>, a);
        case 5: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<5>, a);
        case 6: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<6>, a);
        case 7: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<7>, a);
        default: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<8>, a);
    }
}

}  // namespace rz
