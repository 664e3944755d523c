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
// e, which keeps most pairs of the rotation in a lane.  A CTA of 4 warps works the heads of one
// token (several CTAs share a token's heads when there are few tokens) and forms
// the token's cosines and sines once: the angle as a fraction of a turn is
// position * F_i mod 2^64 with F_i = 2^64 theta^(-2i/head_dim) / (2 pi), a product of
// integers, which drops whole turns exactly at any position.  Blocks are quantised four at a
// time, 8 lanes with 4 values each to a block: keys go through shared memory into that
// order, values are loaded in it.
//
// The cache holds the codes that the definition gives in 64 bits, whatever the order of
// the sums: a key that rounds to the other side of a border in f32 would be off by a
// whole step, and in a long prompt some would.  V is f32, and its codes are decided exactly (the
// sign of |x| - h |d| at a border h is exact in one fused multiply-add, since h |d| has 16
// significant bits).  K is carried as sums of two floats from the load to the code: squares,
// the inverse root (one Newton step), cosines and sines, rotation; each is good to about 2^-45, so
// a key is off by 2^-40 of its pair, but for the angle: its fraction of a turn for each position is a double's, so that
// it is off by position * 2^-52, which is more from position 4096 on (the f64 form's own angle is rounded at that size).
// That costs some 250 more instructions for a key head.  f64 costs more here: working
// only the doubtful heads (one in a hundred) in f64 took 12 us of 18 at 33 tokens of 32 + 64 heads of 128
// and 23 us of 79 at 4096 tokens of 32 + 16; f32 with bounds of its errors and the sums of two floats only for
// heads in doubt takes 6.8 us instead of 5.9 and 50.7 instead of 50.3.  Queries are f32.
//
// Bound: 4096 tokens of 32 + 16 heads of 128 read and write 206 MB and take 50.3 us, 4.1 TB/s or 60% of a copy's
// rate; the issue slots are 75% full (keys: 8 heads of 48 take 40% of the instructions).  Queries alone run at 6.7
// TB/s.  10 CTAs of 4 warps an SM (48 registers): 9 take 49.7 us there and 0.1 us more at 33 tokens, 12 (spills) 56.8,
// 8 50.0.  Two rows ahead in flight instead of one: 53.3.  Heads of 160 to 256 spill some registers at that (256: up to
// 200 bytes stored, 148 loaded a thread); 4096 tokens of 16 + 8 heads of 256, the same bytes, take 45.7 us all the
// same.  33 tokens of 32 + 64 heads: 5.9 us, latency.
#include <math.h>

#include <algorithm>

#include "paged_q4.cuh"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr double kInvTwoPi = 0.15915494309189533576888376337251;

// cos(2 pi j / 64) as the sum of two floats; sin is the same from the other end
__device__ const float2 kCos64[17] = {
    {0x1p+0f, 0x0p+0f},          {0x1.fd88dap-1f, 0x1.e89292p-28f},  {0x1.f6297cp-1f, 0x1.feeb96p-26f},
    {0x1.e9f416p-1f, -0x1.273a44p-26f}, {0x1.d906bcp-1f, 0x1.e651a8p-26f},  {0x1.c38b3p-1f, -0x1.cfe84ap-26f},
    {0x1.a9b662p-1f, 0x1.21d434p-26f},  {0x1.8bc806p-1f, 0x1.62a2e8p-26f},  {0x1.6a09e6p-1f, 0x1.9fcef4p-27f},
    {0x1.44cf32p-1f, 0x1.424776p-27f},  {0x1.1c73b4p-1f, -0x1.9465cep-27f}, {0x1.e2b5d4p-2f, -0x1.fe4272p-28f},
    {0x1.87de2ap-2f, 0x1.abaa58p-28f},  {0x1.294062p-2f, 0x1.dab3ep-27f},   {0x1.8f8b84p-3f, -0x1.cb2cfap-30f},
    {0x1.917a6cp-4f, -0x1.eb25eap-31f}, {0x0p+0f, 0x0p+0f}};

// ---------------------------------------------------------------- sums of two floats
// h + l, |l| at most half a step of h: Knuth's sum with its error (two_sum), Dekker's shorter one for |a| >= |b|, the
// error of a product by a fused multiply-add, and Dekker's sums and products of pairs.  Products by __fmul_rn: a
// product whose error is taken must not be fused into what uses it.
struct Two {
    float h, l;
};

__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = a + b, bb = s - a;
    return Two{s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ Two quick_sum(float a, float b)  // |a| >= |b|
{
    const float s = a + b;
    return Two{s, b - (s - a)};
}
__device__ __forceinline__ Two two_prod(float a, float b)
{
    const float p = __fmul_rn(a, b);
    return Two{p, fmaf(a, b, -p)};
}
// a * b, not brought to |l| <= half a step
__device__ __forceinline__ Two mul(Two a, float b)
{
    const Two p = two_prod(a.h, b);
    return Two{p.h, fmaf(a.l, b, p.l)};
}
__device__ __forceinline__ Two mul(Two a, Two b)
{
    const Two p = two_prod(a.h, b.h);
    return Two{p.h, p.l + fmaf(a.h, b.l, a.l * b.h)};
}
__device__ __forceinline__ Two add(Two a, Two b)
{
    const Two s = two_sum(a.h, b.h);
    return quick_sum(s.h, s.l + (a.l + b.l));
}

// Cosine and sine of a fraction of a turn, turn / 2^64: the nearest 64th of a turn from
// the table, the rest (at most 0.05) by its power series.
__device__ __forceinline__ void turn_cos_sin(uint64_t turn, const float2 *cos64, Two &c, Two &s)
{
    const uint64_t k = (turn + (1ull << 57)) >> 58;
    const int64_t r = static_cast<int64_t>(turn - (k << 58));
    const float rh = static_cast<float>(r), rl = static_cast<float>(r - static_cast<int64_t>(rh));
    // delta = 2 pi r / 2^64
    Two d = two_prod(rh, 0x1.921fb6p-62f);
    d.l += fmaf(rh, -0x1.777a5cp-87f, rl * 0x1.921fb6p-62f);
    Two d2 = two_prod(d.h, d.h);
    d2.l = fmaf(2.0f * d.h, d.l, d2.l);
    const float u = d2.h;
    const Two sd = {d.h, fmaf(d.h * u, fmaf(u, fmaf(u, -1.0f / 5040, 1.0f / 120), -1.0f / 6), d.l)};
    const Two cm = {-0.5f * d2.h, fmaf(u * u, fmaf(u, -1.0f / 720, 1.0f / 24), -0.5f * d2.l)};  // cos(delta) - 1
    const int j = static_cast<int>(k) & 15, quarter = static_cast<int>(k >> 4) & 3;
    const float2 tc = cos64[j], ts = cos64[16 - j];
    const Two C{tc.x, tc.y}, S{ts.x, ts.y};
    // cos(a + delta) = C + C cm - S sd, sin(a + delta) = S + S cm + C sd
    const Two ss = mul(S, sd), cs = mul(C, sd);
    const Two co = add(C, add(mul(C, cm), Two{-ss.h, -ss.l})), si = add(S, add(mul(S, cm), cs));
    c = quarter == 0 ? co : quarter == 1 ? Two{-si.h, -si.l} : quarter == 2 ? Two{-co.h, -co.l} : si;
    s = quarter == 0 ? si : quarter == 1 ? co : quarter == 2 ? Two{-si.h, -si.l} : Two{-co.h, -co.l};
}

// ---------------------------------------------------------------- a head in a warp
// NaN wins in both
__device__ __forceinline__ float redux_max(float v)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// Rotation of a head held as x[e] = value 32 e + lane: z[e] = x[e] cos + o[e] sin', o the
// other value of the pair and sin' its sine, negative in the pair's first value.
//   kMode 0: pairs (2i, 2i + 1), the neighbouring lane
//   kMode 1: pairs (i, i + hd/2), another register of the lane where hd/2 is a multiple of
//            32, else one of lane ^ 16: at e + NB/2 or e - NB/2 - 1 for lanes below 16, at
//            e + NB/2 + 1 or e - NB/2 for the others
template <int NB, int kMode>
struct Pairs {
    static constexpr bool same_lane = kMode == 1 && NB % 2 == 0;
    static constexpr int n = same_lane ? NB / 2 : NB;  // pairs of a lane with angles of their own

    static __device__ __forceinline__ bool first(int e, int lane)
    {
        if (kMode == 0) return (lane & 1) == 0;
        if (same_lane) return e < NB / 2;
        return lane < 16 ? e + NB / 2 < NB : e + NB / 2 + 1 < NB;
    }
    static __device__ __forceinline__ int pair(int e, int lane)
    {
        if (kMode == 0) return 16 * e + (lane >> 1);
        if (same_lane) return 32 * (e % n) + lane;
        return 32 * e + lane - (first(e, lane) ? 0 : 16 * NB);
    }
    static __device__ __forceinline__ void other(const float (&x)[NB], float (&o)[NB], int lane)
    {
        if (kMode == 0) {
#pragma unroll
            for (int e = 0; e < NB; ++e) o[e] = __shfl_xor_sync(0xffffffffu, x[e], 1);
        } else if (same_lane) {
#pragma unroll
            for (int e = 0; e < NB; ++e) o[e] = x[e < NB / 2 ? e + NB / 2 : e - NB / 2];
        } else {
            constexpr int h = NB / 2;
            float r[NB];
#pragma unroll
            for (int e = 0; e < NB; ++e) r[e] = __shfl_xor_sync(0xffffffffu, x[e], 16);
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const float low = r[e + h < NB ? e + h : e - h - 1], high = r[e + h + 1 < NB ? e + h + 1 : e - h];
                o[e] = lane < 16 ? low : high;
            }
        }
    }
};

// A head whose squares leave f32's range, scaled by a power of two (exact); returns eps
// scaled alike, which leaves the norm's result as it is.
template <int NB>
__device__ __forceinline__ float into_range(float (&x)[NB], float eps)
{
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < NB; ++e) mx = fmaxf(mx, fabsf(x[e]));
    mx = redux_max(mx);
    if (mx == 0.0f || !(mx < INFINITY)) return eps;
    int up = 127 - (__float_as_int(mx) >> 23);
    // eps may not leave the range either (where it counts, the squares need not)
    if (eps > 0.0f) up = min(up, (127 + 40 - (__float_as_int(eps) >> 23)) / 2);
    up = max(min(up, 126), -126);
    const float f = __int_as_float((up + 127) << 23);
#pragma unroll
    for (int e = 0; e < NB; ++e) x[e] *= f;
    return eps * f * f;
}
__device__ __forceinline__ bool in_range(float ss) { return ss > 1e-30f && ss < 1e37f; }

// Sum of squares of a head.
template <int NB>
__device__ __forceinline__ Two squares(const float (&x)[NB])
{
    Two a{0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < NB; ++e) {
        const Two p = two_prod(x[e], x[e]), t = two_sum(a.h, p.h);
        a = Two{t.h, a.l + (t.l + p.l)};
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Two t = two_sum(a.h, __shfl_xor_sync(0xffffffffu, a.h, o));
        a = Two{t.h, (a.l + __shfl_xor_sync(0xffffffffu, a.l, o)) + t.l};
    }
    return a;
}

// 1 / sqrt(ss / n + eps)
__device__ __forceinline__ Two inverse_rms(Two ss, int n, float eps)
{
    const float r = 1.0f / n, m = __fmul_rn(ss.h, r);
    const float ml = (fmaf(-m, static_cast<float>(n), ss.h) + ss.l) * r;
    const Two a = two_sum(m, eps);
    const float al = a.l + ml, y = rsqrtf(a.h);
    const Two y2 = two_prod(y, y), t = two_prod(a.h, y2.h);
    const float e = (1.0f - t.h) - (t.l + fmaf(a.h, y2.l, al * y2.h));  // 1 - a y^2
    // an infinite sum: 0, and no correction of it
    return Two{y, a.h < INFINITY ? y * e * fmaf(0.375f, e, 0.5f) : 0.0f};
}

// Codes and scale of a block of 32 values held by 8 lanes, 4 values z[k] + l[k] each (values
// 4 (lane & 7) ..): this lane's codes in 4 bytes, the values they stand for, the f16 bits of d.
struct Block4 {
    uint32_t codes;
    float4 value;
    uint16_t d;
};

__device__ __forceinline__ float max8(float v)
{
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <bool kTwo>
__device__ __forceinline__ Block4 quantise(const float (&z)[4], const float (&l)[4])
{
    float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), mn = fminf(fminf(z[0], z[1]), fminf(z[2], z[3]));
    // fmaxf passes over a NaN: a sum of zeros times the values does not
    const float odd = (z[0] * 0.0f + z[1] * 0.0f) + (z[2] * 0.0f + z[3] * 0.0f);
    mx = max8(mx);
    mn = -max8(-mn);
    const unsigned bad = __ballot_sync(0xffffffffu, odd != 0.0f || odd != odd);
    Block4 o;
    if (bad >> (threadIdx.x & 24) & 0xffu) {  // a NaN or an infinity in these 8 lanes' block
        const float nan = __int_as_float(0x7fffffff);
        mx = mn = 0.0f;
        o = Block4{0x08080808u, make_float4(nan, nan, nan, nan), 0x7e00};
    }
    float s = mx >= -mn ? mx : mn;
    if (kTwo) {  // of two peaks of one size in the high parts, the low ones tell which is larger
        const unsigned tie = __ballot_sync(0xffffffffu, mx == -mn && mx != 0.0f);
        if (tie) {
            float top = -INFINITY, low = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (z[k] == mx) top = fmaxf(top, l[k]);
                if (z[k] == mn) low = fmaxf(low, -l[k]);
            }
            top = max8(top);
            low = max8(low);
            if (mx == -mn && top < low) s = mn;
        }
    }
    if (bad >> (threadIdx.x & 24) & 0xffu) return o;
    o.d = __half_as_ushort(__float2half_rn(fminf(fmaxf(s * -0.125f, -65504.0f), 65504.0f)));
    if ((o.d & 0x7fffu) == 0) return Block4{0x08080808u, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0};
    const float d = h2f(o.d), ad = fabsf(d), rd = rcp_approx(ad);
    float v[4];
    o.codes = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float az = fabsf(z[k]);
        const float n = floorf(fminf(az * rd, 64.0f));
        const float t = __fmaf_rn(-(n + 0.5f), ad, az);
        int m = static_cast<int>(n);
        // beyond the border, or on it: then the low part tells, and of a tie the even code is taken
        bool up = t > 0.0f;
        if (t == 0.0f) {
            const float al = kTwo ? (z[k] < 0.0f ? -l[k] : l[k]) : 0.0f;
            up = al > 0.0f || (al == 0.0f && (m & 1));
        }
        m += up;
        const int c = min(max((z[k] < 0.0f) != (d < 0.0f) ? 8 - m : 8 + m, 0), 15);
        o.codes |= static_cast<uint32_t>(c) << (8 * k);
        v[k] = static_cast<float>(c - 8) * d;
    }
    o.value = make_float4(v[0], v[1], v[2], v[3]);
    return o;
}

// A block's bytes into its token's record.  Every lane calls it; live: this lane has a block.
template <int NB, bool kIsV>
__device__ __forceinline__ void put(const Block4 &o, int b, int lane, uint8_t *rec, int tok, bool live)
{
    const int q = lane & 7;
    const uint32_t bytes = o.codes | __shfl_down_sync(0xffffffffu, o.codes, 4) << 4;
    if (!live) return;
    if (q < 4) {  // bytes 4 q .. 4 q + 3
        if (kIsV) {
            uint8_t *p = rec + q4_v_byte(NB, tok, b, 4 * q);
#pragma unroll
            for (int k = 0; k < 4; ++k) p[16 * q4_v_run(NB) * k] = static_cast<uint8_t>(bytes >> (8 * k));
        } else {
            *reinterpret_cast<uint32_t *>(rec + q4_k_byte(NB, tok, b, 4 * q)) = bytes;
        }
    }
    if (q == 0) reinterpret_cast<uint16_t *>(rec + (kIsV ? q4_v_scale(NB, tok) : q4_k_scale(NB, tok)))[b] = o.d;
}

__device__ __forceinline__ void load4(float (&x)[4], const float *p, bool vector)
{
    if (vector) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = p[k];
    }
}
__device__ __forceinline__ void store4(float *p, const float4 &v, bool vector)
{
    if (vector) {
        *reinterpret_cast<float4 *>(p) = v;
    } else {
        p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
    }
}

static_assert(q4_v_byte(4, 5, 1, 7) - q4_v_byte(4, 5, 1, 4) == 3 * 16 * q4_v_run(4) &&
                  q4_v_byte(3, 5, 1, 15) - q4_v_byte(3, 5, 1, 12) == 3 * 16 * q4_v_run(3),
              "V's bytes of 4 values from a multiple of 4 on lie evenly");

// grid (tokens, splits): CTA (t, y) works rows y * per .. of token t's n_heads queries, then
// n_kv_heads keys, then its values 4 blocks at a time, a row a warp; a row's values are on their
// way while the warp works the one before.  The values come first, while the angles are formed.
template <int NB, int kMode>
__global__ void __launch_bounds__(kThreads, 10) qk_norm_rope_kernel(const __grid_constant__ HeadsArgs a)
{
    constexpr int hd = 32 * NB;
    using P = Pairs<NB, kMode>;
    __shared__ float4 tab[hd / 2];  // cos h, sin h, cos l, sin l of each pair
    __shared__ float2 cos64[17];
    __shared__ __align__(16) float keys[kWarps][2][hd];  // a rotated key, high and low parts
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    if (tid < 17) cos64[tid] = kCos64[tid];
    pdl_launch_dependents();
    pdl_wait();
    const int H = a.n_heads, K = a.n_kv_heads;
    const int v_rows = a.kv.pages ? (K * NB + 3) / 4 : 0, rows = H + K + v_rows;
    const int per = (rows + gridDim.y - 1) / gridDim.y;
    const int r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
    // position, slot, a row of values and one of a query or key are on their way together
    const int pos = a.positions[t];
    const int64_t slot = a.kv.pages ? a.slots[t] : -1;
    const bool v_vector = ((reinterpret_cast<uintptr_t>(a.v) | static_cast<uintptr_t>(a.ld_v) * 4) & 15) == 0;
    auto load_v = [&](float (&x)[4], int r) {  // 4 values of block beta of the token's values
        const int beta = 4 * (r - H - K) + (lane >> 3);
        load4(x, a.v + t * a.ld_v + (beta < K * NB ? 32 * beta + 4 * (lane & 7) : 0), v_vector);
    };
    int rv = r0 + warp;
    if (rv < H + K) rv += (H + K - rv + kWarps - 1) / kWarps * kWarps;
    float nv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (rv < r1) load_v(nv, rv);
    auto load = [&](float (&x)[NB], int r) {
        const float *p = r < H ? a.q + t * a.ld_q + (int64_t)r * hd : a.k + t * a.ld_k + (int64_t)(r - H) * hd;
#pragma unroll
        for (int e = 0; e < NB; ++e) x[e] = p[32 * e + lane];
    };
    float nx[NB];
    const int last = min(r1, H + K);  // of the rows of whole heads
    if (r0 + warp < last) load(nx, r0 + warp);
    if (pos < 0) return;  // the same for the whole CTA: a padding row

    // where the token lies in the cache
    uint8_t *rec = nullptr;
    int tok = 0;
    {
        const int lg = a.kv.page_log + 4;
        if (slot >= 0 && (slot >> lg) < a.kv.n_pages) {
            const int in_page = static_cast<int>(slot & ((1 << lg) - 1));
            tok = in_page & 15;
            rec = a.kv.pages + ((((slot >> lg) * K) << a.kv.page_log) + (in_page >> 4)) * (int64_t)q4_record_bytes(hd);
        } else if (slot >= 0 && tid == 0) {
            set_error(a.err, DEV_BAD_SLOT);
        }
    }
    __syncthreads();  // cos64
    for (int i = tid; i < hd / 2; i += kThreads) {
        Two c, s;
        turn_cos_sin(static_cast<uint64_t>(pos) * a.turn[i], cos64, c, s);
        tab[i] = make_float4(c.h, s.h, c.l, s.l);
    }
    // ---- values: rows H + K .., which need no angles
    const bool o_vector = (reinterpret_cast<uintptr_t>(a.v_out) & 15) == 0;
    for (; rv < r1; rv += kWarps) {
        const int beta = 4 * (rv - H - K) + (lane >> 3), h = beta / NB, b = beta - h * NB;
        const bool live = beta < K * NB;
        const float x[4] = {nv[0], nv[1], nv[2], nv[3]};
        if (rv + kWarps < r1) load_v(nv, rv + kWarps);
        const Block4 blk = quantise<false>(x, x);
        if (a.v_out && live) store4(a.v_out + t * (int64_t)(K * hd) + 32 * beta + 4 * (lane & 7), blk.value, o_vector);
        put<NB, true>(blk, b, lane, rec + ((int64_t)h << a.kv.page_log) * q4_record_bytes(hd), tok, live && rec != nullptr);
    }
    __syncthreads();

    int r = r0 + warp;
    auto next = [&](float (&x)[NB]) {  // row r's values, and the next row's on their way
#pragma unroll
        for (int e = 0; e < NB; ++e) x[e] = nx[e];
        if (r + kWarps < last) load(nx, r + kWarps);
    };
    // ---- queries
    if (r < min(r1, H)) {
        float g[NB], c[P::n], s[P::n];
#pragma unroll
        for (int e = 0; e < NB; ++e) g[e] = a.q_gamma ? __ldg(a.q_gamma + 32 * e + lane) : 1.0f;
#pragma unroll
        for (int e = 0; e < P::n; ++e) {
            const float4 v = tab[P::pair(e, lane)];
            c[e] = v.x;
            s[e] = v.y;
        }
        for (; r < min(r1, H); r += kWarps) {
            float x[NB], o[NB];
            next(x);
            if (a.q_gamma) {
                float ss = 0.0f, eps = a.eps;
#pragma unroll
                for (int e = 0; e < NB; ++e) ss = fmaf(x[e], x[e], ss);
                ss = warp_sum(ss);
                if (!in_range(ss)) {
                    eps = into_range(x, eps);
                    ss = 0.0f;
#pragma unroll
                    for (int e = 0; e < NB; ++e) ss = fmaf(x[e], x[e], ss);
                    ss = warp_sum(ss);
                }
                const float inv = rsqrtf(fmaf(ss, 1.0f / hd, eps));
#pragma unroll
                for (int e = 0; e < NB; ++e) x[e] = x[e] * inv * g[e];
            }
            P::other(x, o, lane);
            float *out = a.q_out + t * a.ld_qo + (int64_t)r * hd + lane;
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const float sn = s[e % P::n];
                out[32 * e] = fmaf(o[e], P::first(e, lane) ? -sn : sn, x[e] * c[e % P::n]);
            }
        }
    }
    // ---- keys
    const bool k_vector = a.k_out && (reinterpret_cast<uintptr_t>(a.k_out) & 15) == 0;
    for (; r < last; r += kWarps) {
        float x[NB], o[NB], xl[NB], ol[NB];
        next(x);
#pragma unroll
        for (int e = 0; e < NB; ++e) xl[e] = 0.0f;
        if (a.k_gamma) {
            float eps = a.eps;
            Two ss = squares(x);
            if (!in_range(ss.h)) {
                eps = into_range(x, eps);
                ss = squares(x);
            }
            const Two inv = inverse_rms(ss, hd, eps);
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const Two y = mul(mul(inv, __ldg(a.k_gamma + 32 * e + lane)), x[e]);
                x[e] = y.h;
                xl[e] = y.l;
            }
        }
        P::other(x, o, lane);
        P::other(xl, ol, lane);
        const int h = r - H;
        float *out = a.k_out ? a.k_out + (t * K + h) * (int64_t)hd : nullptr;
        uint8_t *base = rec ? rec + ((int64_t)h << a.kv.page_log) * q4_record_bytes(hd) : nullptr;
#pragma unroll
        for (int e = 0; e < NB; ++e) {
            const float4 cs = tab[P::pair(e, lane)];
            const bool first = P::first(e, lane);
            const Two z = add(mul(Two{x[e], xl[e]}, Two{cs.x, cs.z}),
                              mul(Two{o[e], ol[e]}, first ? Two{-cs.y, -cs.w} : Two{cs.y, cs.w}));
            if (a.kv.pages) {
                keys[warp][0][32 * e + lane] = z.h;
                keys[warp][1][32 * e + lane] = z.l;
            } else if (out) {
                out[32 * e + lane] = z.h;
            }
        }
        if (!a.kv.pages) continue;
        __syncwarp();
#pragma unroll
        for (int b0 = 0; b0 < NB; b0 += 4) {
            const int b = b0 + (lane >> 3);
            const bool live = b < NB;
            float zh[4], zl[4];
            load4(zh, keys[warp][0] + (live ? 32 * b : 0) + 4 * (lane & 7), true);
            load4(zl, keys[warp][1] + (live ? 32 * b : 0) + 4 * (lane & 7), true);
            const Block4 blk = quantise<true>(zh, zl);
            if (out && live) store4(out + 32 * b + 4 * (lane & 7), blk.value, k_vector);
            put<NB, false>(blk, b, lane, base, tok, live && base != nullptr);
        }
        __syncwarp();  // keys is read
    }
}

template <int kMode>
cudaError_t launch(const cudaLaunchConfig_t &cfg, const HeadsArgs &a, int nb)
{
    switch (nb) {
        case 1: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<1, kMode>, a);
        case 2: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<2, kMode>, a);
        case 3: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<3, kMode>, a);
        case 4: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<4, kMode>, a);
        case 5: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<5, kMode>, a);
        case 6: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<6, kMode>, a);
        case 7: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<7, kMode>, a);
        default: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<8, kMode>, a);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(HeadsArgs &a, int64_t rows, int head_dim, float rope_theta, cudaStream_t s)
{
    // theta^(-2i/head_dim) as the product of two powers, i = 16 j + k: fewer calls of pow
    double low[16], high[8];
    for (int k = 0; k < 16; ++k) low[k] = pow((double)rope_theta, -2.0 * k / head_dim);
    for (int j = 0; 16 * j < head_dim / 2; ++j) high[j] = pow((double)rope_theta, -32.0 * j / head_dim) * kInvTwoPi;
    for (int i = 0; i < head_dim / 2; ++i) {
        const double turns = low[i % 16] * high[i / 16];
        a.turn[i] = static_cast<uint64_t>(static_cast<int64_t>((turns - floor(turns)) * 0x1p62)) << 2;
    }
    const int per_token = a.n_heads + a.n_kv_heads + (a.kv.pages ? (a.n_kv_heads * (head_dim / 32) + 3) / 4 : 0);
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
    return a.rope_mode == 0 ? launch<0>(cfg, a, head_dim / 32) : launch<1>(cfg, a, head_dim / 32);
}

}  // namespace rz
