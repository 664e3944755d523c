// moe_gemv.cu -- products grouped by expert of few rows: Q4_K weights of each expert against
// the Q8_1 rows that chose it, with exact integer dots; and the sum of a token's rows.
//
//   h[r][i] = silu(G_e[i] . x_t) * (U_e[i] . x_t)     row r of expert e, token t = rows[r] / k
//   o[r][i] = D_e[i] . h_r
//   y[t][i] = residual[t][i] + sum_j weights[t][j] * o[places[t][j]][i]
// with the product of rz_q4k_q8_gemv (exact integer dots of 32 codes, f32 sums).
//
// A CTA has a row and 32 outputs: 8 warps of 4 outputs, 4 lanes for a super-block of 256 weights (64 each), 8 super-blocks side by
// side.  The weights come straight from global memory, 12 loads of 16 bytes in flight for a lane; those of an expert with a
// second row come from L2 again.  (Four rows of an expert at once took 170 registers, spilled, and 37.9 instead of 26.3 us for
// one token of 2 of 8 experts, 4096 > 14336; 24.6 instead of 19.7 us for 4 tokens of 8 of 64, 2048 > 1024.)
//
// Bound: bytes where the weights are large (one token, 2 of 8 experts: gate and up 4096 > 14336 25.3 us, 5.2 TB/s; down 14336 >
// 4096 13.8 us, 4.8 TB/s), else the latency of dependent loads behind a launch (one token, 8 of 64: gate and up 2048 > 1024 6.3 us,
// 3.0 TB/s; down 1024 > 2048 6.7 us).
#include <algorithm>

#include "q4k_dot.cuh"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;    // outputs of a CTA
constexpr int kRows = 4;     // weight rows that a warp works at once

struct Weights64 {  // a lane's 64 weights: a header and 32 bytes of codes
    int4 h, a, b;
};

__device__ __forceinline__ int4 load_stream(const void *p)
{
    int4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The expert of row r, -1 where there is none; by each warp for itself.
__device__ __forceinline__ int find_expert(const MoeGemvArgs &a, int r, int lane)
{
    int found = -1;
#pragma unroll 4
    for (int e0 = 0; e0 < a.n_experts; e0 += 32) {
        const int e = min(e0 + lane, a.n_experts - 1), lo = a.offsets[e], hi = a.offsets[e + 1];
        const uint32_t here = __ballot_sync(0xffffffffu, lo <= r && r < hi && lo >= 0 && hi <= a.n_pairs);
        if (here && found < 0) found = min(e0 + __ffs(here) - 1, a.n_experts - 1);
    }
    return found;
}

// acc[k] += the lane's share of weight row k times row src of x.
__device__ __forceinline__ void dot_rows(const MoeGemvArgs &a, const uint8_t *const (&wr)[kRows], int src, int sub, int c, const LaneConst &L,
                                         float (&acc)[kRows])
{
    const int nsb = a.in_dim / 256, nb = a.in_dim / 32;
#pragma unroll 1
    for (int sb = sub; sb < nsb; sb += 8) {
        Weights64 w[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const uint8_t *p = wr[k] + sb * 144;
            w[k].h = load_stream(p);
            w[k].a = load_stream(p + 16 + 32 * c);
            w[k].b = load_stream(p + 32 + 32 * c);
        }
        float ds0[kRows], ds1[kRows], dm0[kRows], dm1[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const float d = h2f(static_cast<uint16_t>(static_cast<uint32_t>(w[k].h.x) & 0xffffu));
            const float dmin = h2f(static_cast<uint16_t>(static_cast<uint32_t>(w[k].h.x) >> 16));
            const uint32_t A = static_cast<uint32_t>(w[k].h.y) >> L.sh, B = static_cast<uint32_t>(w[k].h.z) >> L.sh,
                           C = static_cast<uint32_t>(w[k].h.w) >> L.sh;
            const uint32_t scp = (A & L.mask_lo) | (C & L.mask_c) | ((A >> 2) & L.mask_hi);
            const uint32_t mnp = (B & L.mask_lo) | ((C >> 4) & L.mask_c) | ((B >> 2) & L.mask_hi);
            ds0[k] = d * static_cast<float>(scp & 0xffu);
            ds1[k] = d * static_cast<float>((scp >> 8) & 0xffu);
            dm0[k] = dmin * static_cast<float>(mnp & 0xffu);
            dm1[k] = dmin * static_cast<float>((mnp >> 8) & 0xffu);
        }
        const int64_t j = static_cast<int64_t>(src) * nb + sb * 8 + 2 * c;
        const int4 *xp = reinterpret_cast<const int4 *>(a.xq + j * 32);
        const int4 x0 = __ldg(xp), x1 = __ldg(xp + 1), x2 = __ldg(xp + 2), x3 = __ldg(xp + 3);
        const float2 d8 = __ldg(reinterpret_cast<const float2 *>(a.xd + j)), s8 = __ldg(reinterpret_cast<const float2 *>(a.xs + j));
        const int xa[16] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w, x2.x, x2.y, x2.z, x2.w, x3.x, x3.y, x3.z, x3.w};
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int q[8] = {w[k].a.x, w[k].a.y, w[k].a.z, w[k].a.w, w[k].b.x, w[k].b.y, w[k].b.z, w[k].b.w};
            int i0 = 0, i1 = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                i0 = __dp4a(q[i] & 0x0f0f0f0f, xa[i], i0);
                i1 = __dp4a((q[i] >> 4) & 0x0f0f0f0f, xa[8 + i], i1);
            }
            float v = fmaf(ds0[k], d8.x * static_cast<float>(i0), acc[k]);
            v = fmaf(ds1[k], d8.y * static_cast<float>(i1), v);
            v = fmaf(-dm0[k], s8.x, v);
            acc[k] = fmaf(-dm1[k], s8.y, v);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 2) moe_swiglu_kernel(const MoeGemvArgs a)
{
    __shared__ float out[kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = lane & 3, sub = lane >> 2;
    const int nsb = a.in_dim / 256;
    const LaneConst L = lane_const(c);
    pdl_launch_dependents();
    pdl_wait();
    const int r = blockIdx.y;
    const int pair = a.rows[r], e = find_expert(a, r, lane);
    if (e < 0) return;
    const bool fine = pair >= 0 && pair < a.n_pairs;
    if (!fine && tid == 0) set_error(a.err, DEV_BAD_LENGTH);
    const int src = fine ? pair / a.top_k : 0;  // the row of x
    const int64_t wbase = static_cast<int64_t>(e) * a.out_dim;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        // a warp's outputs 4 warp .. + 3, gate and up of two of them at once
        const int o0 = 4 * warp + 2 * pass;
        const uint8_t *wr[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t o = min(static_cast<int64_t>(blockIdx.x) * kTile + o0 + (k >> 1), a.out_dim - 1);
            wr[k] = (k & 1 ? a.w2 : a.w1) + (wbase + o) * nsb * 144;
        }
        float acc[kRows] = {};
        dot_rows(a, wr, src, sub, c, L, acc);
#pragma unroll
        for (int k = 0; k < kRows; ++k) acc[k] = warp_sum(acc[k]);
        if (lane < 2) {
            const float g = lane ? acc[2] : acc[0], u = lane ? acc[3] : acc[1];
            out[o0 + lane] = g / (1.0f + expf(-g)) * u;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int64_t o = static_cast<int64_t>(blockIdx.x) * kTile + lane, at = static_cast<int64_t>(r) * a.out_dim + o;
        const float v = o < a.out_dim ? out[lane] : 0.0f;
        if (a.y && o < a.out_dim) a.y[at] = v;
        if (a.yq) {  // out_dim is a multiple of 32
            // as integers, which keep the order of the sizes and put NaN above them: a block with one has the scale NaN
            const float d = __fdiv_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v)))), 127.0f);
            const int code = q8_code(v, q8_scale(d)), total = warp_sum_int(code);
            a.yq[at] = static_cast<int8_t>(code);
            if (lane == 0) {
                a.yd[at / 32] = d;
                a.ys[at / 32] = __fmul_rn(d, static_cast<float>(total));
            }
        }
    }
}

__device__ __forceinline__ void copy_word(void *to, const void *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// Whether a place is among the rows lo .. hi of its expert, and those are rows: of another no product was made.
__device__ __forceinline__ bool is_row_of(int place, int lo, int hi, int n_pairs) { return lo >= 0 && lo <= place && place < hi && hi <= n_pairs; }

// y[t] = residual[t] + sum_j w_j D_e h_r in one launch, for few rows of an expert: a CTA has a token and 4 * quads outputs,
// a warp 4 outputs of one of its choices at a time.  What two tokens share comes from L2 again.
__global__ void __launch_bounds__(kThreads, 2) moe_down_tokens_kernel(const MoeGemvArgs a, const MoeCombineArgs b, int quads)
{
    __shared__ float out[kMoeMaxTopK][kTile];
    __shared__ int expert[kMoeMaxTopK], place_of[kMoeMaxTopK], bounds[kMoeMaxTopK][2];
    __shared__ float weight_of[kMoeMaxTopK];
    __shared__ bool live[kMoeMaxTopK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = lane & 3, sub = lane >> 2;
    const int nsb = a.in_dim / 256;
    const LaneConst L = lane_const(c);
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.y;
    const int64_t o0 = static_cast<int64_t>(blockIdx.x) * 4 * quads;
    // A lane of the last warp has a choice, whether it counts and its weight.  Its words come by asynchronous copies: in
    // registers across the dots they cost 2 to 3% more (two tokens of 8 in 64, 1024 > 2048: 11.5 instead of 11.3 us).
    if (warp == kThreads / 32 - 1 && lane < a.top_k) {
        const int e = b.experts[t * a.top_k + lane], at = min(max(e, 0), a.n_experts - 1);
        expert[lane] = e;
        copy_word(&bounds[lane][0], a.offsets + at);
        copy_word(&bounds[lane][1], a.offsets + at + 1);
        copy_word(&place_of[lane], b.places + t * a.top_k + lane);
        copy_word(&weight_of[lane], b.weights + t * a.top_k + lane);
    }
    for (int u = warp; u < a.top_k * quads; u += kThreads / 32) {
        const int j = u / quads, q = u - j * quads;
        const int e = b.experts[t * a.top_k + j], place = b.places[t * a.top_k + j];
        if (e < 0 || e >= a.n_experts || place < 0 || place >= a.n_pairs) continue;
        const uint8_t *wr[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) wr[k] = a.w1 + (e * a.out_dim + min(o0 + 4 * q + k, a.out_dim - 1)) * nsb * 144;
        float acc[kRows] = {};
        dot_rows(a, wr, place, sub, c, L, acc);
#pragma unroll
        for (int k = 0; k < kRows; ++k) acc[k] = warp_sum(acc[k]);
        if (lane < 4) out[j][4 * q + lane] = lane == 0 ? acc[0] : lane == 1 ? acc[1] : lane == 2 ? acc[2] : acc[3];
    }
    if (warp == kThreads / 32 - 1 && lane < a.top_k) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        const int e = expert[lane], place = place_of[lane];
        const bool fine = e >= 0 && e < a.n_experts && is_row_of(place, bounds[lane][0], bounds[lane][1], a.n_pairs);
        if (!fine && (e >= 0 || place >= 0)) set_error(a.err, DEV_BAD_LENGTH);
        live[lane] = fine;
    }
    __syncthreads();
    const int64_t col = o0 + tid;
    if (tid < 4 * quads && col < a.out_dim) {
        float v = b.residual ? b.residual[t * b.out_pad + col] : 0.0f;
        for (int j = 0; j < a.top_k; ++j)
            if (live[j]) v = fmaf(weight_of[j], out[j][tid], v);
        b.y[t * b.out_pad + col] = v;
    }
    // zeros behind out_dim, by the last CTA of the token
    if (blockIdx.x == gridDim.x - 1)
        for (int64_t z = a.out_dim + tid; z < b.out_pad; z += kThreads) b.y[t * b.out_pad + z] = 0.0f;
}

// y[t] = residual[t] + sum_j w_j o[place_j], zeros behind out_dim; a thread has kVec columns.  kParts: o is the sum of its parts, in
// order (a loop of one part for all would cost the large batches their loads side by side: 4095 tokens of 8, 366 to 399 us).
template <int kVec, bool kParts>
__global__ void __launch_bounds__(256) moe_combine_kernel(const MoeCombineArgs a)
{
    __shared__ int place_of[kMoeMaxTopK];
    __shared__ float weight_of[kMoeMaxTopK];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    if (threadIdx.x < a.top_k) {
        const int64_t pair = t * a.top_k + threadIdx.x;
        const int e = a.experts[pair], place = a.places[pair];
        weight_of[threadIdx.x] = a.weights[pair];
        const bool fine = e >= 0 && e < a.n_experts && is_row_of(place, a.offsets[e], a.offsets[e + 1], a.n_pairs);
        if (!fine && (e >= 0 || place >= 0)) set_error(a.err, DEV_BAD_LENGTH);
        place_of[threadIdx.x] = fine ? place : -1;
    }
    __syncthreads();
    const int col = (blockIdx.y * 256 + threadIdx.x) * kVec;
    if (col >= a.out_pad) return;
    const int parts = kParts ? *a.parts : 1;
    const int64_t part = static_cast<int64_t>(a.n_pairs) * a.out_dim;
    float v[kVec];
    if (col < a.out_dim) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = a.residual ? a.residual[t * a.out_pad + col + e] : 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int place = place_of[j];
            if (place < 0) continue;
            const float w = weight_of[j];
            const float *o = a.o + static_cast<int64_t>(place) * a.out_dim + col;
            if constexpr (kVec == 4) {
                float4 x = __ldg(reinterpret_cast<const float4 *>(o));
                for (int p = 1; p < parts; ++p) {
                    const float4 more = __ldg(reinterpret_cast<const float4 *>(o + p * part));
                    x = make_float4(x.x + more.x, x.y + more.y, x.z + more.z, x.w + more.w);
                }
                v[0] = fmaf(w, x.x, v[0]);
                v[1] = fmaf(w, x.y, v[1]);
                v[2] = fmaf(w, x.z, v[2]);
                v[3] = fmaf(w, x.w, v[3]);
            } else {
                float x = __ldg(o);
                for (int p = 1; p < parts; ++p) x += __ldg(o + p * part);
                v[0] = fmaf(w, x, v[0]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = 0.0f;
    }
    if constexpr (kVec == 4)
        *reinterpret_cast<float4 *>(a.y + t * a.out_pad + col) = make_float4(v[0], v[1], v[2], v[3]);
    else
        a.y[t * a.out_pad + col] = v[0];
}

template <typename K, typename A>
cudaError_t launch(K kernel, dim3 grid, const A &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_moe_swiglu(const MoeGemvArgs &a, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>((a.out_dim + kTile - 1) / kTile), static_cast<unsigned>(a.n_pairs));  // fewer than 11 kMoeMaxExperts
    return launch(moe_swiglu_kernel, grid, a, s);
}

cudaError_t launch_moe_down_tokens(const MoeGemvArgs &a, const MoeCombineArgs &b, int64_t n_tokens, cudaStream_t s)
{
    const int quads = moe_down_quads(a.top_k);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.out_dim + 4 * quads - 1) / (4 * quads)), static_cast<unsigned>(n_tokens));  // fewer than 11 kMoeMaxExperts
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, moe_down_tokens_kernel, a, b, quads);
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, int64_t n_tokens, cudaStream_t s)
{
    const int vec = a.out_dim % 4 == 0 && a.out_pad % 4 == 0 ? 4 : 1;
    const dim3 grid(static_cast<unsigned>(n_tokens), static_cast<unsigned>((a.out_pad + 256 * vec - 1) / (256 * vec)));
    if (a.parts) return vec == 4 ? launch(moe_combine_kernel<4, true>, grid, a, s) : launch(moe_combine_kernel<1, true>, grid, a, s);
    return vec == 4 ? launch(moe_combine_kernel<4, false>, grid, a, s) : launch(moe_combine_kernel<1, false>, grid, a, s);
}

}  // namespace rz
