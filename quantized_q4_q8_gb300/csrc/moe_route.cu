// moe_route.cu -- the router of an FFN of experts: the top k of each token's logits, their
// softmax weights, and the (token, choice) rows grouped by expert.
//
// Selection is exact: logits are compared as they are (as integers in the order of the
// floats, -0 as +0), of equal ones the lowest index first.  A logit of -infinity masks its expert.  A warp has a
// token, a lane the experts lane, lane + 32, ...; each of the k rounds takes the largest key of
// the warp and of its experts the lowest (two warp reductions).
//
// Grouping is a counting sort that keeps the order of the tokens.  Few tokens: one CTA
// selects, counts and places, one launch.  More: each CTA of the first launch selects for a
// range of tokens and writes down how many rows each expert gets from it; each CTA of the second adds up what the CTAs
// before it wrote and places its own range.  Atomics only count and set bits, so that nothing depends on their order.
//
// Bound: latency.  4 bytes a logit and 16 a row are read and written.  Few tokens: a launch, a trip to memory and the rounds (1 token, 8 of 64
// experts: 3.6 us).  Many: the second launch, each CTA of which reads the counts of all of the first (4095 tokens, 8 of 32, 128 and 512 experts: 6.8, 12.8 and
// 34 us; with one choice in place of 8, 5.9, 10.4 and 30 us).
#include <math.h>

#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {


// Order-preserving: -infinity (masked) and what is taken become 0, NaN 1, numbers more.
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (isnan(f)) return 1u;
    if (f == -INFINITY) return 0u;
    const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The choices of token t: expert ids and weights, and one count for each expert chosen.
template <int J>
__device__ __forceinline__ void select_token(const MoeRouteArgs &a, int64_t t, int lane, int *count)
{
    const int k = a.top_k;
    const bool idle = a.row_seq && a.row_seq[t] < 0;
    int mine = -1;        // lane j holds choice j
    float weight = 0.0f;
    if (!idle) {
        float v[J];
        uint32_t key[J];
        float sum = 0.0f;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = lane + 32 * j;
            v[j] = e < a.n_experts ? a.logits[t * a.ld + e] : -INFINITY;
            key[j] = order_key(v[j]);
            nan |= isnan(v[j]);
        }
        nan = __any_sync(0xffffffffu, nan);
        float top = 0.0f, logit = 0.0f;
        for (int c = 0; c < k; ++c) {
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < J; ++j) best = max(best, key[j]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0) break;  // none is left that is not masked
            int idx = 32 * J;
#pragma unroll
            for (int j = J - 1; j >= 0; --j)
                if (key[j] == best) idx = lane + 32 * j;
            idx = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(idx)));
            float chosen = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (idx == lane + 32 * j) {
                    chosen = v[j];
                    key[j] = 0;
                }
            chosen = __shfl_sync(0xffffffffu, chosen, idx & 31);
            if (c == 0) top = chosen;
            if (lane == c) {
                mine = idx;
                logit = chosen;
            }
        }
        if (mine >= 0) weight = expf(logit - top);
        if (a.renormalise) {
            sum = weight;
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (v[j] != -INFINITY) sum += expf(v[j] - top);
        }
        sum = warp_sum(sum);
        weight = mine < 0 ? 0.0f : nan ? NAN : weight / sum * a.scale;
    }
    if (lane < k) {
        a.experts[t * k + lane] = mine;
        a.weights[t * k + lane] = weight;
        if (mine >= 0) atomicAdd(count + mine, 1);
    }
}

__device__ __forceinline__ void select_any(const MoeRouteArgs &a, int64_t t, int lane, int *count)
{
    if (a.n_experts <= 32) return select_token<1>(a, t, lane, count);
    if (a.n_experts <= 64) return select_token<2>(a, t, lane, count);
    if (a.n_experts <= 128) return select_token<4>(a, t, lane, count);
    if (a.n_experts <= 256) return select_token<8>(a, t, lane, count);
    return select_token<16>(a, t, lane, count);
}

// next[e] = the first row of expert e: the sum of total[] before e, one warp for all
__device__ __forceinline__ int scan_experts(const int *total, int *next, int n_experts, int lane)
{
    int base = 0;
    for (int e0 = 0; e0 < n_experts; e0 += 32) {
        const int e = e0 + lane;
        const int own = e < n_experts ? total[e] : 0;
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (e < n_experts) next[e] = base + v - own;
        base += __shfl_sync(0xffffffffu, v, 31);
    }
    return base;
}

// The rows of tokens [t0, t1) in order, all of the CTA: each to the next place of its expert.  A token has an expert once, so
// that of 32 tokens a row's rank is the number of those before it that chose the same expert: bits of a word, whatever order they are set in.
template <int kThreads>
__device__ __forceinline__ void place_rows(const MoeRouteArgs &a, int64_t t0, int64_t t1, int *next, unsigned *chosen, int tid)
{
    for (int64_t t = t0; t < t1; t += 32) {
        for (int e = tid; e < a.n_experts; e += kThreads) chosen[e] = 0;
        __syncthreads();
        const int rows = static_cast<int>(min(static_cast<int64_t>(32), t1 - t)) * a.top_k;
        const int64_t base = t * a.top_k;
        static_assert(2 * kThreads >= 32 * kMoeMaxTopK, "rows of 32 tokens");
        int mine[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int p = tid + u * kThreads;
            mine[u] = p < rows ? a.experts[base + p] : -1;
            if (mine[u] >= 0) atomicOr(chosen + mine[u], 1u << (p / a.top_k));
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int p = tid + u * kThreads;
            if (p >= rows) break;
            const int at = mine[u] < 0 ? -1 : next[mine[u]] + __popc(chosen[mine[u]] & ((1u << (p / a.top_k)) - 1u));
            a.places[base + p] = at;
            if (at >= 0) a.rows[at] = static_cast<int>(base) + p;
        }
        __syncthreads();
        for (int e = tid; e < a.n_experts; e += kThreads) next[e] += __popc(chosen[e]);
        __syncthreads();
    }
}

// kPlace: one CTA does all.  Otherwise CTA c selects tokens [c * chunk, (c + 1) * chunk) and writes
// its counts to hist[c][e].
template <int kThreads, bool kPlace>
__global__ void __launch_bounds__(kThreads) moe_select_kernel(MoeRouteArgs a)
{
    __shared__ int count[kMoeMaxExperts], next[kMoeMaxExperts];
    __shared__ unsigned chosen[kPlace ? kMoeMaxExperts : 1];
    __shared__ int used;
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.n_experts; e += kThreads) count[e] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.n_tokens);
    for (int64_t t = t0 + warp; t < t1; t += kWarps) select_any(a, t, lane, count);
    __syncthreads();
    if constexpr (kPlace) {
        if (warp == 0) {
            const int all = scan_experts(count, next, a.n_experts, lane);
            for (int e = lane; e < a.n_experts; e += 32) a.offsets[e] = next[e];
            if (lane == 0) {
                a.offsets[a.n_experts] = all;
                used = all;
            }
        }
        place_rows<kThreads>(a, 0, a.n_tokens, next, chosen, tid);
        for (int64_t r = used + tid; r < a.n_tokens * a.top_k; r += kThreads) a.rows[r] = -1;
    } else {
        for (int e = tid; e < a.n_experts; e += kThreads) a.hist[blockIdx.x * a.n_experts + e] = count[e];
    }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) moe_place_kernel(MoeRouteArgs a)
{
    __shared__ int total[kMoeMaxExperts], before[kMoeMaxExperts], next[kMoeMaxExperts];
    __shared__ unsigned chosen[kMoeMaxExperts];
    __shared__ int used;
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.n_experts; e += kThreads) total[e] = before[e] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    // warps share the ranges, lanes the experts
    for (int e = lane; e < a.n_experts; e += 32) {
        int all = 0, mine = 0;
#pragma unroll 16
        for (int c = warp; c < static_cast<int>(gridDim.x); c += kWarps) {
            const int v = a.hist[c * a.n_experts + e];
            all += v;
            if (c < static_cast<int>(blockIdx.x)) mine += v;
        }
        atomicAdd(total + e, all);
        atomicAdd(before + e, mine);
    }
    __syncthreads();
    if (warp == 0) {
        const int all = scan_experts(total, next, a.n_experts, lane);
        for (int e = lane; e < a.n_experts; e += 32) {
            if (blockIdx.x == 0) a.offsets[e] = next[e];
            next[e] += before[e];
        }
        if (lane == 0) {
            if (blockIdx.x == 0) a.offsets[a.n_experts] = all;
            used = all;
        }
    }
    const int64_t t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.n_tokens);
    place_rows<kThreads>(a, t0, t1, next, chosen, tid);
    for (int64_t r = used + static_cast<int64_t>(blockIdx.x) * kThreads + tid; r < a.n_tokens * a.top_k;
         r += static_cast<int64_t>(gridDim.x) * kThreads)
        a.rows[r] = -1;
}

template <typename K>
cudaError_t launch(K kernel, int grid, int threads, const MoeRouteArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Up to 16 tokens, one CTA and one launch (8 of 128 experts: 16 tokens 4.8 us, 32 tokens 7.2; two launches 6.8); up to 512, CTAs of 512
// threads, a token for each warp (128 tokens 7.5 us, in CTAs of 1024 threads 8.6); more, of 1024 (4095 tokens 12.6 us, in the smaller ones
// 15.2: each CTA of the second launch reads what all of the first have counted).
constexpr int64_t kOneCta = 16, kSmallCtas = 512;
constexpr int64_t kMostCtas = 128;

int64_t route_chunk(int64_t n_tokens)
{
    if (n_tokens <= kOneCta) return n_tokens;
    if (n_tokens <= kSmallCtas) return 16;
    const int64_t least = (n_tokens + kMostCtas - 1) / kMostCtas;
    return (least + 31) / 32 * 32;
}

}  // namespace

int64_t moe_route_workspace_bytes(int64_t n_tokens, int n_experts)
{
    if (n_tokens <= kOneCta) return 0;
    const int64_t chunk = route_chunk(n_tokens);
    return (n_tokens + chunk - 1) / chunk * n_experts * 4;
}

cudaError_t launch_moe_route(MoeRouteArgs a, cudaStream_t s)
{
    a.chunk = route_chunk(a.n_tokens);
    if (a.n_tokens <= kOneCta) return launch(moe_select_kernel<512, true>, 1, 512, a, s);
    const int grid = static_cast<int>((a.n_tokens + a.chunk - 1) / a.chunk);
    const bool small = a.n_tokens <= kSmallCtas;
    const cudaError_t e = small ? launch(moe_select_kernel<512, false>, grid, 512, a, s) : launch(moe_select_kernel<1024, false>, grid, 1024, a, s);
    if (e != cudaSuccess) return e;
    return small ? launch(moe_place_kernel<512>, grid, 512, a, s) : launch(moe_place_kernel<1024>, grid, 1024, a, s);
}

}  // namespace rz
