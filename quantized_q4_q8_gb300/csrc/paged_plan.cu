// paged_plan.cu -- page tables and slot maps from request lengths, on the GPU.
//
// For request i with cached_i tokens held and fresh_i new ones (fresh_i < 0: it has
// ended and its pages go back):
//   pages it needs  n_i = max(0, ceil((cached_i + fresh_i) / page_size) - owned_i)
//   free pages      a stack: the pages given back lie on top of it, in order of request
//                   and block; page number k handed out is the k-th from its top
//   served          n_i == 0, or n_0 + ... + n_i fits into the stack
//   row r of the packed new tokens belongs to the request whose [cu_i, cu_i+1) holds it,
//   at position cached_i + r - cu_i and at slot page * page_size + position % page_size.
// Two prefix sums over the requests (rows; then pages) give every output.
//
// Bound by latency: the largest case moves some 100 KB.  One launch of one cluster; each
// of its CTAs forms the prefix sums for itself (1024 requests are 12 KB of L2 reads), so
// nothing but one cluster barrier, between the reads of the state and its updates, joins
// them, and each writes its share of the pages and rows.  A row whose page is new takes it from
// the stack, not from the table, so it needs not wait for the table's update.
#include <cooperative_groups.h>

#include <algorithm>

#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kPlanMaxSeqs / kThreads;  // requests of a thread: tid * kPer ..

// Inclusive prefix sum over the CTA's threads of one value each; tmp holds kWarps + 1 values.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *tmp, int lane, int warp)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // tmp of the scan before is read
    if (lane == 31) tmp[warp] = v;
    __syncthreads();
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) before += w < warp ? tmp[w] : 0;
    return v + before;
}

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a)
{
    __shared__ int64_t tmp[kWarps];
    __shared__ int32_t cu[kPlanMaxSeqs + 1];    // rows before request i
    __shared__ int32_t first[kPlanMaxSeqs];     // number of its first new page; -1: refused
    __shared__ int32_t cached[kPlanMaxSeqs], owned[kPlanMaxSeqs], back[kPlanMaxSeqs];
    __shared__ int32_t last_cu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const cg::cluster_group cluster = cg::this_cluster();
    const int n_ctas = gridDim.x, cta = blockIdx.x;  // the grid is one cluster
    pdl_launch_dependents();
    pdl_wait();

    if (tid == 0) last_cu = 0;
    const int64_t max_pages_seq = a.max_blocks;
    bool bad = false;
    int c[kPer], f[kPer], o[kPer], odd[kPer];
    int64_t rows = 0, give = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        c[j] = f[j] = o[j] = odd[j] = 0;
        if (i < a.n_seqs) {
            c[j] = a.cached[i];
            f[j] = a.fresh[i];
            o[j] = a.owned[i];
            if (o[j] < 0 || o[j] > a.max_blocks) {
                bad = true;
                odd[j] = o[j];
                o[j] = 0;
                c[j] = -1;  // refused
            }
            rows += max(f[j], 0);
            if (f[j] < 0) give += o[j];
        }
    }
    int64_t free0 = *a.free_count;
    if (free0 < 0 || free0 > a.n_pages) {
        bad = true;
        free0 = 0;
    }
    // rows: the requests whose rows end beyond the last row have none
    int64_t r = block_scan(rows, tmp, lane, warp) - rows;
    int fits = 0;
    bool fit[kPer];
    int64_t at[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        at[j] = r;
        r += max(f[j], 0);
        fit[j] = r <= a.max_rows;
        if (fit[j]) fits = static_cast<int>(r);
        else if (f[j] > 0) bad = true;
    }
    atomicMax(&last_cu, fits);
    // pages returned, and whether the stack has room for them
    const int64_t gave = block_scan(give, tmp, lane, warp);
    int64_t g = gave - give;
    __shared__ int64_t all_back;
    if (tid == kThreads - 1) all_back = gave;
    __syncthreads();
    int64_t total = free0 + all_back;
    if (total > a.n_pages) {
        bad = true;
        total = a.n_pages;
    }
    // pages needed
    int64_t need = 0, n[kPer];
    bool ok[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        n[j] = 0;
        ok[j] = f[j] < 0 || (c[j] >= 0 && (fit[j] || f[j] == 0));
        if (f[j] >= 0 && ok[j]) {
            const int64_t blocks = ((int64_t)c[j] + f[j] + a.page_size - 1) / a.page_size;
            if (blocks > max_pages_seq || (int64_t)c[j] > (int64_t)o[j] * a.page_size) {
                ok[j] = false;  // longer than its table row, or tokens held in no page
            } else {
                n[j] = max(blocks - o[j], (int64_t)0);
            }
        }
        if (!ok[j]) bad = true;
        need += n[j];
    }
    int64_t p = block_scan(need, tmp, lane, warp) - need;
    int64_t taken = 0;
    bool refused = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        const int64_t mine = p;
        p += n[j];
        const bool served = ok[j] && (n[j] == 0 || p <= total);
        if (ok[j] && !served) refused = true;
        if (served) taken += n[j];
        if (i < a.n_seqs) {
            cu[i] = fit[j] ? static_cast<int>(at[j]) : last_cu;
            cached[i] = c[j];
            owned[i] = o[j];
            first[i] = served ? (n[j] ? static_cast<int>(mine) : 0) : -1;
            back[i] = f[j] < 0 ? static_cast<int>(min(g, a.n_pages)) : -1;
            if (f[j] < 0) g += o[j];
        }
        // kept for the writes after the barrier: served requests' new page counts
        n[j] = served ? n[j] : 0;
        ok[j] = served;
    }
    const int64_t handed = block_scan(taken, tmp, lane, warp);
    if (tid == kThreads - 1) all_back = handed;
    if (tid == 0) cu[a.n_seqs] = last_cu;
    __syncthreads();
    if (cta == 0) {
        if (bad) set_error(a.err, DEV_BAD_LENGTH);
        if (refused) set_error(a.err, DEV_NO_PAGES);
    }
    // pages of ended requests on top of the stack, a warp for each request
    for (int i = cta * kWarps + warp; i < a.n_seqs; i += n_ctas * kWarps) {
        if (back[i] < 0) continue;
        const int64_t to = free0 + back[i];
        for (int b = lane; b < owned[i]; b += 32)
            if (to + b < a.n_pages) a.free_pages[to + b] = a.table[i * a.table_ld + b];
    }
    // every CTA has read the state, and the stack is whole
    cluster.sync();
    auto page_number = [&](int64_t k) { return __ldcg(a.free_pages + (total - 1 - k)); };
    for (int i = cta * kWarps + warp; i < a.n_seqs; i += n_ctas * kWarps) {
        if (back[i] >= 0 || first[i] < 0) continue;
        const int64_t len = (int64_t)cached[i] + (cu[i + 1] - cu[i]);
        const int fresh_pages = static_cast<int>((len + a.page_size - 1) / a.page_size) - owned[i];
        for (int b = lane; b < fresh_pages; b += 32)
            a.table[i * a.table_ld + owned[i] + b] = page_number((int64_t)first[i] + b);
    }
    // what is known for each request
    if (cta == 0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            if (i < a.n_seqs) {
                a.cu_rows[i] = cu[i];
                a.kv_len[i] = ok[j] && f[j] >= 0 ? c[j] + f[j] : 0;
                // a count outside its range stays as it is, for whoever looks for the fault
                a.owned_out[i] = f[j] < 0 ? 0 : (odd[j] ? odd[j] : o[j]) + static_cast<int>(n[j]);
            }
        }
        if (tid == 0) {
            a.cu_rows[a.n_seqs] = last_cu;
            *a.free_count_out = static_cast<int>(total - all_back);
        }
    }
    // rows
    const int total_rows = cu[a.n_seqs];
    for (int64_t row = (int64_t)cta * kThreads + tid; row < a.max_rows; row += (int64_t)n_ctas * kThreads) {
        int32_t seq = -1, pos = -1;
        int64_t slot = -1;
        if (row < total_rows) {
            int lo = 0, hi = a.n_seqs;  // cu[lo] <= row < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= row) lo = mid;
                else hi = mid;
            }
            seq = lo;
            if (first[lo] >= 0) {
                pos = cached[lo] + static_cast<int>(row - cu[lo]);
                const int blk = pos / a.page_size;
                const int32_t page = blk < owned[lo] ? a.table[lo * a.table_ld + blk]
                                                     : page_number((int64_t)first[lo] + (blk - owned[lo]));
                slot = (int64_t)page * a.page_size + pos % a.page_size;
            }
        }
        a.row_seq[row] = seq;
        a.positions[row] = pos;
        a.slots[row] = slot;
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t s)
{
    // one CTA until its share of the rows is over some rows for each thread
    const int ctas = a.max_rows <= 4 * kThreads && a.n_seqs <= kThreads ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
}

}  // namespace rz
