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
//
// Measured, in a graph whose empty kernels take 2.5 us each: 8 decodes 5.0 us; 1000 requests of up to 32768 tokens, 37
// with up to 777 new ones (6964 rows in all) and 90 that end, 13.0 us (its reads, two sums, a barrier, the stack's pages, the
// rows' table entries: six dependent trips to L2).
#include <cooperative_groups.h>

#include <algorithm>

#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

namespace cg = cooperative_groups;

// One CTA alone: 8 requests take as long, 64 with 85 rows 6.3 us (8 CTAs: 5.3), 500 with a row each 17.0 (6.9), 1000 with
// 6964 rows 46.9 (13.0).
constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kPlanMaxSeqs / kThreads;  // requests of a thread: tid * kPer ..
constexpr int kAhead = 8, kRows = 4;           // loads of a lane on their way at once

// Inclusive prefix sums over the CTA's threads of N values each; returns the totals in all.
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t (&all)[N], int64_t (*tmp)[kWarps], int lane, int warp)
{
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v[k], o);
            if (lane >= o) v[k] += u;
        }
        if (lane == 31) tmp[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int64_t before = 0;
        all[k] = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int64_t x = tmp[k][w];
            all[k] += x;
            before += w < warp ? x : 0;
        }
        v[k] += before;
    }
}

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a)
{
    __shared__ int64_t tmp[3][kWarps];
    __shared__ int32_t cu[kPlanMaxSeqs + 1];    // rows before request i
    __shared__ int32_t first[kPlanMaxSeqs];     // number of its first new page; -1: refused
    __shared__ int32_t cached[kPlanMaxSeqs], owned[kPlanMaxSeqs], back[kPlanMaxSeqs];
    __shared__ int32_t last_cu, all_handed;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const cg::cluster_group cluster = cg::this_cluster();
    const int n_ctas = kCtas, cta = blockIdx.x;  // the grid is one cluster
    pdl_launch_dependents();
    pdl_wait();

    if (tid == 0) last_cu = all_handed = 0;
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
    // rows: the requests whose rows end beyond the last row have none.  Pages returned,
    // and whether the stack has room for them
    int64_t sums[2] = {rows, give}, totals[2];
    block_scan(sums, totals, tmp, lane, warp);
    int64_t r = sums[0] - rows, g = sums[1] - give;
    int64_t total = free0 + totals[1];
    if (total > a.n_pages) {
        bad = true;
        total = a.n_pages;
    }
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
    fits = __reduce_max_sync(0xffffffffu, fits);
    if (lane == 0 && fits) atomicMax(&last_cu, fits);
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
    int64_t upto[1] = {need}, wanted[1];
    block_scan(upto, wanted, tmp + 2, lane, warp);  // and last_cu is whole
    int64_t p = upto[0] - need;
    int handed = 0;  // the pages of this and the served requests before it
    bool refused = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        const int64_t mine = p;
        p += n[j];
        const bool served = ok[j] && (n[j] == 0 || p <= total);
        if (ok[j] && !served) refused = true;
        if (served && n[j]) handed = static_cast<int>(p);
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
    handed = __reduce_max_sync(0xffffffffu, handed);
    if (lane == 0 && handed) atomicMax(&all_handed, handed);
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
        const int32_t *row = a.table + i * a.table_ld;
        const int n_back = static_cast<int>(min((int64_t)owned[i], a.n_pages - to));
        for (int b0 = 0; b0 < n_back; b0 += 32 * kAhead) {
            int32_t v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int b = b0 + 32 * u + lane;
                v[u] = b < n_back ? row[b] : 0;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int b = b0 + 32 * u + lane;
                if (b < n_back) a.free_pages[to + b] = v[u];
            }
        }
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
            *a.free_count_out = static_cast<int>(total - all_handed);
        }
    }
    // rows
    const int total_rows = cu[a.n_seqs], page_log = __ffs(a.page_size) - 1;
    // kRows at a time, so that their loads of the table are on their way together
    for (int64_t row0 = (int64_t)cta * kThreads + tid; row0 < a.max_rows; row0 += (int64_t)n_ctas * kThreads * kRows) {
        int32_t seq[kRows], pos[kRows];
        int64_t page[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t row = row0 + (int64_t)u * n_ctas * kThreads;
            seq[u] = pos[u] = -1;
            page[u] = -1;
            if (row < total_rows) {
                int lo = 0, hi = a.n_seqs;  // cu[lo] <= row < cu[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (cu[mid] <= row) lo = mid;
                    else hi = mid;
                }
                seq[u] = lo;
                if (first[lo] >= 0) {
                    pos[u] = cached[lo] + static_cast<int>(row - cu[lo]);
                    const int blk = pos[u] >> page_log;
                    const int32_t *from = blk < owned[lo] ? a.table + lo * a.table_ld + blk
                                                          : a.free_pages + (total - 1 - first[lo] - (blk - owned[lo]));
                    page[u] = __ldcg(from);
                }
            }
        }
        bool lost = false;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t row = row0 + (int64_t)u * n_ctas * kThreads;
            if (row < a.max_rows) {
                a.row_seq[row] = seq[u];
                a.positions[row] = pos[u];
                // a page below 0 would be a slot below 0, which stands for a row that is not to be appended
                lost |= pos[u] >= 0 && page[u] < 0;
                a.slots[row] = page[u] < 0 ? -1 : (page[u] << page_log) + (pos[u] & (a.page_size - 1));
            }
        }
        if (lost) set_error(a.err, DEV_BAD_PAGE);
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
}

}  // namespace rz
