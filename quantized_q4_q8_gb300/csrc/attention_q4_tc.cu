// attention_q4_tc.cu -- attention of many new rows (a prompt chunk) over the pages of
// the 4-bit KV cache, on tcgen05.mma.
//
// The formulas, the cache and the arguments are those of attention_q4.cu; this kernel
// works the requests with more than kTcRows query rows for a kv head, that one the others.
//
// An item is (request, kv head, 128 query rows); a tile is 128 tokens.  For each tile
//   S = Q K^T     128 x 128, A = Q and B = K from shared memory, S in tensor memory
//   O += P V      128 x hd, A = P from tensor memory, B = V from shared memory
// Precision: f16 operands in two pieces each.  q and the weights are split into a high and a
// low half (22 bits); a key is d * (code - 8), 15 significant bits, so its high and low
// halves hold it exactly.  high * high + low * high + high * low is three products, off by 2^-22
// at most; three products of codes without scales would be two, but every block of 32 would then
// need accumulators of its own, and 4 times the reads of tensor memory, which have to be
// multiplied and added.  K and V are brought near 1 by a power of two for each tile
// (exact), so that f16 holds them whatever their scale; it goes into the exponents.
//
// Softmax: a thread has a row of a tile, two groups of warps the tiles in turn: what one needs of the other is the
// running maximum, early.  (One group of twice the width, two threads for a row, took as long for a tile as the
// products of nearly two: loads, exchanges and stores one after another.)  The sums O stay in
// tensor memory and are rescaled there when a row's maximum has grown by over 2^8, and not before
// (see attention_q4.cu).
//
// Sums.  The tensor cores cut what they add to an accumulator instead of rounding it: 24 steps a
// tile let O drift towards zero by 1.6e-8 a step (1.2e-5 after 4000 tokens).  So O starts again every
// kPeriod tiles, and the sums before are added up in the workspace (rounded adds, one thread after the other
// for each value, in the unit of the row's maximum when its first sums went there, or when it had grown by
// 2^60 since).  S's low products come
// first, while its accumulators are small.
//
// The tensor pipe is never to wait: while it works P V of tile i, warps unpack K of tile i + 3
// and V of tile i + 1 and form the weights of tiles i + 1 and i + 2 from S, of which there are three (P takes its S's place):
//   warp 0       copies records (K, V's scales; V's codes) with the bulk-copy engine
//   warp 1       issues the products as their operands come, QK up to two tiles ahead of PV
//   warps 4-11   softmax (4-7 the even tiles, 8-11 the odd ones), and the outputs
//   warps 12-15  unpack K, warps 16-19 V
// Operands lie in core matrices of 8 rows x 16 bytes without a swizzle.  Within every 4 values of the
// inner dimension the order is 0, 2, 1, 3, that in which a word of packed codes unpacks into two
// pairs: for K over the head's values (Q is laid out alike), for V over the tokens (so S's columns,
// K's rows, are in that order too).
//
// Bound: a tile takes 3 + 3 products of 128 x 128 x hd.  1000 new rows beside 7 decodes over up to 4000 tokens, 32 heads on
// 8 kv heads of 128: 227 us; 4000 new rows of 8000 tokens: 1102 us, 357 TFLOP/s of the formula's or 1070 of the tensor
// cores', 57% of a large matrix product's rate.  The tensor pipe is busy 38% of the time at the first; the rest is waiting of
// a tile's stages for one another (softmax of 128 x 128, unpacking, putting O aside) and the start and end of items.
//
// Work is shared among the CTAs (one for each SM) as in attention_q4.cu.  Every wait is
// bounded; after one that runs out every role stops, copies and products in flight are waited
// for, and tensor memory is freed.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "mma_f16.cuh"
#include "paged_q4.cuh"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

constexpr int kRows = 128;  // query rows of an item
constexpr int kTile = 128;  // tokens of a tile
constexpr int kGroups = kTile / 16;
constexpr int kThreads = 640;
constexpr int kItemCost = 2;  // of an item's start and end, in tiles
constexpr float kLazy = 8.0f, kBias = 7.0f;
// Tiles that O sums before it starts again.  1000 new rows of a request holding 4096 (32 query heads, 8 of keys
// and values, of 128): never 204 us and off by 1.2e-5; 5 tiles 218 us and 2.8e-6; 3 tiles 224 us and 2.0e-6;
// 2 tiles 235 us and 1.6e-6.
constexpr int kPeriod = 3;
constexpr int kScaleTop = 8;  // the largest |d| of a tile becomes 2^8 .. 2^9

// Tensor memory columns: S three times (tile i in i mod 3), O.  P takes S's place: of every 32
// tokens, 16 columns of high pieces, then 16 of low ones.
constexpr uint32_t kColO = 256;
__device__ __forceinline__ uint32_t s_column(int third) { return third == 2 ? 384u : 128u * third; }

template <int NB>
struct Lay {
    static constexpr int hd = 32 * NB;
    static constexpr int q = kRows * hd * 2;        // one piece of Q (and of K)
    static constexpr int v = hd * kTile * 2;        // one piece of V
    static constexpr int raw_k = kGroups * 10 * hd; // K codes and scales, V scales
    static constexpr int raw_v = kGroups * 8 * hd;  // V codes
    static constexpr int off_q = 0, off_k = off_q + 2 * q, off_v = off_k + 2 * q;
    static constexpr int off_raw_k = off_v + 2 * v, off_raw_v = off_raw_k + 2 * raw_k;
    static constexpr int off_scale = off_raw_v + raw_v;                   // f16: K [128][NB], V of 3 tiles
    static constexpr int off_row = off_scale + 4 * kTile * NB * 2;        // the rows' maxima after even and odd tiles, sums, units of the workspace's sums
    static constexpr int off_misc = off_row + 5 * kRows * 4;
    static constexpr int bytes = off_misc + 512;
};

struct Bars {
    uint64_t raw_k_full[2], raw_k_empty[2], raw_v_full, raw_v_empty;
    uint64_t k_ready, scales_ready[3], v_ready, pv_done[2], s_full[3], p_ready[3], m_ready[2], q_ready, k_sync, out_sync, pair[4], done;
    uint32_t tmem;
    int gave_up, last;      // a wait ran out; this CTA adds the parts up
    int exps[4][2];         // of tiles i mod 4: K's and V's exponents
    uint32_t nan_v[4][4];   // of 32 tokens of theirs: byte e is the first with a V scale of block e that is no number (255: none)
    uint32_t warp_max[2][4];
    int parts, first_part;
};

__device__ __forceinline__ float ex2f(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// a * b - c
__device__ __forceinline__ uint32_t hfms2u(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("{\n\t.reg .b32 n;\n\tneg.f16x2 n, %3;\n\tfma.rn.f16x2 %0, %1, %2, n;\n\t}" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t codes_low(uint32_t w) { return hsub2u(lop_and_or(w, 0x000f000fu, 0x64006400u), 0x64086408u); }
__device__ __forceinline__ uint32_t codes_high(uint32_t w)
{
    return hfma2u(lop_and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
}
__device__ __forceinline__ float power2(int e) { return __int_as_float((127 + min(max(e, -126), 127)) << 23); }
// token of position p within 4: 0, 2, 1, 3 (its own inverse)
__device__ __forceinline__ int swapped(int p) { return (p & ~3) | ((p & 1) << 1) | ((p >> 1) & 1); }

// ---------------------------------------------------------------- tcgen05
// K-major operand of 16-bit values, core matrices 128 bytes apart along K, groups of 8 rows
// `stride` bytes apart, no swizzle
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t stride)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46);
}
__host__ __device__ constexpr uint32_t idesc_f16(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define RZ_O16(r)                                                                                                     \
    "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),      \
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
#define RZ_I16(r)                                                                                              \
    "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), \
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])

// 16 columns of the warp's 32 rows, waited for in the same statement
__device__ __forceinline__ void tm_load16(uint32_t at, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : RZ_O16(r)
        : "r"(at)
        : "memory");
}
// 32 columns
__device__ __forceinline__ void tm_load32(uint32_t at, float (&v)[32])
{
    uint32_t r[2][16];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : RZ_O16(r[k])
            : "r"(at + 16 * k)
            : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            asm volatile("" : "+r"(r[k][e]));  // not before the wait
            v[16 * k + e] = __uint_as_float(r[k][e]);
        }
}
__device__ __forceinline__ void tm_store16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::
            RZ_I16(r),
        "r"(at)
        : "memory");
}
__device__ __forceinline__ void tm_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- the line of work
struct Item {
    int row0, m, n;  // of the request: first row, rows, held tokens
    int s, h, it;
    int items;       // of a kv head
    int tokens, tiles, lo, hi;
    int64_t at;      // where the item begins on the line
};

__device__ __forceinline__ bool load_request(Item &w, const PagedAttnArgs &a, int group)
{
    const int c0 = a.cu_rows[w.s], c1 = a.cu_rows[w.s + 1], n = a.kv_len[w.s];
    const int64_t most = (int64_t)a.max_blocks << (a.kv.page_log + 4);
    const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.n_rows;  // what is not is reported by the other kernel
    w.row0 = ok ? c0 : 0;
    w.m = ok ? c1 - c0 : 0;
    w.n = n > most ? 0 : max(n, 0);
    const int rows = w.m * group;
    w.items = rows > kTcRows ? (rows + kRows - 1) / kRows : 0;
    return w.items > 0;
}
__device__ __forceinline__ int item_tokens(const Item &w, int group, int it)
{
    const unsigned last = static_cast<unsigned>(min((it + 1) * kRows, w.m * group) - 1) / static_cast<unsigned>(group);
    return max(w.n - w.m + static_cast<int>(last) + 1, 0);
}
__device__ __forceinline__ int64_t item_span(const Item &w, int group, int it)
{
    return kItemCost + (item_tokens(w, group, it) + kTile - 1) / kTile;
}

struct Line {
    int64_t total, step;
    int ctas, rest;
    __device__ __forceinline__ int64_t begin(int c) const
    {
        return c * step + static_cast<unsigned>(c * rest) / static_cast<unsigned>(ctas);
    }
};
__device__ __forceinline__ Line make_line(int64_t total, int grid)
{
    Line l;
    l.total = total;
    l.ctas = total < grid ? max(1, static_cast<int>(total)) : grid;
    l.step = total / l.ctas;
    l.rest = static_cast<int>(total - l.step * l.ctas);
    return l;
}
__device__ __forceinline__ int tile_at(int64_t x, int tiles)
{
    return x <= kItemCost ? 0 : x - kItemCost >= tiles ? tiles : static_cast<int>(x - kItemCost);
}
__device__ __forceinline__ void load_item(Item &w, const Line &l, int group)
{
    w.tokens = item_tokens(w, group, w.it);
    w.tiles = (w.tokens + kTile - 1) / kTile;
    w.lo = tile_at(l.begin(blockIdx.x) - w.at, w.tiles);
    w.hi = tile_at(l.begin(blockIdx.x + 1) - w.at, w.tiles);
}
__device__ __forceinline__ bool has_work(const Item &w, const Line &l)
{
    return w.lo < w.hi || (w.tiles == 0 && w.at >= l.begin(blockIdx.x));
}
__device__ __forceinline__ bool next_item(Item &w, const PagedAttnArgs &a, const Line &l, int group)
{
    w.at += item_span(w, group, w.it);
    if (w.at >= l.begin(blockIdx.x + 1)) return false;
    if (++w.it == w.items) {
        w.it = 0;
        if (++w.h == a.kv.n_kv_heads) {
            w.h = 0;
            do {
                if (++w.s >= a.n_seqs) return false;
            } while (!load_request(w, a, group));
        }
    }
    load_item(w, l, group);
    return true;
}

// Whether a phase is complete, at once (try_wait would sleep on one that is not).
__device__ __forceinline__ bool test_phase(uint64_t *bar, unsigned par)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(par)
        : "memory");
    return ok != 0;
}

// Warp-wide bounded wait; false after a timeout or when another role gave up.
__device__ __forceinline__ bool wait_for(uint64_t *bar, unsigned par, Bars &b, unsigned *err)
{
    bool ok = false;
    volatile int *gave_up = &b.gave_up;
    for (uint32_t i = 0; i < kWaitLimit / 8; ++i) {
        if (mbar_try_wait(bar, par)) {
            ok = true;
            break;
        }
        if ((i & 63u) == 63u && *gave_up) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && !*gave_up) {
        *gave_up = 1;
        set_error(err, DEV_TIMEOUT_PAGED);
    }
    return ok;
}

// A barrier of some warps at which none waits for ever; phase counts its uses.
__device__ __forceinline__ bool sync_warps(uint64_t *bar, unsigned &phase, Bars &b, unsigned *err)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    return wait_for(bar, phase++ & 1u, b, err);
}

// 32 values of one output row (a block) to the outputs.
__device__ __forceinline__ void write_block(const PagedAttnArgs &a, const float (&v)[32], int64_t row, int col, int q_dim, int q_pad)
{
    if (a.att) {
        float4 *o = reinterpret_cast<float4 *>(a.att + row * q_dim + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    if (a.att_q8) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(v[i]));
        const float d = __fdiv_rn(mx, 127.0f);
        const Q8Scale sc = q8_scale(d);
        int8_t *q = static_cast<int8_t *>(a.att_q8);
        float *qd = reinterpret_cast<float *>(q + a.n_rows * q_pad), *qs = qd + a.n_rows * (q_pad / 32);
        int sum = 0;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = q8_code(v[4 * i + k], sc);
                sum += c;
                w[i] |= static_cast<uint32_t>(c & 255) << (8 * k);
            }
        }
        uint4 *o = reinterpret_cast<uint4 *>(q + row * q_pad + col);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        qd[row * (q_pad / 32) + col / 32] = d;
        qs[row * (q_pad / 32) + col / 32] = __fmul_rn(d, (float)sum);
    }
}

template <int NB>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_tc_kernel(const __grid_constant__ PagedAttnArgs a)
{
    using L = Lay<NB>;
    constexpr int hd = L::hd;
    extern __shared__ __align__(1024) uint8_t sm[];
    Bars &b = *reinterpret_cast<Bars *>(sm + L::off_misc);
    static_assert(sizeof(Bars) <= 512, "");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = a.kv.n_kv_heads, group = a.n_heads / K;
    pdl_launch_dependents();
    pdl_wait();

    // ---- the line, and this CTA's first item on it
    Item first;
    Line line;
    {
        int64_t *pre = reinterpret_cast<int64_t *>(sm);  // before the operands; n_seqs + 1
        int64_t *tmp = pre + kPagedMaxSeqs + 8;
        const int per = (a.n_seqs + kThreads - 1) / kThreads;
        int64_t mine = 0;
        for (int i = tid * per; i < min(a.n_seqs, (tid + 1) * per); ++i) {
            Item w;
            w.s = i;
            int64_t span = 0;
            if (load_request(w, a, group))
                for (int it = 0; it < w.items; ++it) span += item_span(w, group, it);
            pre[i + 1] = span * K;
            mine += span * K;
        }
        int64_t v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) tmp[warp] = v;
        __syncthreads();
        for (int k = 0; k < warp; ++k) v += tmp[k];
        v -= mine;
        for (int i = tid * per; i < min(a.n_seqs, (tid + 1) * per); ++i) {
            v += pre[i + 1];
            pre[i + 1] = v;
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
        line = make_line(pre[a.n_seqs], gridDim.x);
        if (line.total == 0 || blockIdx.x >= line.ctas) return;  // the same for the whole CTA
        const int64_t x0 = line.begin(blockIdx.x);
        int lo = 0, hi = a.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= x0) lo = mid;
            else hi = mid;
        }
        first.s = lo;
        load_request(first, a, group);
        const int64_t head = (pre[lo + 1] - pre[lo]) / K;
        first.h = static_cast<int>((x0 - pre[lo]) / head);
        first.at = pre[lo] + first.h * head;
        first.it = 0;
        for (; first.it + 1 < first.items; ++first.it) {
            const int64_t span = item_span(first, group, first.it);
            if (first.at + span > x0) break;
            first.at += span;
        }
        load_item(first, line, group);
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.raw_k_full[i], 1);
            mbar_init(&b.raw_k_empty[i], 4);
            mbar_init(&b.m_ready[i], 4);
            mbar_init(&b.pv_done[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.p_ready[i], 4);
            mbar_init(&b.scales_ready[i], 4);
        }
        mbar_init(&b.raw_v_full, 1);
        mbar_init(&b.raw_v_empty, 4);
        mbar_init(&b.k_ready, 4);
        mbar_init(&b.v_ready, 4);
        mbar_init(&b.q_ready, 8);
        mbar_init(&b.k_sync, 4);
        mbar_init(&b.out_sync, 8);
        for (int i = 0; i < 4; ++i) mbar_init(&b.pair[i], 2);
        mbar_init(&b.done, 1);
        b.gave_up = b.last = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&b.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();  // pre is read, the barriers and tensor memory are there
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&b.tmem);
    Item w = first;
    bool more = true, ok = true;
    int i = 0;  // tiles of this CTA so far

    // Registers: launched with 96 a thread, 480 for the five warpgroups together: 80 for the first,
    // 120 each for the softmax warps', 80 each for those that unpack.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0) {
        // ------------------------------------------------------------ copies
        // K(i + 1) before V(i), the order in which they are unpacked
        const int lg = a.kv.page_log;
        constexpr int kRec = q4_record_bytes(hd);
        const int64_t head_bytes = (int64_t)kRec << lg;
        asm volatile("fence.proxy.async;" ::: "memory");
        const bool stalled = a.stall && blockIdx.x == 0;  // test aid: the first tile's K is not copied
        int n_k = 0, n_v = 0;
        const uint8_t *v_src = nullptr;  // this lane's group of the tile whose V is next
        int v_groups = 0;
        auto copy_v = [&]() {
            if (!wait_for(&b.raw_v_empty, (n_v & 1) ^ 1u, b, a.err)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&b.raw_v_full, v_groups * 8 * hd);
            __syncwarp();
            if (lane < v_groups) bulk_g2s(sm + L::off_raw_v + lane * 8 * hd, v_src + 9 * hd, 8 * hd, &b.raw_v_full);
            ++n_v;
            return true;
        };
        while (more && ok) {
            const int32_t *row = a.table + (int64_t)w.s * a.table_ld;
            for (int tile = w.lo; tile < w.hi; ++tile) {
                const int g0 = tile * kGroups, groups = min(kGroups, ((w.tokens + 15) >> 4) - g0);
                const uint8_t *src = nullptr;
                if (lane < groups) {
                    int32_t page = row[(g0 + lane) >> lg];
                    if (page < 0 || page >= a.kv.n_pages) {
                        set_error(a.err, DEV_BAD_PAGE);
                        page = 0;  // a page there is; the request's rows are not to be used
                    }
                    src = a.kv.pages + ((int64_t)page * K + w.h) * head_bytes + ((g0 + lane) & ((1 << lg) - 1)) * kRec;
                }
                const int slot = n_k & 1;
                if (!(ok = wait_for(&b.raw_k_empty[slot], ((n_k >> 1) & 1) ^ 1u, b, a.err))) break;
                const bool copy = !(stalled && n_k == 0);
                if (lane == 0 && copy) mbar_arrive_expect_tx(&b.raw_k_full[slot], groups * 10 * hd);
                __syncwarp();
                if (lane < groups && copy) {
                    uint8_t *dst = sm + L::off_raw_k + slot * L::raw_k + lane * 10 * hd;
                    bulk_g2s(dst, src, 9 * hd, &b.raw_k_full[slot]);
                    bulk_g2s(dst + 9 * hd, src + 17 * hd, hd, &b.raw_k_full[slot]);
                }
                ++n_k;
                if (n_k > 1 && !(ok = copy_v())) break;
                v_src = src;
                v_groups = groups;
            }
            if (ok) more = next_item(w, a, line, group);
        }
        if (ok && n_k > 0) copy_v();
        // no copy outlives the CTA
        for (int k = max(stalled ? 1 : 0, n_k - 2); k < n_k; ++k) mbar_wait(&b.raw_k_full[k & 1], (k >> 1) & 1);
        if (n_v > 0) mbar_wait(&b.raw_v_full, (n_v - 1) & 1);
        } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // descriptors of the first pieces; 16 values on are 256 bytes, 16 in a descriptor's unit
        constexpr uint32_t stride_q = hd * 16, stride_v = kTile * 16;  // 8 rows
        const uint64_t q0 = operand_desc(smem_u32(sm + L::off_q), stride_q), k0 = operand_desc(smem_u32(sm + L::off_k), stride_q),
                       v0 = operand_desc(smem_u32(sm + L::off_v), stride_v);
        int item = 0;
        // QK(j): A = Q, B = K; low * high, high * low, high * high.  One commit a product: a wait or a
        // commit costs this warp some hundred cycles.
        auto qk = [&](int j, int third) {
            if (lane == 0) {
                const uint32_t d = tmem + s_column(third);
#pragma unroll
                for (int p = 0; p < 3; ++p)
#pragma unroll
                    for (int k = 0; k < hd / 16; ++k)
                        mma_ss(d, q0 + (p == 0 ? L::q / 16 : 0) + 16 * k, k0 + (p == 1 ? L::q / 16 : 0) + 16 * k,
                               idesc_f16(kTile), p || k);
                commit(&b.s_full[third]);
            }
            __syncwarp();
        };
        // PV(j): A = P, B = V
        auto pv = [&](int j, int third, bool start) {
            if (lane == 0) {
                const uint32_t d = tmem + kColO, p0 = tmem + s_column(third);
#pragma unroll
                for (int p = 0; p < 3; ++p)
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ts(d, p0 + 32 * (k >> 1) + 8 * (k & 1) + (p == 1 ? 16 : 0), v0 + (p == 2 ? L::v / 16 : 0) + 16 * k,
                               idesc_f16(hd), !start || p || k);
                commit(&b.pv_done[j & 1]);
            }
            __syncwarp();
        };
        // Products in the order in which their operands are there: QK up to two tiles ahead of PV.
        //   QK(j): K(j) unpacked, and P(j - 3), in whose place S(j) goes, used up: PV(j - 3) done
        //   PV(j): P(j) and V(j) there, and PV(j - 2) known to be done (of each parity one is on its way)
        int j_qk = 0, j_pv = 0, done = 0;      // the next ones, and how many PV are done
        int third_qk = 0, third_pv = 0;        // j mod 3
        auto test = [&](uint64_t *bar, unsigned par) { return __all_sync(0xffffffffu, test_phase(bar, par)) != 0; };
        volatile int *gave_up = &b.gave_up;
        while (more && ok) {
            if (w.lo < w.hi) {
                ok = wait_for(&b.q_ready, item & 1, b, a.err);
                ++item;
                const int first_j = j_pv, last_j = j_pv + (w.hi - w.lo);
                uint32_t idle = 0;
                while (ok && j_pv < last_j) {
                    bool moved = false;
                    if (done < j_pv && test(&b.pv_done[done & 1], (done >> 1) & 1)) {
                        ++done;
                        moved = true;
                    }
                    if (j_pv < j_qk && done >= j_pv - 1 && test(&b.p_ready[third_pv], (j_pv / 3) & 1) && test(&b.v_ready, j_pv & 1)) {
                        fence_after();
                        pv(j_pv, third_pv, (j_pv - first_j) % kPeriod == 0);
                        ++j_pv;
                        third_pv = third_pv == 2 ? 0 : third_pv + 1;
                        moved = true;
                    }
                    if (j_qk < last_j && j_qk <= j_pv + 2 && done >= j_qk - 2 && test(&b.k_ready, j_qk & 1)) {
                        fence_after();
                        qk(j_qk, third_qk);
                        ++j_qk;
                        third_qk = third_qk == 2 ? 0 : third_qk + 1;
                        moved = true;
                    }
                    idle = moved ? 0 : idle + 1;
                    if (idle >= kWaitLimit * 4 || ((idle & 63u) == 63u && __any_sync(0xffffffffu, *gave_up))) {
                        if (!*gave_up) set_error(a.err, DEV_TIMEOUT_PAGED);
                        *gave_up = 1;
                        ok = false;
                    }
                }
            }
            if (ok) more = next_item(w, a, line, group);
        }
        // every product issued has completed once this arrives
        if (lane == 0) {
            commit(&b.done);
            mbar_wait(&b.done, 0);
        }
        __syncwarp();
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ unpacking
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const bool for_v = warp >= 16;
        const int tok128 = (tid - 384) & 127, w4 = warp & 3, g = lane >> 2, t = lane & 3;
        uint16_t *sk = reinterpret_cast<uint16_t *>(sm + L::off_scale), *sv = sk + kTile * NB;
        unsigned phase = 0;
        // two words' codes c0, c1 times their scales, high and low piece, to 8 bytes of a chunk
        auto put = [&](uint8_t *p, int piece, uint32_t c0, uint32_t c1, uint32_t d0, uint32_t d1) {
            const uint32_t h0 = hmul2u(c0, d0), h1 = hmul2u(c1, d1);
            *reinterpret_cast<uint2 *>(p) = make_uint2(h0, h1);
            *reinterpret_cast<uint2 *>(p + piece) = make_uint2(hfms2u(c0, d0, h0), hfms2u(c1, d1, h1));
        };
        // The scales of tile j, a token a thread, times 2^up: the tile's largest of K and of V to
        // 2^8 .. 2^9.  A tile without a value but zeros counts as one of the smallest f16: its exponent enters the rows'
        // maxima, and may not lift them over those of tiles that have values.  V's last for 3 tiles: K(j) is copied after
        // V(j - 2), which is once V(j - 3) is unpacked.
        auto scales = [&](int j, int valid) {
            if (!wait_for(&b.raw_k_full[j & 1], (j >> 1) & 1, b, a.err)) return false;
            const uint8_t *raw = sm + L::off_raw_k + (j & 1) * L::raw_k + (tok128 >> 4) * 10 * hd + 8 * hd;
            uint16_t d[2][NB];
            uint32_t most[2] = {0, 0}, firsts = 0xffffffffu;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint16_t *src = reinterpret_cast<const uint16_t *>(raw + v * hd) + (tok128 & 15) * NB;
#pragma unroll
                for (int e = 0; e < NB; ++e) {
                    d[v][e] = tok128 < valid ? src[e] : uint16_t(0);
                    const uint32_t abs = d[v][e] & 0x7fffu;
                    if (abs < 0x7c00u) most[v] = max(most[v], abs);
                    if (v) {
                        const unsigned bads = __ballot_sync(0xffffffffu, abs >= 0x7c00u);
                        if (bads) firsts = (firsts & ~(255u << (8 * e))) | (uint32_t)(__ffs(bads) - 1) << (8 * e);
                    }
                }
                most[v] = __reduce_max_sync(0xffffffffu, most[v]);
            }
            if (lane == 0) {
                b.warp_max[0][w4] = most[0];
                b.warp_max[1][w4] = most[1];
                b.nan_v[j & 3][w4] = firsts;
            }
            if (!sync_warps(&b.k_sync, phase, b, a.err)) return false;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint32_t top = max(max(b.warp_max[v][0], b.warp_max[v][1]), max(b.warp_max[v][2], b.warp_max[v][3]));
                const int up = kScaleTop + 127 - (__float_as_int(h2f((uint16_t)max(top, 1u))) >> 23);
                if (tok128 == 0) b.exps[j & 3][v] = up;
                uint16_t *dst = (v ? sv + (j % 3) * kTile * NB : sk) + tok128 * NB;
#pragma unroll
                for (int e = 0; e < NB; ++e) {
                    // a V scale that is no number: nothing is added, and the block's values of the rows that see it are made NaN
                    const bool drop = v && (d[v][e] & 0x7fffu) >= 0x7c00u;
                    dst[e] = drop ? uint16_t(0) : __half_as_ushort(__float2half_rn(h2f(d[v][e]) * power2(up)));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.scales_ready[j % 3]);
            return sync_warps(&b.k_sync, phase, b, a.err);
        };
        auto unpack_k = [&](int j) {
            const uint8_t *raw = sm + L::off_raw_k + (j & 1) * L::raw_k;
            // the operand is free once QK(j - 1) is done
            if (j > 0 && !wait_for(&b.s_full[(j - 1) % 3], ((j - 1) / 3) & 1, b, a.err)) return false;
            // groups 2 w4, 2 w4 + 1; lane (g, t): word t of each block of rows 8 hf + g
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const int gr = 2 * w4 + (k >> 1), hf = k & 1, tok = swapped(8 * hf + g);
                const uint32_t *r = reinterpret_cast<const uint32_t *>(raw + gr * 10 * hd + tok * (hd / 2) + t * 4 * NB);
                uint32_t x[NB], s2[NB / 2];
                if constexpr (NB == 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(r);
                    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                    const uint2 d = *reinterpret_cast<const uint2 *>(sk + (gr * 16 + tok) * NB);
                    s2[0] = d.x, s2[1] = d.y;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(r);
                    x[0] = v.x, x[1] = v.y;
                    s2[0] = *reinterpret_cast<const uint32_t *>(sk + (gr * 16 + tok) * NB);
                }
                uint8_t *dst = sm + L::off_k + (2 * gr + hf) * (hd * 16) + g * 16 + (t >> 1) * 128 + (t & 1) * 8;
#pragma unroll
                for (int e = 0; e < NB; ++e) {
                    const uint32_t y = x[e] >> 8, d = __byte_perm(s2[e >> 1], 0, (e & 1) ? 0x3232 : 0x1010);
                    put(dst + e * 512, L::q, codes_low(x[e]), codes_low(y), d, d);
                    put(dst + e * 512 + 256, L::q, codes_high(x[e]), codes_high(y), d, d);
                }
            }
            return true;
        };
        auto unpack_v = [&](int j) {
            if (!wait_for(&b.raw_v_full, j & 1, b, a.err) || !wait_for(&b.scales_ready[j % 3], (j / 3) & 1, b, a.err)) return false;
            // the operand is free once PV(j - 1) is done
            if (j > 0 && !wait_for(&b.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, b, a.err)) return false;
#pragma unroll 1
            for (int gr = 2 * w4; gr < 2 * w4 + 2; ++gr) {
                // scales of tokens 4 t .. 4 t + 3: half i * NB + e
                uint32_t d[2 * NB];
                const uint4 *dp = reinterpret_cast<const uint4 *>(sv + (j % 3) * kTile * NB + (gr * 16 + 4 * t) * NB);
#pragma unroll
                for (int k = 0; k < NB / 2; ++k) {
                    const uint4 v = dp[k];
                    d[4 * k] = v.x, d[4 * k + 1] = v.y, d[4 * k + 2] = v.z, d[4 * k + 3] = v.w;
                }
                constexpr int run = q4_v_run(NB);
                const uint8_t *raw = sm + L::off_raw_v + gr * 8 * hd + lane * run * 4;
                uint8_t *dst = sm + L::off_v + g * 16 + (2 * gr + (t >> 1)) * 128 + (t & 1) * 8;
#pragma unroll
                for (int q = 0; q < 2 * NB / run; ++q) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(raw + q * 32 * run * 4);
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 4 * q + k, e = r >> 1;
                        const uint32_t sel = (e & 1) ? 0x7632 : 0x5410;
                        const uint32_t d0 = __byte_perm(d[e / 2], d[(2 * NB + e) / 2], sel), d1 = __byte_perm(d[(NB + e) / 2], d[(3 * NB + e) / 2], sel);
                        // rows (values) 32 e + 8 (r % 2) + g and 16 more; columns 16 gr + 4 t ..
                        uint8_t *p = dst + (4 * e + (r & 1)) * (kTile * 16);
                        put(p, L::v, codes_low(x[k]), codes_low(x[k] >> 8), d0, d1);
                        put(p + 2 * (kTile * 16), L::v, codes_high(x[k]), codes_high(x[k] >> 8), d0, d1);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&b.v_ready);
                mbar_arrive(&b.raw_v_empty);
            }
            return true;
        };
        while (more && ok) {
            for (int tile = w.lo; tile < w.hi && ok; ++tile, ++i) {
                if (for_v) {
                    ok = unpack_v(i);
                    continue;
                }
                if (!(ok = scales(i, w.tokens - tile * kTile)) || !(ok = unpack_k(i))) break;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&b.k_ready);
                    mbar_arrive(&b.raw_k_empty[i & 1]);
                }
            }
            if (ok) more = next_item(w, a, line, group);
        }
    } else {
        // ------------------------------------------------------------ softmax and outputs
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        const int half = (warp - 4) >> 2, r = (tid - 128) & 127;  // this thread's tiles (and values of the output), its row
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int q_dim = a.n_heads * hd, q_pad = (q_dim + 255) / 256 * 256;
        volatile float *maxima = reinterpret_cast<float *>(sm + L::off_row) + r;
        // this row's sums of the periods before: 4 values of all rows after another
        float *kept = a.kept + (int64_t)blockIdx.x * kRows * hd + 4 * r;
        // what the row's other thread gives for v, and both threads' bits (in the place of the maximum of the tile before
        // the last, which both have done with)
        unsigned pair_phase = 0;
        auto exchange = [&](float v, float &got, unsigned &bits) {
            volatile float *at = maxima + 2 * kRows;
            volatile uint16_t *two = reinterpret_cast<volatile uint16_t *>(maxima + (i & 1) * kRows);
            at[half * kRows] = v;
            two[half] = static_cast<uint16_t>(bits);
            bool fine = sync_warps(&b.pair[warp & 3], pair_phase, b, a.err);
            got = at[(half ^ 1) * kRows];
            bits |= two[half ^ 1];
            return sync_warps(&b.pair[warp & 3], pair_phase, b, a.err) && fine;  // read, before it is written again
        };
        unsigned phase = 0;
        int third = 0;  // i mod 3
        while (more && ok) {
            if (!has_work(w, line)) {
                more = next_item(w, a, line, group);
                continue;
            }
            const int n_rows = w.m * group, my = w.it * kRows + r;
            const bool live = my < n_rows;
            const int tok_q = min(my, n_rows - 1) / group;
            const int before = w.n - w.m + 1;
            const int sees = max(before + tok_q, 0), all_see = max(before + (w.it * kRows + (r & ~31)) / group, 0);
            const int64_t row = w.row0 + tok_q;
            const int col0 = (w.h * group + (min(my, n_rows - 1) - tok_q * group)) * hd;
            float unit = 0.0f, m = -1e37f, l = 0.0f;
            unsigned nan_blocks = 0;  // the blocks of this row's values that are NaN
            if (w.lo < w.hi) {
                // ---- Q's pieces (both threads look for the largest, each writes half; plain loads, as in attention_q4.cu).  The products of the
                // item before that read them are done: their S was waited for.
                const float4 *src = reinterpret_cast<const float4 *>(a.q + row * a.ld_q + col0);
                float mx = 0.0f;
#pragma unroll 8
                for (int k = 0; k < hd / 4; ++k) {
                    const float4 v = src[k];
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
                }
                const int up = mx == 0.0f || !live ? 0 : min(14 - ((__float_as_int(mx) >> 23) - 127), 126);
                const float sc = live ? power2(up) : 0.0f;
                unit = a.scale * 1.4426950408889634f * power2(-up);
                uint8_t *dst = sm + L::off_q + (r >> 3) * (hd * 16) + (r & 7) * 16;
#pragma unroll 4
                for (int k = half * (hd / 16); k < (half + 1) * (hd / 16); ++k) {
                    const float4 x = src[2 * k], y = src[2 * k + 1];
                    const float f[8] = {x.x, x.z, x.y, x.w, y.x, y.z, y.y, y.w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = live ? f[2 * e] * sc : 0.0f, q = live ? f[2 * e + 1] * sc : 0.0f;
                        hi[e] = pack2(p, q);
                        const float2 h = unpack2(hi[e]);
                        lo[e] = pack2(p - h.x, q - h.y);
                    }
                    *reinterpret_cast<uint4 *>(dst + k * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(dst + L::q + k * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.q_ready);
            }
            for (int tile = w.lo; tile < w.hi; ++tile, ++i, third = third == 2 ? 0 : third + 1) {
                if ((i & 1) != half) continue;
                if (!(ok = wait_for(&b.s_full[third], (i / 3) & 1, b, a.err))) break;
                fence_after();
                // blocks of which this row sees a V scale that is no number
                if ((b.nan_v[i & 3][0] & b.nan_v[i & 3][1] & b.nan_v[i & 3][2] & b.nan_v[i & 3][3]) != 0xffffffffu) {
#pragma unroll 1
                    for (int c = 0; c < 4 * NB; ++c) {
                        const int tok = b.nan_v[i & 3][c / NB] >> (8 * (c % NB)) & 255;
                        if (tok < 32 && 32 * (c / NB) + tok < sees - tile * kTile) nan_blocks |= 1u << (c % NB);
                    }
                }
                // (u of a normal f32 at least: a masked score, -infinity, times 0 would be NaN)
                const float u = fmaxf(unit * power2(-b.exps[i & 3][0]), 0x1p-126f), sub = static_cast<float>(-b.exps[i & 3][1]);
                // The scores are read twice, 32 at a time in loops that are not unrolled, and not kept: code for
                // all values at once, of 8 warps beside 8 others with code of their own, waits for its instructions.
                const uint32_t at = tmem + lanes + s_column(third);
                const int left = sees - tile * kTile;
                const bool masked = (tile + 1) * kTile > all_see;  // the same for the warp
                float top = -INFINITY, top2 = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < kTile; c += 32) {
                    float s[32];
                    tm_load32(at + c, s);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c + ((e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1)) >= left) s[e] = -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        top = fmaxf(top, s[e]);
                        top2 = fmaxf(top2, s[e + 1]);
                    }
                }
                top = fmaf(fmaxf(top, top2), u, sub);  // log2 of the largest weight of V as it is unpacked
                // the running maximum of the tile before, this one's for the next
                float before_m = -1e37f;
                if (tile > w.lo) {
                    if (!(ok = wait_for(&b.m_ready[(i - 1) & 1], ((i - 1) >> 1) & 1, b, a.err))) break;
                    before_m = maxima[((i - 1) & 1) * kRows];
                }
                const bool grown = top > before_m + kLazy;
                const float m_new = grown ? top : before_m;
                maxima[(i & 1) * kRows] = m_new;
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.m_ready[i & 1]);
                l *= ex2f(m - m_new);
                m = m_new;
                const bool again = tile > w.lo && (tile - w.lo) % kPeriod == 0;  // O starts again with this tile
                if (again) {
                    // its sums so far (in the unit of the maximum before) to the workspace
                    if (!(ok = wait_for(&b.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, b, a.err))) break;
                    fence_after();
                    const bool first = tile - w.lo == kPeriod;
                    float ref = first ? before_m : maxima[4 * kRows];
                    if (before_m - ref > 60.0f) {  // f32's range is not to be left
                        const float f = ex2f(ref - before_m);
#pragma unroll 1
                        for (int c = 0; c < hd / 4; ++c) {
                            float4 *p = reinterpret_cast<float4 *>(kept) + c * kRows;
                            const float4 x = __ldcg(p);
                            *p = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
                        }
                        ref = before_m;
                    }
                    maxima[4 * kRows] = ref;
                    const float f = ex2f(before_m - ref);
#pragma unroll 1
                    for (int c = 0; c < hd; c += 32) {
                        float o[32];
                        tm_load32(tmem + lanes + kColO + c, o);
                        float *p = kept + (c / 4 * kRows) * 4;
#pragma unroll
                        for (int e = 0; e < 32; e += 4, p += kRows * 4) {
                            if (first) *reinterpret_cast<float4 *>(p) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                            else
                                asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(o[e] * f),
                                             "f"(o[e + 1] * f), "f"(o[e + 2] * f), "f"(o[e + 3] * f)
                                             : "memory");
                        }
                    }
                    fence_before();
                } else if (tile > w.lo && __any_sync(0xffffffffu, grown)) {
                    // O is at rest once the tile before is done
                    if (!(ok = wait_for(&b.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, b, a.err))) break;
                    fence_after();
                    const float f = ex2f(before_m - m);
#pragma unroll 1
                    for (int c = 0; c < hd; c += 16) {
                        uint32_t o[16];
                        tm_load16(tmem + lanes + kColO + c, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tm_store16(tmem + lanes + kColO + c, o);
                    }
                }
                const float off = sub + (kBias - m);
                float sum = 0.0f, sum2 = 0.0f;
#pragma unroll 1
                for (int c = 0; c < kTile; c += 32) {
                    float s[32];
                    tm_load32(at + c, s);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c + ((e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1)) >= left) s[e] = -INFINITY;
                    }
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p = ex2f(fmaf(s[2 * e], u, off)), q = ex2f(fmaf(s[2 * e + 1], u, off));
                        sum += p;
                        sum2 += q;
                        hi[e] = pack2(p, q);
                        const float2 h = unpack2(hi[e]);
                        lo[e] = pack2(p - h.x, q - h.y);
                    }
                    tm_store16(at + c, hi);  // in the place of the scores that were read
                    tm_store16(at + c + 16, lo);
                }
                l = fmaf(sum + sum2, power2(b.exps[i & 3][1]), l);
                tm_store_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_ready[third]);
            }
            if (!ok) break;
            // ---- the row's sum is that of its two threads, at the last tile's maximum; each writes half of its values
            if (w.lo < w.hi) {
                if (!(ok = wait_for(&b.m_ready[(i - 1) & 1], ((i - 1) >> 1) & 1, b, a.err))) break;
                const float last_m = maxima[((i - 1) & 1) * kRows];
                l *= ex2f(m - last_m);
                m = last_m;
            }
            float l2;
            if (!(ok = exchange(l, l2, nan_blocks))) break;
            const bool more_sums = w.hi - w.lo > kPeriod;
            const float kept_ref = more_sums ? maxima[4 * kRows] : -INFINITY;
            const float kept_f = kept_ref == -INFINITY ? 0.0f : ex2f(kept_ref - m);
            if (more_sums) __threadfence();  // the other thread's adds are past, too
            l = half ? l2 + l : l + l2;
            if (w.lo < w.hi) {
                if (!(ok = wait_for(&b.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, b, a.err))) break;
                fence_after();
            }
            const bool whole = w.lo == 0 && w.hi == w.tiles;
            float *part = a.part + (2 * (int64_t)blockIdx.x + (w.lo == 0)) * (kRows * (hd + 2));
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
            for (int c = half * (hd / 2); c < (half + 1) * (hd / 2); c += 32) {
                float v[32];
                if (w.lo < w.hi) {
                    uint32_t o[16];
                    tm_load16(tmem + lanes + kColO + c, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]);
                    tm_load16(tmem + lanes + kColO + c + 16, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[16 + e] = __uint_as_float(o[e]);
                    if (more_sums) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 x = __ldcg(reinterpret_cast<const float4 *>(kept + ((c + e) / 4 * kRows) * 4));
                            v[e] = fmaf(x.x, kept_f, v[e]);
                            v[e + 1] = fmaf(x.y, kept_f, v[e + 1]);
                            v[e + 2] = fmaf(x.z, kept_f, v[e + 2]);
                            v[e + 3] = fmaf(x.w, kept_f, v[e + 3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                }
                if (nan_blocks >> (c >> 5) & 1) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __int_as_float(0x7fffffff);
                }
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = l == 0.0f ? 0.0f : v[e] * inv;
                    if (live) write_block(a, v, row, col0 + c, q_dim, q_pad);
                } else if (live) {
                    float4 *o = reinterpret_cast<float4 *>(part + r * hd + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
            }
            if (!whole) {
                if (live && half == 0) *reinterpret_cast<float2 *>(part + kRows * hd + 2 * r) = make_float2(m, l);
                // the CTAs with a part of the item, in order: CTA c0 has the first, the parts follow one another
                if (tid == 128) {
                    int c = static_cast<int>(min(w.at / max(line.step, (int64_t)1), (int64_t)line.ctas - 1));
                    while (line.begin(c) > w.at) --c;
                    while (tile_at(line.begin(c + 1) - w.at, w.tiles) == 0) ++c;
                    int n = 0;
                    for (int k = c; k < line.ctas && tile_at(line.begin(k) - w.at, w.tiles) < w.tiles; ++k) ++n;
                    b.first_part = c;
                    b.parts = n;
                }
                __threadfence();
                if (!(ok = sync_warps(&b.out_sync, phase, b, a.err))) break;
                if (tid == 128) {
                    int *counter = a.counters + b.first_part;
                    const int arrived = atomicAdd(counter, 1);
                    b.last = arrived == b.parts - 1;
                    if (b.last) *counter = 0;
                }
                if (!(ok = sync_warps(&b.out_sync, phase, b, a.err))) break;
                if (b.last) {
                    __threadfence();
                    const int c0 = b.first_part, n = b.parts;
                    if (live) {
                        const int64_t size = kRows * (hd + 2);
                        auto part_of = [&](int k) {
                            return a.part + (2 * (int64_t)(c0 + k) + (tile_at(line.begin(c0 + k) - w.at, w.tiles) == 0)) * size;
                        };
                        float mm = -1e37f, ll = 0.0f;
                        for (int k = 0; k < n; ++k) mm = fmaxf(mm, __ldcg(part_of(k) + kRows * hd + 2 * r));
                        for (int k = 0; k < n; ++k) {
                            const float2 x = __ldcg(reinterpret_cast<const float2 *>(part_of(k) + kRows * hd + 2 * r));
                            ll = fmaf(x.y, ex2f(x.x - mm), ll);
                        }
                        const float iv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll 1
                        for (int c = half * (hd / 2); c < (half + 1) * (hd / 2); c += 32) {
                            float v[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                            for (int k = 0; k < n; ++k) {
                                const float *p = part_of(k);
                                const float f = ex2f(__ldcg(p + kRows * hd + 2 * r) - mm) * iv;
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(p + r * hd + c) + e);
                                    v[4 * e] = fmaf(x.x, f, v[4 * e]);
                                    v[4 * e + 1] = fmaf(x.y, f, v[4 * e + 1]);
                                    v[4 * e + 2] = fmaf(x.z, f, v[4 * e + 2]);
                                    v[4 * e + 3] = fmaf(x.w, f, v[4 * e + 3]);
                                }
                            }
                            write_block(a, v, row, col0 + c, q_dim, q_pad);
                        }
                    }
                }
                if (!(ok = sync_warps(&b.out_sync, phase, b, a.err))) break;  // first_part, parts and last are read
            }
            // the zero padding of the Q8_1 rows, with kv head 0 and its first query head
            if (a.att_q8 && w.h == 0 && w.lo == 0 && live && half == 0 && col0 == 0) {
                int8_t *q8 = static_cast<int8_t *>(a.att_q8);
                float *qd = reinterpret_cast<float *>(q8 + a.n_rows * q_pad), *qs = qd + a.n_rows * (q_pad / 32);
                for (int c = q_dim; c < q_pad; c += 32) {
                    uint4 *o = reinterpret_cast<uint4 *>(q8 + row * q_pad + c);
                    o[0] = o[1] = make_uint4(0u, 0u, 0u, 0u);
                    qd[row * (q_pad / 32) + c / 32] = 0.0f;
                    qs[row * (q_pad / 32) + c / 32] = 0.0f;
                }
            }
            // O is read: the next item's first product may overwrite it (p_ready orders it)
            fence_before();
            more = next_item(w, a, line, group);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int NB>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t s)
{
    using L = Lay<NB>;
    static_assert(L::bytes <= 227 * 1024, "");
    static std::atomic<uint64_t> done{0};  // devices on which the kernel may have that much
    const uint64_t bit = 1ull << (dev_info().device & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(paged_attention_tc_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)dev_info().sm_count);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, paged_attention_tc_kernel<NB>, a);
}

}  // namespace

// two partial records for each CTA, then its sums of earlier periods
size_t paged_attention_tc_part_bytes(int head_dim)
{
    return (size_t)dev_info().sm_count * kRows * (2 * (head_dim + 2) + head_dim) * 4;
}

bool paged_attention_tc_takes(int head_dim) { return head_dim == 64 || head_dim == 128; }

cudaError_t launch_paged_attention_tc(const PagedAttnArgs &args, cudaStream_t s)
{
    PagedAttnArgs a = args;
    a.kept = a.part + (size_t)dev_info().sm_count * kRows * 2 * (a.kv.head_dim + 2);
    return a.kv.head_dim == 64 ? launch<2>(a, s) : launch<4>(a, s);
}

}  // namespace rz
