// attention_q4.cu -- attention of each request's new tokens over its pages of the
// 4-bit KV cache, read as they are held.
//
//   row i of a request with m new rows and n held tokens sees tokens j < n - m + i + 1:
//   att = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q . k_j - max)
//   k_j = d_jb (code - 8) for each block b of 32 values, v_j alike; a row that sees
//   nothing comes out as zeros.
//
// Products.  m16n8k16, the tokens in the rows and the queries in the columns: for the
// scores A holds 16 tokens' codes and B the queries, for the sums A holds 16 values' codes of 16
// tokens and B the weights.  So each code is unpacked once for all of a warp's
// queries.  Codes become f16 integers -8..7, exactly: a nibble ORed into the low bits of
// 1024 is 1024 + code (high nibbles: 1024 + 16 code), and one packed subtraction or
// multiply-add takes the rest off, two codes at a time.  (A code left in the low bits alone
// is a subnormal, exact too and without the subtraction, but the tensor cores align a
// product by its operands' exponents and not by its size: sums came out at 2^-17.)  q and the
// weights p * d of V are two f16 pieces each (22 bits) in neighbouring columns, 4 queries to a
// product, so that a thread finds both halves of its query's sum in one register pair and adds them;
// sums are f32.  q is scaled by a power of two for each row (exact) so that its pieces
// fill f16's range.  The weights come out of the scores' layout with a lane for a token and have to
// go into B's with a lane for a query: one movmatrix for 8 tokens and a block.
//
// Softmax.  The running maximum M of a row is one of log2(p) + log2 |d of V|, so that the
// weights p * d that are split stay within f16 (2^7 near the maximum, up to 2^15)
// whatever the values' scale; the sums are rescaled when a weight would
// leave that range, by 2^8 over the maximum, and not before.
//
// Work.  An item is (request, kv head, up to 8 W query rows: token-major, the group's
// heads within a token); it reads units of 32 tokens.  All items' units, weighted by
// their cost, are one line that the CTAs (two for each SM) share evenly, so that one long
// request or many ragged ones load all SMs alike; a CTA whose share ends within an item
// leaves its sums in the workspace and the CTA that finishes last adds them up, in the order of
// the units (the result does not depend on which one it is).  Of a CTA's W consumer
// warps, W / (row groups of 8) work a row group, each its own units; with up to 4 rows
// a warp works both groups of 16 tokens of a unit at once.  A producer warp copies units into a ring
// of slots with the bulk-copy engine, a lane for a unit.
//
// Bound: the instructions of a unit and how few warps there are to hide their latency; no pipe is full.  32 tokens of a
// head of 128 take a warp some 700: 288 unpack codes, 112 split the weights, 32 are products, 48 scale scores; 12 warps an SM
// (168 registers a thread) fill 53% of the issue slots, 43% of the ALU's and 20% of the tensor cores'.  64 requests of 8192
// tokens, 32 heads on 8 kv heads of 128: 141 us, 4.3 TB/s of the cache as it is held or 63% of a copy's rate; of 1000 to
// 16384 tokens 116 us, 56%.  1 request of 1000 tokens: 10.5 us, of which 4 join the parts.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "mma_f16.cuh"
#include "paged_q4.cuh"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

// Consumer warps W of a CTA, two CTAs on an SM: 5 and a producer are 3 warps a scheduler, 168
// registers a thread (7, with 128 registers: 64 requests of 16384 tokens take 130 us instead
// of 122, a chunk of 1000 rows 849 instead of 699); heads of over 128 values need 255, and 3 and
// a producer.
__host__ __device__ constexpr int consumers(int nb) { return nb <= 4 ? 5 : 3; }
constexpr int kPad = 8;     // floats after a row of sums: its 4 rows fall into other banks
constexpr int kUnit = 32;    // tokens of a unit
constexpr int kFlush = 32;  // groups of 16 tokens summed in the tensor cores' accumulators at a time
constexpr float kLazy = 8.0f;  // weights may grow by 2^8 over the running maximum
constexpr float kBias = 7.0f;  // log2 of a weight p * |d| at the running maximum

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ int add_acq_rel(int *p, int v)
{
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

template <int W>
__device__ __forceinline__ void consumer_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
}

// Codes - 8 of a word's nibbles 0 and 4 (low) or 1 and 5 (high), as two f16.
__device__ __forceinline__ uint32_t low_codes(uint32_t w)
{
    return hsub2u(lop_and_or(w, 0x000f000fu, 0x64006400u), 0x64086408u);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w)
{
    return hfma2u(lop_and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);  // / 16 - 72
}

// ---------------------------------------------------------------- the line of work
struct Seq {
    int row0, m, n;  // first row, rows, held tokens
    int rg;          // query row groups of 8 in an item
    int items;       // items of one kv head
};

// Row groups of an item: as few as hold the request's rows, else one for each warp.
template <int W>
__device__ __forceinline__ int row_groups(int rows)
{
    return rows <= 8 ? 1 : rows <= 16 && W > 3 ? 2 : W;
}

// What shared memory holds of a request: first row, rows, held tokens (checked).
struct SeqRow {
    int row0, m, n;
};

__device__ __forceinline__ SeqRow read_seq(const PagedAttnArgs &a, int s, bool &bad)
{
    const int c0 = a.cu_rows[s], c1 = a.cu_rows[s + 1], n = a.kv_len[s];
    const int64_t most = (int64_t)a.max_blocks << (a.kv.page_log + 4);
    const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.n_rows;
    if (!ok || n < 0 || n > most) bad = true;
    // one with many rows has none here: attention_q4_tc.cu works it
    const bool here = ok && (c1 - c0) * (a.n_heads / a.kv.n_kv_heads) <= a.most_rows;
    return SeqRow{here ? c0 : 0, here ? c1 - c0 : 0, n > most ? 0 : max(n, 0)};
}

template <int W>
__device__ __forceinline__ Seq make_seq(const SeqRow &r, int group)
{
    Seq q;
    q.row0 = r.row0;
    q.m = r.m;
    q.n = r.n;
    const int rows = q.m * group;
    q.rg = row_groups<W>(rows);
    q.items = (rows + 8 * q.rg - 1) / (8 * q.rg);
    return q;
}

// Tokens that item it of a request sees (its last row's).
__device__ __forceinline__ int item_tokens(const Seq &q, int group, int it)
{
    const unsigned last = static_cast<unsigned>(min((it + 1) * 8 * q.rg, q.m * group) - 1) / static_cast<unsigned>(group);
    return max(q.n - q.m + static_cast<int>(last) + 1, 0);
}
__device__ __forceinline__ int item_units(const Seq &q, int group, int it)
{
    return (item_tokens(q, group, it) + kUnit - 1) / kUnit;
}
// Cost of a unit, which one of W / rg warps works while the others work the next ones; of
// an item's start and end; and of what a CTA is worth starting for (a unit for each warp).
template <int W>
__device__ __forceinline__ int unit_cost(int rg)
{
    return 2 * W / (W / rg);
}
template <int W>
constexpr int kItemCost = 4 * W;
template <int W>
constexpr int kShare = 2 * W;

// The line, shared by as many CTAs as are worth starting: CTA c's share begins at
// c * step + c * rest / ctas.
struct Line {
    int64_t total, step;
    int ctas, rest;
    __device__ __forceinline__ int64_t begin(int c) const
    {
        return c * step + static_cast<unsigned>(c * rest) / static_cast<unsigned>(ctas);
    }
};
template <int W>
__device__ __forceinline__ Line make_line(int64_t total, int grid)
{
    Line l;
    l.total = total;
    l.ctas = total < kShare<W> * (int64_t)grid ? max(1, static_cast<int>(total) / kShare<W>) : grid;
    l.step = total < (1ll << 31) ? static_cast<unsigned>(total) / static_cast<unsigned>(l.ctas) : total / l.ctas;
    l.rest = static_cast<int>(total - l.step * l.ctas);
    return l;
}

// The parts of items that one CTA works, in order.  Every warp walks its own copy.
struct Walk {
    int64_t x0, x1;  // this CTA's share of the line
    int64_t at;      // where the current item begins
    Seq q;
    int s, h, it;
    int tokens, units, lo, hi;  // the current item's tokens and units, the part [lo, hi) of them
};

template <int W>
__device__ __forceinline__ int64_t item_span(const Seq &q, int group, int it)
{
    return kItemCost<W> + (int64_t)item_units(q, group, it) * unit_cost<W>(q.rg);
}
// The first unit at or after offset x of an item (kItemCost, then units).
template <int W>
__device__ __forceinline__ int unit_at(int64_t x, int units, int cost)
{
    if (x <= kItemCost<W>) return 0;
    if (x >= kItemCost<W> + (int64_t)units * cost) return units;
    return static_cast<unsigned>(x - kItemCost<W> + cost - 1) / static_cast<unsigned>(cost);
}

template <int W>
__device__ __forceinline__ void load_item(Walk &w, const PagedAttnArgs &a, int group)
{
    w.tokens = item_tokens(w.q, group, w.it);
    w.units = (w.tokens + kUnit - 1) / kUnit;
    const int cost = unit_cost<W>(w.q.rg);
    w.lo = unit_at<W>(w.x0 - w.at, w.units, cost);
    w.hi = unit_at<W>(w.x1 - w.at, w.units, cost);
}

// To the first item of the share.  pre[s]: the line before request s.
template <int W>
__device__ __forceinline__ bool walk_begin(Walk &w, const PagedAttnArgs &a, const Line &line, const int64_t *pre, const SeqRow *seqs,
                                           int group)
{
    if (line.total == 0 || blockIdx.x >= line.ctas) return false;
    w.x0 = line.begin(blockIdx.x);
    w.x1 = line.begin(blockIdx.x + 1);
    if (w.x0 >= w.x1) return false;
    int lo = 0, hi = a.n_seqs;  // pre[lo] <= x0 < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= w.x0) lo = mid;
        else hi = mid;
    }
    w.s = lo;
    w.q = make_seq<W>(seqs[w.s], group);
    const int64_t span = pre[lo + 1] - pre[lo], in = w.x0 - pre[lo];
    int64_t head;
    if (span < (1ll << 31)) {
        head = static_cast<unsigned>(span) / static_cast<unsigned>(a.kv.n_kv_heads);
        w.h = static_cast<unsigned>(in) / static_cast<unsigned>(head);
    } else {
        head = span / a.kv.n_kv_heads;
        w.h = static_cast<int>(in / head);
    }
    w.at = pre[lo] + w.h * head;
    w.it = 0;
    for (; w.it + 1 < w.q.items; ++w.it) {
        const int64_t span = item_span<W>(w.q, group, w.it);
        if (w.at + span > w.x0) break;
        w.at += span;
    }
    load_item<W>(w, a, group);
    return true;
}
template <int W>
__device__ __forceinline__ bool walk_next(Walk &w, const PagedAttnArgs &a, const SeqRow *seqs, int group)
{
    w.at += item_span<W>(w.q, group, w.it);
    if (w.at >= w.x1) return false;
    if (++w.it == w.q.items) {
        w.it = 0;
        if (++w.h == a.kv.n_kv_heads) {
            w.h = 0;
            do {
                if (++w.s >= a.n_seqs) return false;
                w.q = make_seq<W>(seqs[w.s], group);
            } while (w.q.items == 0);
        }
    }
    load_item<W>(w, a, group);
    return true;
}
// Whether this CTA has something to do for the current item: units, or an item without
// any that begins in its share.
__device__ __forceinline__ bool walk_has(const Walk &w)
{
    return w.lo < w.hi || (w.units == 0 && w.at >= w.x0);
}

// ---------------------------------------------------------------- one warp's sums
// NT tiles of 4 queries; this lane (g, t) sums for query 4 j + t of tile j.
template <int NB, int NT>
struct Warp {
    // B fragments of the queries, {low half, high half} of a block: in registers for one tile; for two, beside
    // twice the sums, in shared memory (32 lanes' uint4 for each tile and block)
    uint4 q[NT == 1 ? NB : 1];
    const uint4 *q_shared;
    __device__ __forceinline__ uint4 query(int j, int b) const { return NT == 1 ? q[b] : q_shared[(j * NB + b) * 32]; }
    float unit[NT];            // log2(e) * scale * the unit of the products
    float o[NT][NB][2][4];     // sums of V: tile, block, half, {c0..c3}
    float m[NT], l[NT];        // running maximum (see the top), sum of p
    float *row;                // this lane's row of sums in shared memory (tile 0)
    int since;                 // groups of tokens in o
    bool flushed;              // part of the sums is in shared memory
};

// The sums to shared memory, high and low pieces together.  The tensor cores cut what they
// add to an accumulator instead of rounding it, so that a sum of n steps drifts towards zero by
// up to n / 2 steps of 2^-24: 3.6e-6 after 4000 tokens.  Every kFlush groups the sums are
// added to those in shared memory instead, rounded.
template <int NB, int NT>
__device__ __forceinline__ void flush(Warp<NB, NT> &w, int g)
{
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float *p = w.row + 4 * j * (32 * NB + kPad) + 32 * b + 16 * hf + g;
                float(&c)[4] = w.o[j][b][hf];
                p[0] = (c[0] + c[1]) + (w.flushed ? p[0] : 0.0f);
                p[8] = (c[2] + c[3]) + (w.flushed ? p[8] : 0.0f);
                c[0] = c[1] = c[2] = c[3] = 0.0f;
            }
    w.flushed = true;
    w.since = 0;
}

// The queries in fragment order: this lane holds, for tile j, values 4 t .. 4 t + 3 (of both
// halves of each block) of query 4 j + g / 2 at ptr[j], its high piece (g even) or its low one.  (Plain loads: the
// launch before may write q while this kernel is resident already, which the read-only path does not allow for.)
template <int NB, int NT>
__device__ __forceinline__ void load_query(Warp<NB, NT> &w, uint4 *q_shared, const float *const (&ptr)[NT], float scale, int g,
                                           int t)
{
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float4 v[NB][2];
        float mx = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                v[b][hf] = ptr[j] ? *reinterpret_cast<const float4 *>(ptr[j] + 32 * b + 16 * hf + 4 * t)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v[b][hf].x), fabsf(v[b][hf].y)),
                                     fmaxf(fabsf(v[b][hf].z), fabsf(v[b][hf].w))));
            }
        mx = quad_max(mx);
        // 2^up brings the largest value to [2^14, 2^15); powers of two, so exact
        const int ex = (__float_as_int(mx) >> 23) - 127;
        const int up = mx == 0.0f ? 0 : min(14 - ex, 126);
        const float sc = __int_as_float((up + 127) << 23);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t piece[2][2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float x[4] = {v[b][hf].x * sc, v[b][hf].z * sc, v[b][hf].y * sc, v[b][hf].w * sc};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t hi = pack_f16(x[2 * k], x[2 * k + 1]);
                    const float2 h = unpack_f16(hi);
                    piece[hf][k] = (g & 1) ? pack_f16(x[2 * k] - h.x, x[2 * k + 1] - h.y) : hi;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) w.o[j][b][hf][k] = 0.0f;
            }
            const uint4 v = make_uint4(piece[0][0], piece[0][1], piece[1][0], piece[1][1]);
            if (NT == 1) w.q[b] = v;
            else q_shared[(j * NB + b) * 32] = v;
        }
        // the unit of query t is with lane g = 2 t.  2^-126 at least (scores are below 2^42: the exponents are 0 all the
        // same): a masked score, -infinity, times 0 would be NaN
        w.unit[j] = fmaxf(scale * 1.4426950408889634f * __int_as_float((127 - __shfl_sync(0xffffffffu, up, 8 * t)) << 23), 0x1p-126f);
        w.m[j] = -1e37f;
        w.l[j] = 0.0f;
    }
    w.q_shared = q_shared;
    w.since = 0;
    w.flushed = false;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t *r, const uint8_t *p)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            r[i] = v.x;
            r[i + 1] = v.y;
            r[i + 2] = v.z;
            r[i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p + 4 * i);
            r[i] = v.x;
            r[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = *reinterpret_cast<const uint32_t *>(p + 4 * i);
    }
}

// f16 value i of a run of words
template <int N>
__device__ __forceinline__ float half_at(const uint32_t (&w)[N], int i)
{
    const float2 v = unpack_f16(w[i >> 1]);
    return (i & 1) ? v.y : v.x;
}

__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// NG groups of 16 tokens (records one after another) for the warp's 4 NT queries.
// sees[j]: how many of the tokens this lane's query of tile j sees (kMasked), else all.
// Row g of a product is token 2 g of the group, row g + 8 token 2 g + 1.
template <int NB, int NT, int NG, bool kMasked>
__device__ __forceinline__ void attend(Warp<NB, NT> &w, const uint8_t *rec, int g, int t, const int (&sees)[NT])
{
    constexpr int hd = 32 * NB, kRec = q4_record_bytes(hd);
    // ---- scores of tokens 2 g, 2 g + 1 of each group
    float s[NT][2 * NG];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
        const uint8_t *r = rec + u * kRec;
        uint32_t k0[NB], k1[NB], ks[NB];
        lds_words<NB>(k0, r + 2 * g * (hd / 2) + t * 4 * NB);
        lds_words<NB>(k1, r + (2 * g + 1) * (hd / 2) + t * 4 * NB);
        lds_words<NB>(ks, r + q4_k_scale(NB, 2 * g));
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j][2 * u] = s[j][2 * u + 1] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t h0 = k0[b] >> 8, h1 = k1[b] >> 8;
            const uint32_t lo[4] = {low_codes(k0[b]), low_codes(k1[b]), low_codes(h0), low_codes(h1)};
            const uint32_t hi[4] = {high_codes(k0[b]), high_codes(k1[b]), high_codes(h0), high_codes(h1)};
            const float d0 = half_at(ks, b), d1 = half_at(ks, NB + b);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const uint4 q = w.query(j, b);
                mma16816(c, lo, q.x, q.y, c);
                mma16816(c, hi, q.z, q.w, c);
                s[j][2 * u] = fmaf(d0, c[0] + c[1], s[j][2 * u]);
                s[j][2 * u + 1] = fmaf(d1, c[2] + c[3], s[j][2 * u + 1]);
            }
        }
    }
    uint32_t vs[NG][NB];
    uint32_t dm = 0;  // the largest |d| of this lane's tokens, two f16
#pragma unroll
    for (int u = 0; u < NG; ++u) {
        lds_words<NB>(vs[u], rec + u * kRec + q4_v_scale(NB, 2 * g));
        if (kMasked) {
            // what the last query does not see is whatever the page holds: its scales are dropped
            // here (0), and each query's own mask below takes its score
            int most = sees[0];
#pragma unroll
            for (int j = 1; j < NT; ++j) most = max(most, sees[j]);
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (16 * u + 2 * g + i >= most) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int k = i * NB + b;
                        vs[u][k >> 1] &= (k & 1) ? 0x0000ffffu : 0xffff0000u;
                    }
                }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (16 * u + 2 * g + i >= sees[j]) s[j][2 * u + i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const uint32_t v = vs[u][i] & 0x7fff7fffu;
            asm("max.f16x2 %0, %0, %1;" : "+r"(dm) : "r"(v));
        }
    }
    // ---- running maximum of log2 p + log2 |d|; the exponent above the largest |d| (0: of the smallest f16)
    const float2 dm2 = unpack_f16(dm);
    const float ev = static_cast<float>((__float_as_int(fmaxf(fmaxf(dm2.x, dm2.y), 0x1p-25f)) >> 23) - 126);
    float y[NT];
    bool grown = false;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float top = s[j][0];
#pragma unroll
        for (int i = 1; i < 2 * NG; ++i) top = fmaxf(top, s[j][i]);
        y[j] = fmaf(top, w.unit[j], ev);
        grown |= y[j] > w.m[j] + kLazy;
    }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float top = y[j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float m = top > w.m[j] + kLazy ? top : w.m[j];
            const float f = ex2(w.m[j] - m);
            w.m[j] = m;
            w.l[j] *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) w.o[j][b][hf][k] *= f;
                    if (w.flushed) {
                        float *p = w.row + 4 * j * (hd + kPad) + 32 * b + 16 * hf + g;
                        p[0] *= f;
                        p[8] *= f;
                    }
                }
        }
    }
    // ---- weights p, then the sums of V
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const float off = kBias - w.m[j];
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) {
            s[j][i] = ex2(fmaf(s[j][i], w.unit[j], off));
            w.l[j] += s[j][i];
        }
    }
#pragma unroll
    for (int u = 0; u < NG; ++u) {
        uint32_t vw[2 * NB];
        constexpr int run = q4_v_run(NB);
#pragma unroll
        for (int r = 0; r < 2 * NB; r += run)
            lds_words<run>(vw + r, rec + u * kRec + 9 * hd + ((r / run) * 32 + 4 * g + t) * run * 4);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float d0 = half_at(vs[u], b), d1 = half_at(vs[u], NB + b);
            uint32_t pb[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float x0 = s[j][2 * u] * d0, x1 = s[j][2 * u + 1] * d1;
                if (kMasked) {  // a NaN or infinite scale that another query sees
                    if (16 * u + 2 * g >= sees[j]) x0 = 0.0f;
                    if (16 * u + 2 * g + 1 >= sees[j]) x1 = 0.0f;
                }
                const uint32_t h = pack_f16(x0, x1);
                const float2 hf = unpack_f16(h);
                const uint32_t l = pack_f16(x0 - hf.x, x1 - hf.y);
                pb[j][0] = transposed(__byte_perm(h, l, 0x5410));
                pb[j][1] = transposed(__byte_perm(h, l, 0x7632));
            }
            const uint32_t w0 = vw[2 * b], w1 = vw[2 * b + 1], h0 = w0 >> 8, h1 = w1 >> 8;
            const uint32_t lo[4] = {low_codes(w0), low_codes(w1), low_codes(h0), low_codes(h1)};
            const uint32_t hi[4] = {high_codes(w0), high_codes(w1), high_codes(h0), high_codes(h1)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                mma16816(w.o[j][b][0], lo, pb[j][0], pb[j][1], w.o[j][b][0]);
                mma16816(w.o[j][b][1], hi, pb[j][0], pb[j][1], w.o[j][b][1]);
            }
        }
    }
}

// ---------------------------------------------------------------- shared memory
// slots of 2 records | query fragments | the warps' sums, their (m, l) | mbarriers, flags, counts (512 bytes) |
// the parts of an item | the line's prefix | the requests
constexpr int kMaxSlots = 24;  // at most 32: a lane of the producer waits for each at the end
constexpr int kMaxCtas = 512;  // of the grid
template <int NB>
struct Layout {
    static constexpr int W = consumers(NB), hd = 32 * NB, rows = 8 * W;
    static constexpr int slot = 2 * q4_record_bytes(hd);
    static constexpr int sums = rows * (hd + kPad) * 4;
    static constexpr int queries = W * 2 * NB * 512;  // fragments of two tiles of queries for each warp
    static constexpr int fixed = queries + sums + rows * 8 + 512 + 2 * kMaxCtas * 2;  // and 20 bytes for each request and 8
    static constexpr int64_t part = (int64_t)rows * (hd + 2);  // floats of a partial record: sums, then (m, l)
};

// Four values of one row, divided by its sum, to the outputs.  Every lane of the warp
// calls it (8 lanes hold a block of 32 values); live: this lane's row exists.
__device__ __forceinline__ void write_row4(const PagedAttnArgs &a, float4 v, bool live, int64_t row, int col, int q_pad)
{
    const int q_dim = a.n_heads * a.kv.head_dim;
    if (a.att && live) *reinterpret_cast<float4 *>(a.att + row * q_dim + col) = v;
    if (a.att_q8) {
        float mx = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float d = __fdiv_rn(mx, 127.0f);
        const Q8Scale sc = q8_scale(d);
        const int c0 = q8_code(v.x, sc), c1 = q8_code(v.y, sc), c2 = q8_code(v.z, sc), c3 = q8_code(v.w, sc);
        int sum = c0 + c1 + c2 + c3;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (live) {
            int8_t *q = static_cast<int8_t *>(a.att_q8);
            float *qd = reinterpret_cast<float *>(q + a.n_rows * q_pad);
            float *qs = qd + a.n_rows * (q_pad / 32);
            *reinterpret_cast<char4 *>(q + row * q_pad + col) = make_char4(c0, c1, c2, c3);
            if ((threadIdx.x & 7) == 0) {
                qd[row * (q_pad / 32) + col / 32] = d;
                qs[row * (q_pad / 32) + col / 32] = __fmul_rn(d, (float)sum);
            }
        }
    }
}

// n slots on
__device__ __forceinline__ void ring_advance(RingPos &r, int n, int slots)
{
    const unsigned s = r.s + n, laps = s < static_cast<unsigned>(slots) ? 0 : s / static_cast<unsigned>(slots);
    r.s = s - laps * slots;
    r.par ^= laps & 1;
}
// the same for n <= slots
__device__ __forceinline__ void ring_step(RingPos &r, int n, int slots)
{
    r.s += n;
    if (r.s >= slots) {
        r.s -= slots;
        r.par ^= 1u;
    }
}

// Most polls of a wait: those that the test aid gives its CTA 0, else the usual number.
__device__ __forceinline__ uint32_t wait_limit(const PagedAttnArgs &a) { return a.stall && blockIdx.x == 0 ? a.stall : kWaitLimit; }

// Bounded wait that ends, too, when another warp has given up.
__device__ __forceinline__ bool wait_unless(uint64_t *bar, unsigned par, uint32_t limit, const volatile int *gave_up)
{
    for (uint32_t i = 0; i < limit; ++i) {
        if (mbar_try_wait(bar, par)) return true;
        if (*gave_up) return false;
    }
    return false;
}

// A consumer warp's share of the current part of an item: its sums to shared memory.
template <int NB, int NT, int NG>
__device__ __forceinline__ void work(const PagedAttnArgs &a, const Walk &w, const uint8_t *ring, int slots, uint64_t *full,
                                     uint64_t *empty, volatile int *gave_up, RingPos &pos, float *sums, float2 *ml, uint4 *queries, int warp,
                                     int lane)
{
    using L = Layout<NB>;
    constexpr int W = L::W, hd = L::hd;
    const int g = lane >> 2, t = lane & 3, group = a.n_heads / a.kv.n_kv_heads;
    const int rg = w.q.rg, copies = W / rg;
    const int qg = warp % rg, ks = warp / rg;
    const int row8 = (w.it * rg + qg) * 8;  // this warp's first query row
    const int n_rows = w.q.m * group;       // of the request and kv head
    const bool idle = row8 >= n_rows || ks >= copies;
    // tokens that a row sees (rows beyond the last see what the last sees, and are not
    // written): this lane's rows, the warp's first and its last
    const int before = w.q.n - w.q.m + 1;
    auto tokens_of = [&](int row) { return max(before + min(row, n_rows - 1) / group, 0); };
    int sees[NT];
    const float *ptr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        sees[j] = tokens_of(row8 + 4 * j + t);
        const int my = row8 + 4 * j + (g >> 1), tok = my / group;
        ptr[j] = my < n_rows ? a.q + (w.q.row0 + tok) * a.ld_q + (int64_t)(w.h * group + (my - tok * group)) * hd : nullptr;
    }
    const int all_see = tokens_of(row8), any_see = idle ? 0 : tokens_of(row8 + 4 * NT - 1);
    const int slot = (ks * rg + qg) * 8 + t;  // of this lane's row, copy ks
    // a unit's readers together arrive W times on its slot's barrier
    const int arrive = qg == 0 ? W + 1 - min(rg, (n_rows - w.it * rg * 8 + 7) >> 3) : 1;
    Warp<NB, NT> acc;
    acc.row = sums + slot * (hd + kPad);
    load_query<NB, NT>(acc, queries + warp * 2 * NB * 32 + lane, ptr, a.scale, g, t);
    RingPos mine = pos;
    ring_step(mine, ks, slots);
    for (int u = idle || __any_sync(0xffffffffu, *gave_up) ? w.hi : w.lo + ks; u < w.hi; u += copies) {
        if (!__all_sync(0xffffffffu, mbar_wait(full + mine.s, mine.par, wait_limit(a)))) {
            *gave_up = 1;
            set_error(a.err, DEV_TIMEOUT_PAGED);
            break;
        }
        const uint8_t *st = ring + (size_t)mine.s * L::slot;
#pragma unroll 1
        for (int r = 0; r < 2 / NG; ++r) {
            const int t0 = u * kUnit + 16 * r;
            if (t0 >= any_see) break;
            const uint8_t *rec = st + r * q4_record_bytes(hd);
            int left[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) left[j] = sees[j] - t0;
            if (t0 + 16 * NG <= all_see)
                attend<NB, NT, NG, false>(acc, rec, g, t, left);
            else
                attend<NB, NT, NG, true>(acc, rec, g, t, left);
            if ((acc.since += NG) >= kFlush) flush(acc, g);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_n(empty + mine.s, arrive);
        ring_step(mine, copies, slots);
    }
    ring_advance(pos, w.hi - w.lo, slots);
    if (ks < copies) {
        flush(acc, g);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float l = acc.l[j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (g == 0) ml[slot + 4 * j] = make_float2(acc.m[j], l);
        }
    }
}

template <int NB>
__global__ void __launch_bounds__((consumers(NB) + 1) * 32, 2)
    paged_attention_kernel(const __grid_constant__ PagedAttnArgs a, int most_slots)
{
    using L = Layout<NB>;
    constexpr int W = L::W, hd = L::hd, ld = hd + kPad, kSlot = L::slot;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;
    uint4 *queries = reinterpret_cast<uint4 *>(ring + (size_t)most_slots * kSlot);
    float *sums = reinterpret_cast<float *>(queries + L::queries / 16);
    float2 *ml = reinterpret_cast<float2 *>(sums + L::sums / 4);
    uint64_t *full = reinterpret_cast<uint64_t *>(ml + L::rows), *empty = full + kMaxSlots;
    int *flags = reinterpret_cast<int *>(empty + kMaxSlots);  // [0] a wait ran out, [1] this CTA adds the parts up
    int *part_count = flags + 2;  // 2
    uint64_t *listed = empty + kMaxSlots + 2;  // the lists of parts are there
    int16_t *part_list = reinterpret_cast<int16_t *>(reinterpret_cast<uint8_t *>(full) + 512);
    int64_t *pre = reinterpret_cast<int64_t *>(part_list + 2 * kMaxCtas);
    SeqRow *seqs = reinterpret_cast<SeqRow *>(pre + a.n_seqs + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = a.kv.n_kv_heads, group = a.n_heads / K;
    if (tid == 0) {
        for (int i = 0; i < most_slots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, W);
        }
        mbar_init(listed, 1);
        mbar_init(listed + 1, 1);
        fence_mbar_init();
        flags[0] = flags[1] = 0;
        part_count[0] = part_count[1] = 0;
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---- the line: what comes before each request
    bool halves = false;  // items of two row groups, W / 2 copies of each
    {
        int64_t *tmp = reinterpret_cast<int64_t *>(sums);
        const int per = (a.n_seqs + W * 32 - 1) / (W * 32);
        int64_t mine = 0;
        bool bad = false;
        if (tid < W * 32)
            for (int i = tid * per; i < min(a.n_seqs, (tid + 1) * per); ++i) {
                seqs[i] = read_seq(a, i, bad);
                const Seq q = make_seq<W>(seqs[i], group);
                halves |= W > 3 && q.rg == 2 && q.items > 0;
                int64_t span = 0;
                for (int it = 0; it < q.items; ++it) span += item_span<W>(q, group, it);
                pre[i + 1] = span * K;
                mine += span * K;
            }
        if (bad && blockIdx.x == 0) set_error(a.err, DEV_BAD_LENGTH);
        int64_t v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) tmp[warp] = v;
        halves = __syncthreads_or(halves);
        if (tid < W * 32) {
            for (int k = 0; k < warp; ++k) v += tmp[k];
            v -= mine;
            for (int i = tid * per; i < min(a.n_seqs, (tid + 1) * per); ++i) {
                v += pre[i + 1];
                pre[i + 1] = v;
            }
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
    }

    // A multiple of every number of copies that there is (W, W / 2, 1), so that the unit that was in a slot before is one
    // that the same warp has worked: it would take the phase before, whose copies may land later than others', for its own.
    const int step = halves ? W / 2 * W : W, slots = most_slots / step * step;
    volatile int *gave_up = flags;
    Walk w;
    const Line line = make_line<W>(pre[a.n_seqs], gridDim.x);
    const bool any = walk_begin<W>(w, a, line, pre, seqs, group);
    if (!any) return;  // the same for the whole CTA

    if (warp == W) {
        // ---------------------------------------------------------------- producer
        const int lg = a.kv.page_log;
        constexpr int kRec = q4_record_bytes(hd);
        const int64_t head_bytes = (int64_t)kRec << lg;
        RingPos pos{0, 0};
        int issued = 0;
        bool more = true;
        const bool stalled = a.stall && blockIdx.x == 0;  // test aid: the first unit is not issued
        // the step's keys and values were written by another kernel through the generic proxy
        asm volatile("fence.proxy.async;" ::: "memory");
        while (more) {
            const int32_t *row = a.table + (int64_t)w.s * a.table_ld;
            for (int u0 = w.lo; u0 < w.hi; u0 += W) {
                // lane i copies unit u0 + i: two groups of 16 tokens, or the last one, of one page or two
                const int n = min(W, w.hi - u0), u = u0 + lane;
                const int g0 = 2 * u, groups = min(2, ((w.tokens + 15) >> 4) - g0);
                RingPos mine = pos;
                ring_step(mine, min(lane, W), slots);
                int32_t page[2] = {0, 0};
                if (lane < n) {
                    page[0] = row[g0 >> lg];
                    page[1] = lg == 0 && groups == 2 ? row[g0 + 1] : page[0];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (page[i] < 0 || page[i] >= a.kv.n_pages) {
                            set_error(a.err, DEV_BAD_PAGE);
                            page[i] = 0;  // a page there is; the request's rows are not to be used
                        }
                }
                bool ok = !*gave_up;
                if (lane < n && ok) ok = mbar_wait(empty + mine.s, mine.par ^ 1u, wait_limit(a));
                if (!__all_sync(0xffffffffu, ok)) {
                    if (!*gave_up) set_error(a.err, DEV_TIMEOUT_PAGED);
                    *gave_up = 1;
                    more = false;
                    break;
                }
                if (lane < n && !(stalled && issued + lane == 0)) {
                    uint8_t *dst = ring + (size_t)mine.s * kSlot;
                    const uint8_t *src = a.kv.pages + ((int64_t)page[0] * K + w.h) * head_bytes + (g0 & ((1 << lg) - 1)) * kRec;
                    mbar_arrive_expect_tx(full + mine.s, groups * kRec);
                    if (lg || groups == 1) {
                        bulk_g2s(dst, src, groups * kRec, full + mine.s);
                    } else {
                        bulk_g2s(dst, src, kRec, full + mine.s);
                        bulk_g2s(dst + kRec, a.kv.pages + ((int64_t)page[1] * K + w.h) * head_bytes, kRec, full + mine.s);
                    }
                }
                issued += n;
                ring_step(pos, n, slots);
            }
            if (more && w.lo < w.hi && (w.lo > 0 || w.hi < w.units)) {
                // a part of an item, its copies on their way: the CTAs whose shares hold its units, in order (a CTA
                // has one part that begins its item and one that does not)
                const int cost = unit_cost<W>(w.q.rg);
                int16_t *list = part_list + (w.lo == 0) * kMaxCtas;
                int c = min(static_cast<int>(min(w.at / max(line.step, (int64_t)1), (int64_t)line.ctas)), line.ctas - 1);
                while (line.begin(c) > w.at) --c;
                int parts = 0;
                for (int c0 = c; c0 < line.ctas && line.begin(c0) < w.at + kItemCost<W> + (int64_t)w.units * cost; c0 += 32) {
                    const int k = c0 + lane;
                    const int lo = unit_at<W>(line.begin(k) - w.at, w.units, cost), hi = unit_at<W>(line.begin(k + 1) - w.at, w.units, cost);
                    const bool has = k < line.ctas && lo < hi;
                    const unsigned all = __ballot_sync(0xffffffffu, has);
                    if (has) list[parts + __popc(all & ((1u << lane) - 1))] = static_cast<int16_t>(2 * k + (lo == 0));  // odd: begins the item
                    parts += __popc(all);
                }
                __syncwarp();
                if (lane == 0) {
                    part_count[w.lo == 0] = parts;
                    mbar_arrive(listed + (w.lo == 0));
                }
            }
            if (more) more = walk_next<W>(w, a, seqs, group);
        }
        // No copy outlives the CTA: consumers that give up, now or later, leave copies that they do not wait for.  Lane i
        // waits for the last unit in slot i.
        if (lane < min(issued, slots) && !(stalled && lane == 0) && !mbar_wait(full + lane, lane < pos.s ? pos.par : pos.par ^ 1u))
            set_error(a.err, DEV_TIMEOUT_DRAIN);
        return;
    }

    // -------------------------------------------------------------------- consumers
    const int q_pad = (a.n_heads * hd + 255) / 256 * 256;
    RingPos pos{0, 0};
    bool more = true;
    while (more) {
        if (walk_has(w)) {
            // rg row groups, copies warps for each, the others idle
            const int rg = w.q.rg, copies = W / rg, row_it = w.it * 8 * rg;
            const int n_rows = w.q.m * group;  // of the request and kv head
            if (n_rows <= 4)
                work<NB, 1, 2>(a, w, ring, slots, full, empty, gave_up, pos, sums, ml, queries, warp, lane);
            else
                work<NB, 2, 1>(a, w, ring, slots, full, empty, gave_up, pos, sums, ml, queries, warp, lane);
            consumer_sync<W>();
            const int rows_item = min(8 * rg, n_rows - row_it);
            const bool whole = w.lo == 0 && w.hi == w.units;
            const int quads = 8 * rg * (hd / 4);  // groups of 4 values of the item's rows
            float *part = a.part + (2 * (int64_t)blockIdx.x + (w.lo == 0)) * L::part;
            for (int i0 = 0; i0 < quads; i0 += W * 32) {
                const int i = i0 + tid;
                const int r = i / (hd / 4), c4 = i % (hd / 4) * 4;
                const bool mine = i < quads && r < rows_item;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float m = -1e37f, l = 0.0f;
                if (mine) {
                    for (int k = 0; k < copies; ++k) m = fmaxf(m, ml[k * 8 * rg + r].x);
                    for (int k = 0; k < copies; ++k) {
                        const float2 x = ml[k * 8 * rg + r];
                        const float f = ex2(x.x - m);
                        const float4 u = *reinterpret_cast<const float4 *>(sums + (k * 8 * rg + r) * ld + c4);
                        l = fmaf(x.y, f, l);
                        v.x = fmaf(u.x, f, v.x);
                        v.y = fmaf(u.y, f, v.y);
                        v.z = fmaf(u.z, f, v.z);
                        v.w = fmaf(u.w, f, v.w);
                    }
                }
                if (whole) {
                    // l == 0: the row sees nothing.  A NaN stays one.
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    const int my_row = row_it + r;
                    write_row4(a, v, mine, w.q.row0 + my_row / group, (w.h * group + my_row % group) * hd + c4, q_pad);
                } else if (mine) {
                    *reinterpret_cast<float4 *>(part + r * hd + c4) = v;
                    if (c4 == 0) *reinterpret_cast<float2 *>(part + L::rows * hd + 2 * r) = make_float2(m, l);
                }
            }
            if (!whole) {
                // ---- the last CTA to arrive adds the parts up
                const bool known = wait_unless(listed + (w.lo == 0), 0, wait_limit(a), gave_up);  // false: the producer gave up
                const int parts = known ? part_count[w.lo == 0] : 0;
                const int16_t *list = part_list + (w.lo == 0) * kMaxCtas;
                consumer_sync<W>();  // the part is written
                if (tid == 0) {
                    // (the add releases what the barrier gathered, and acquires the other parts)
                    int *counter = a.counters + (known ? list[0] >> 1 : 0);
                    const int before = known ? add_acq_rel(counter, 1) : -1;
                    flags[1] = known && before == parts - 1;
                    if (flags[1]) *counter = 0;
                }
                consumer_sync<W>();
                if (flags[1]) {
                    for (int i0 = 0; i0 < quads; i0 += W * 32) {
                        const int i = i0 + tid;
                        const int r = i / (hd / 4), c4 = i % (hd / 4) * 4;
                        const bool mine = i < quads && r < rows_item;
                        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        float m = -1e37f, l = 0.0f;
                        if (mine) {
#pragma unroll 8
                            for (int k = 0; k < parts; ++k) {
                                const float *pk = a.part + list[k] * L::part;
                                const float2 x = __ldcg(reinterpret_cast<const float2 *>(pk + L::rows * hd + 2 * r));
                                const float4 u = __ldcg(reinterpret_cast<const float4 *>(pk + r * hd + c4));
                                const float mn = fmaxf(m, x.x), f0 = ex2(m - mn), f1 = ex2(x.x - mn);
                                m = mn;
                                l = fmaf(l, f0, x.y * f1);
                                v.x = fmaf(v.x, f0, u.x * f1);
                                v.y = fmaf(v.y, f0, u.y * f1);
                                v.z = fmaf(v.z, f0, u.z * f1);
                                v.w = fmaf(v.w, f0, u.w * f1);
                            }
                        }
                        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                        const int my_row = row_it + r;
                        write_row4(a, v, mine, w.q.row0 + my_row / group, (w.h * group + my_row % group) * hd + c4, q_pad);
                    }
                }
            }
            // the zero padding of the Q8_1 rows, with kv head 0
            if (a.att_q8 && w.h == 0 && w.lo == 0) {
                const int q_dim = a.n_heads * hd, pad = q_pad - q_dim;
                if (pad) {
                    int8_t *q8 = static_cast<int8_t *>(a.att_q8);
                    float *qd = reinterpret_cast<float *>(q8 + a.n_rows * q_pad);
                    float *qs = qd + a.n_rows * (q_pad / 32);
                    const int r0 = row_it / group;
                    const int r1 = min(w.q.m, (row_it + rows_item - 1) / group + 1);
                    for (int i = tid; i < (r1 - r0) * pad; i += W * 32) {
                        const int64_t rr = w.q.row0 + r0 + i / pad;
                        const int cc = q_dim + i % pad;
                        q8[rr * q_pad + cc] = 0;
                        if (cc % 32 == 0) {
                            qd[rr * (q_pad / 32) + cc / 32] = 0.0f;
                            qs[rr * (q_pad / 32) + cc / 32] = 0.0f;
                        }
                    }
                }
            }
            consumer_sync<W>();  // sums, ml and the flag are read
        }
        more = walk_next<W>(w, a, seqs, group);
    }
}

int grid_ctas() { return std::min(2 * dev_info().sm_count, kMaxCtas); }

template <int NB>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t s)
{
    using L = Layout<NB>;
    // half an SM's shared memory (228 KB, 1 KB of it for each CTA), as many slots as fit
    constexpr int most = 113 * 1024;
    static_assert((most - L::fixed - kPagedMaxSeqs * 20 - 8) / L::slot >= (L::W > 3 ? L::W / 2 * L::W : L::W), "a ring for any number of requests");
    const int fixed = L::fixed + a.n_seqs * 20 + 8;
    const int slots = std::min(kMaxSlots, (most - fixed) / L::slot);
    const int bytes = slots * L::slot + fixed;
    static std::atomic<uint64_t> done{0};  // devices on which the kernel may have that much
    const uint64_t bit = 1ull << (dev_info().device & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid_ctas());
    cfg.blockDim = dim3((L::W + 1) * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, paged_attention_kernel<NB>, a, slots);
}

cudaError_t launch_any(const PagedAttnArgs &a, cudaStream_t s)
{
    switch (a.kv.head_dim / 32) {
        case 1: return launch<1>(a, s);
        case 2: return launch<2>(a, s);
        case 3: return launch<3>(a, s);
        case 4: return launch<4>(a, s);
        case 5: return launch<5>(a, s);
        case 6: return launch<6>(a, s);
        case 7: return launch<7>(a, s);
        default: return launch<8>(a, s);
    }
}

}  // namespace

// counters (zero before the first call, zero again after each), then two partial records for each CTA
size_t paged_attention_workspace_bytes(int head_dim)
{
    const size_t ctas = grid_ctas();
    const size_t parts = 2 * ctas * 8 * consumers(head_dim / 32) * (head_dim + 2) * 4;
    return (ctas * 4 + 255) / 256 * 256 +
           std::max(parts, paged_attention_tc_takes(head_dim) ? paged_attention_tc_part_bytes(head_dim) : size_t(0));
}

cudaError_t launch_paged_attention(const PagedAttnArgs &args, void *workspace, cudaStream_t s)
{
    PagedAttnArgs a = args;
    a.counters = static_cast<int *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + ((size_t)grid_ctas() * 4 + 255) / 256 * 256);
    // Requests with many rows go to the tcgen05 kernel.  Whether there may be one: if every
    // request has a row, one of them has at most n_rows - n_seqs + 1.  (If there is one all the
    // same, because others have none, it is worked here: 777 new rows of 2000 tokens, 32 heads on 8 of 128, take 299 us
    // among 999 idle requests, 135 alone.  A launch in vain costs every step of single tokens 2 us.)
    const int group = a.n_heads / a.kv.n_kv_heads;
    const bool tc = paged_attention_tc_takes(a.kv.head_dim) && (a.n_rows - a.n_seqs + 1) * group > kTcRows;
    a.most_rows = tc ? kTcRows : 0x7fffffff;
    a.stall = g_stall_next_paged;
    g_stall_next_paged = 0;  // one call only
    const cudaError_t e = launch_any(a, s);
    return e != cudaSuccess || !tc ? e : launch_paged_attention_tc(a, s);
}

}  // namespace rz
