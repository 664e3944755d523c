// moe_gemm_tc.cu -- products grouped by expert of many rows on tcgen05.mma: Q4_K weights of
// each expert against the Q8_1 rows that chose it (formulas and arguments of moe_gemv.cu).
//
// A tile is two matrices of 128 weight rows (gate and up of the same outputs; or 256
// outputs) by kN rows of one expert.  For each super-block of 256 weights
//   D = A B,  A [128][256 + 32] the weights' codes, B [256 + 32][kN] the activations
//   sum += g * (2^E * D)                 g a scale for each weight row, E an exponent for each column
// A holds sc * code or sc * (code - 8), at most 945, exact in f16, and, in further columns, what is left of the weights; it is
// made in registers and stored in tensor memory, which leaves shared memory's bandwidth to B.
// B holds d8 * code / 2^E as two f16 pieces (22 bits), so that one super-block is one
// accumulation of 2 x 16 instructions of K = 16, and accumulators are read once for 256 weights:
// products of the codes alone, exact in f16, would have to be read and scaled for each 32
// (rz_q4k_q8_gemm: 344 TFLOP/s of the formula's operations).  A kernel before this one forms B's pieces,
// once for a (token, choice) row however many tiles of outputs read it: a token of k experts has its pieces formed and held k times.
//
// The pieces have 22 bits of the largest scale among the 256 values: with that between 1/2 and 1, f16 has steps of 2^-24, which a block whose scale
// is 2^-k of it feels from k = 3 on (off by up to 2^(k - 24) of its largest value; the integer dots keep every bit).
//
// The rest of a weight, -dmin m or 8 d sc - dmin m, times the sum s of a block of x, goes into the same accumulators: A's
// r_j = -m_j dmin / (8 d) (+ sc_j) and B's 8 s_j / 2^E, two f16 pieces each, all four products.
//
// The tensor cores cut what they add to an accumulator: up to 2^-23 of it for each of 18 instructions (with the low pieces of B
// apart, in columns of their own or before the high ones), always towards zero; then it is added up, rounded, and starts again.
// Of weights around zero codes and mins cancel, so what is cut goes by the sums on the way.  In tiles of 16 and 32 rows the mins of 4
// sub-blocks come beside their codes and every other sub-block is centred, which costs nothing; in those of 128 the mins come first,
// all codes are centred.  Off by 5.5 to 7e-7 of the values of a SwiGLU (1.2e-6 without either; the plain form in f32 0.6 to 1.7e-6).
//
// The scale g of a row is d.  Where dmin is over 2^13 times d, f16 would not hold r_j: g = 2^p d, with p such that 2^12 <= dmin / g < 2^13, and codes
// and r_j are scaled by 2^-p.  The least step of f16 is 2^-24, so that codes lose nothing up to p = 24, dmin = 2^37 d; beyond that (p is at
// most 27, as f16 has no larger dmin and no smaller d) 36 d at most, 2^-33 of dmin.  With d = 0, g = dmin and the codes are 0.
//
// A super-block with a scale that is no number gives its row NaN (g), a block of x its column (B's pieces).
//
// Roles of the warps, one CTA for each SM, items (expert, tile of its outputs, tile of its rows) in turn:
//   warps 0, 1   issue the products of the first and second matrix (what synchronises costs a warp some 50 to 100
//                cycles each, so that one warp for both was the bottleneck)
//   warp 2       copies B, bulk copies of tiles laid out as shared memory takes them (moe_pack_kernel, the launch before)
//   warp 3       copies the raw weights, 128 rows x 144 bytes a box
//   groups of 4  unpack A, a thread for a weight row, two groups for each matrix: every other super-block (kN <= 32; every other slot of each
//                was 135 instead of 126 us, scales and mins looked up twice), or every other slot
//   8 warps      add up: a thread has a weight row of both matrices and half of the columns
// Few rows (kN <= 32): the two pieces of B stand side by side as 2 kN columns, which halves the instructions.
//
// Bound and measured, in a graph.  Tiles of 16 and 32: issue slots, for unpacking (over 70% are taken; 16 tokens of 2 in 8 experts, gate and up 4096 >
// 14336: 113 us, 4.6 TB/s; 129 of 8 in 128, 2048 > 768: 63 us, 3.6 TB/s); code in those loops that is not even run costs (6% what stood there
// for the rare scales of the mins, 4% longer waits).  Tiles of 128: the tensor cores, some 60% of the time (1024 tokens) at 34 instructions for the
// formula's 16 (4096 of 2 in 8, 4096 > 14336: 2980 us, 645 TFLOP/s of the formula's; call by call 3300 us), and accumulators that are read before a
// matrix's next super-block: tensor memory is full.  With the Q8_1 output, whose scales the warps that add up form: 119, 70 and 3670 us.
//
// Every wait is bounded; after one that runs out every role stops, copies and products in flight
// are waited for, and tensor memory is freed.
#include <math.h>
#include <stddef.h>

#include <algorithm>

#include "mma_f16.cuh"
#include "moe_tiles.h"
#include "rz_common.cuh"
#include "rz_kernels.h"

namespace rz {
namespace {

constexpr int kRawBytes = 144 * 128;
constexpr int kHdr = 4;      // super-blocks whose scales are held
constexpr int kItems = 16;   // items whose places are held (copies are some six super-blocks ahead of the sums)
template <int N>
struct Cfg {
    static constexpr bool kStack = N <= 32;           // pieces side by side
    static constexpr int kColsD = kStack ? 2 * N : N;
    static constexpr int kChunks = kStack ? 2 : 1;    // of 64 weights, in a slot of A
    // What A is filled with for a super-block: side by side, two slots of two chunks and their four mins; else the mins, then
    // four slots of a chunk (no room in tensor memory for wider ones)
    static constexpr int kUses = kStack ? 2 : 5;
    // What B's copies bring: side by side, the same two; else the mins, the low pieces of the four chunks, their high ones.  The low
    // pieces come first, while the accumulators are small: what is added to a large one is cut by as much, however small it is.
    static constexpr int kEntries = kStack ? 2 : 9;
    static constexpr int kGroups = 4;                 // that unpack A: two for each matrix, taking its steps in turn
    static constexpr int kBufD = N == 128 ? 2 : 3;    // accumulators: one for each matrix, or three in turn
    static constexpr int kSlotsA = N == 128 ? 4 : 2;  // of A for each matrix
    static constexpr int kMinsB = N * (kStack ? 32 : 64);
    static constexpr int kBytesB = N * (kStack ? 512 : 128);  // two pieces of 128 values, or one of 64
    static constexpr int kSlotB = kBytesB + (kStack ? kMinsB : 0);
    static constexpr int kRingB = kStack ? 5 : 8;
    static constexpr int kCellB = N * 1024 + N * 64;   // of a super-block
    static constexpr int kRingRaw = N == 128 ? 4 : N == 16 ? 8 : 6;
    static constexpr int kColA = kBufD * kColsD;      // tensor memory: accumulators, then A
    static constexpr int kWidthA = 32 * kChunks + (kStack ? 8 : 0);
    static constexpr int kHalf = N / 2;               // columns of a thread that adds up
    static constexpr int kFirstUnpack = 4, kFirstSum = kFirstUnpack + 4 * kGroups;
    static constexpr int kThreads = 32 * (kFirstSum + 8);
    // registers of the roles (0: as launched)
    static constexpr int kRegsIssue = N == 128 ? 40 : 0, kRegsUnpack = N == 128 ? 40 : 0, kRegsSum = N == 128 ? 152 : 0;
    static constexpr int off_b = 0;
    static constexpr int off_raw = off_b + kRingB * kSlotB;
    static constexpr int off_g = off_raw + kRingRaw * kRawBytes;   // [kHdr][2][128]
    static constexpr int off_cs = off_g + kHdr * 2 * 128 * 4;      // [kHdr][N]
    static constexpr int off_item = off_cs + kHdr * N * 4;         // int4 [kItems]
    static constexpr int off_cum = off_item + 16 * kItems;         // int [kMoeMaxExperts + 1]
    static constexpr int off_bars = off_cum + 4 * (kMoeMaxExperts + 1) + 12;
    static constexpr int bytes = off_bars + 768 + 1024;
    static_assert(kColA + 2 * kSlotsA * kWidthA <= 512, "tensor memory");
    static_assert(off_raw % 128 == 0, "copies start on 128 bytes");
    static_assert(bytes <= 227 * 1024, "shared memory");
    static_assert(kRingRaw % 2 == 0, "rings");
    // Scales of super-block k take the place of those of k - kHdr, added up by then: whoever writes them has seen the products of a
    // step at most kRingB (or kSlotsA) before done, whose accumulators were free, which takes all but the last three of those before
    static_assert((kRingB + kEntries - 1) / kEntries + 1 <= kHdr, "scales");
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static_assert(kRegsSum == 0 || 128 * (kRegsIssue + kGroups * kRegsUnpack) + 256 * kRegsSum <= kThreads * kLaunchRegs, "registers");
};

struct Bars {
    uint64_t a_full[2][4], a_empty[2][4], b_full[8], b_empty[8], raw_full[8], raw_empty[8], d_full[3], d_empty[3], h_full[kHdr], cs_full[kHdr], done[2];
    uint32_t tmem, limit;    // polls of a wait; 0 once one has run out
    int parts;
};
static_assert(sizeof(Bars) <= 768, "barriers");

struct TcArgs {
    CUtensorMap map1, map2;
    MoeGemvArgs g;
    const uint8_t *pack;     // B of tile i and super-block j, as its copies go to shared memory: at (i * nsb + j) * kCellB
    const float *col_scale;  // 2^E [tiles][super-blocks][kN]
    uint32_t stall;          // test aid (rz_debug_stall_next_moe), 0 otherwise
};

// Shared-memory operand, K-major, no swizzle: core matrices of 8 rows x 16 bytes, 128 bytes apart along K, groups of 8 rows `stride`
// apart; in two words
__device__ __forceinline__ uint32_t operand_low(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((128u >> 4) << 16); }
__host__ __device__ constexpr uint32_t operand_high(uint32_t stride) { return (stride >> 4) | (1u << 14); }
__host__ __device__ constexpr uint32_t idesc_f16(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }

// One lane of the warp, all of which are here.
__device__ __forceinline__ uint32_t elect()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
// Issued by the elected lane.  A predicate and no branch: the operands are the same for the warp and stay in uniform registers (in a
// branch of one lane each would be moved there for every instruction, some 100 cycles).
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint32_t b_low, uint32_t b_high, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_low), "r"(b_high), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(elected)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t elected, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tm_store8(uint32_t at, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tm_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 8 columns of the warp's 32 rows, waited for in the same statement
__device__ __forceinline__ void tm_load8(uint32_t at, float (&v)[16])
{
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(at)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 8 columns at one place, and 8 at another
__device__ __forceinline__ void tm_load8x2(uint32_t at, uint32_t at2, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at), "r"(at2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// s += g * (v * c) on two values at once
__device__ __forceinline__ void add_scaled(float &s0, float &s1, float v0, float v1, float c0, float c1, float g)
{
    asm("{\n\t.reg .b64 s, v, c, g;\n\t"
        "mov.b64 s, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\tmov.b64 g, {%6, %6};\n\t"
        "mul.rn.f32x2 v, v, c;\n\tfma.rn.f32x2 s, g, v, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "f"(v0), "f"(v1), "f"(c0), "f"(c1), "f"(g));
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
__device__ __forceinline__ uint32_t hneg2u(uint32_t a) { return a ^ 0x80008000u; }

// Shared memory by 32-bit address (a pointer rounded up to 1024 bytes is a generic one to the compiler)
__device__ __forceinline__ uint4 lds4(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds4f(uint32_t at)
{
    const uint4 v = lds4(at);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ float lds1f(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ int lds1i(uint32_t at)
{
    int v;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts1(uint32_t at, uint32_t x) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory"); }

// Barriers by 32-bit address too.
#define RZ_BAR(field) (bars + static_cast<uint32_t>(offsetof(Bars, field)))
__device__ __forceinline__ bool try_phase(uint32_t bar, unsigned par)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(par)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool gave_up(uint32_t bars) { return lds1i(RZ_BAR(limit)) == 0; }

// Bounded waits; false after a timeout or when another role gave up.  Short, as there are many of them.
__device__ __forceinline__ bool wait_one(uint32_t bar, unsigned par, uint32_t bars)
{
    for (uint32_t i = 0;; ++i) {
        if (try_phase(bar, par)) return true;
        if ((i & 63u) == 63u && i >= static_cast<uint32_t>(lds1i(RZ_BAR(limit)))) {
            sts1(RZ_BAR(limit), 0);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, unsigned par, uint32_t bars)
{
    // All lanes wait for the same barrier: lanes that wait for different ones drift apart, and what follows (tcgen05.ld, products
    // issued for the warp) needs the warp together.
    const bool ok = __all_sync(0xffffffffu, wait_one(bar, par, bars));
    __syncwarp();
    return ok;
}
// A copy that is under way lands.
__device__ __forceinline__ void wait_landed(uint32_t bar, unsigned par)
{
    for (uint32_t i = 0; i < kWaitLimit && !try_phase(bar, par); ++i) {
    }
}

// A super-block's two scales; wide: the mins' is over 2^13 times the other (see above).
struct Head {
    float d, dmin;
    bool wide, fine;
    // 2^-p; 0 with d = 0
    __device__ __forceinline__ float shrink() const
    {
        if (!wide || !fine) return 1.0f;
        const uint32_t e = (__float_as_uint(__fdiv_rn(dmin, d)) >> 23) & 255u;  // 140 to 166
        return d == 0.0f ? 0.0f : __uint_as_float((127u + 139u - e) << 23);
    }
};
__device__ __forceinline__ Head head_of(uint32_t word)
{
    const float d = h2f(static_cast<uint16_t>(word & 0xffffu)), dmin = h2f(static_cast<uint16_t>(word >> 16));
    return {d, dmin, fabsf(dmin) > 8192.0f * fabsf(d), isfinite(d) && isfinite(dmin)};
}

// Whether the mins' scale is over 2^13 times the other (in f16, where that is exact or infinite)
__device__ __forceinline__ bool mins_are_unit(uint32_t word)
{
    const __half d = __ushort_as_half(static_cast<unsigned short>(word & 0x7fffu)), m = __ushort_as_half(static_cast<unsigned short>((word >> 16) & 0x7fffu));
    return __hgt(m, __hmul(d, __ushort_as_half(0x7000)));
}

// Whether a phase is complete, at once.
__device__ __forceinline__ bool test_phase(uint32_t bar, unsigned par)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(par)
        : "memory");
    return ok != 0;
}

// Tiles of kN rows before each expert, cut to the workspace's (moe_tiles.h), by one warp.
template <int N>
__device__ __forceinline__ void tiles_before(const MoeGemvArgs &g, int *cum, int lane)
{
    const int most = static_cast<int>(moe_most_tiles(g.n_pairs, g.n_experts, N));
    int base = 0;
    for (int e0 = 0; e0 < g.n_experts; e0 += 32) {
        const int e = e0 + lane;
        const int own = e < g.n_experts ? moe_expert_tiles(g.offsets[e], g.offsets[e + 1], g.n_pairs, N) : 0;
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (e < g.n_experts) cum[e] = moe_cut(base + v - own, most);
        base = moe_cut(base + __shfl_sync(0xffffffffu, v, 31), most);
    }
    if (lane == 0) cum[g.n_experts] = base;
}

// B: a CTA has a tile and some of its super-blocks, a warp a row's super-block at a time, a lane 8 codes.
constexpr int kPackThreads = 256;
template <int N>
__global__ void __launch_bounds__(kPackThreads) moe_pack_kernel(const MoeGemvArgs g, uint8_t *__restrict__ pack, float *__restrict__ col_scale)
{
    using C = Cfg<N>;
    __shared__ int cum[kMoeMaxExperts + 1], src[N];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nsb = g.in_dim / 256;
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 0) tiles_before<N>(g, cum, lane);
    __syncthreads();
    const int tile = blockIdx.x;
    if (tile >= cum[g.n_experts]) return;
    const int e = moe_expert_of(tile, cum, g.n_experts), first = g.offsets[e] + (tile - cum[e]) * N, end = g.offsets[e + 1];
    for (int c = tid; c < N; c += kPackThreads) {
        int r = -1;  // the row of x, -1 beyond the expert's
        if (first + c < end) {
            r = first + c;
            if (g.rows) {
                const int pair = g.rows[r];
                const bool fine = pair >= 0 && pair < g.n_pairs;
                if (!fine) set_error(g.err, DEV_BAD_LENGTH);
                r = fine ? pair / g.top_k : 0;
            }
        }
        src[c] = r;
    }
    __syncthreads();
    const int sb0 = blockIdx.y * nsb / gridDim.y, sb1 = (blockIdx.y + 1) * nsb / gridDim.y;
    // eight rows side by side for a warp's stores: lanes have row lane & 7 of 8, and a quarter of its codes at a time
    const int row = lane & 7, quarter = lane >> 3;
    for (int u = warp; u < (sb1 - sb0) * (N / 8); u += kPackThreads / 32) {
        const int sb = sb0 + u / (N / 8), c = u % (N / 8) * 8 + row, r = src[c];
        const int64_t cell = static_cast<int64_t>(tile) * nsb + sb, from = static_cast<int64_t>(max(r, 0)) * nsb + sb;
        uint8_t *to = pack + cell * C::kCellB;
        // this quarter's blocks 2 quarter, 2 quarter + 1
        float2 d = make_float2(0.0f, 0.0f), s = d;
        if (r >= 0) {
            d = __ldg(reinterpret_cast<const float2 *>(g.xd + from * 8) + quarter);
            s = __ldg(reinterpret_cast<const float2 *>(g.xs + from * 8) + quarter);
        }
        uint4 codes[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) codes[k] = r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(g.xq + from * 256 + 64 * quarter + 16 * k)) : make_uint4(0, 0, 0, 0);
        uint32_t top = max(__float_as_uint(d.x) & 0x7fffffffu, __float_as_uint(d.y) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const uint32_t e2 = min(top >> 23, 252u);
        const float up = __uint_as_float((253u - e2) << 23);  // the largest scale becomes 1/2 .. 1
        const float v[4] = {d.x * up, d.y * up, s.x * up * 8.0f, s.y * up * 8.0f};
        float high[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) high[k] = __half2float(__float2half_rn(v[k]));
        // this quarter is a chunk of 64: its high pieces, and how far behind the low ones are (kN rows on, side by side)
        uint8_t *base = to + (c >> 3) * (C::kChunks * 1024) + row * 16 +
                        (C::kStack ? quarter / 2 * C::kSlotB + quarter % 2 * 1024 : C::kMinsB + (4 + quarter) * C::kBytesB);
        constexpr int kLow = C::kStack ? N * 256 : -4 * C::kBytesB;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 16 codes, half a block
            const uint32_t dh = pack2(high[k >> 1], high[k >> 1]), dl = pack2(v[k >> 1] - high[k >> 1], v[k >> 1] - high[k >> 1]);
            const uint32_t words[4] = {codes[k].x, codes[k].y, codes[k].z, codes[k].w};
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // codes as 1024 + 128 + code, which is f16 0x64xx, in the order 0, 2, 1, 3
                const uint32_t w = words[i] ^ 0x80808080u;
                const uint32_t e02 = hsub2u(__byte_perm(w, 0x64646464u, 0x4240), 0x64806480u), e13 = hsub2u(__byte_perm(w, 0x64646464u, 0x4341), 0x64806480u);
                hi[2 * i] = hmul2u(e02, dh);
                hi[2 * i + 1] = hmul2u(e13, dh);
                lo[2 * i] = hfma2u(e02, dl, hfma2u(e02, dh, hneg2u(hi[2 * i])));  // the inner one is exact
                lo[2 * i + 1] = hfma2u(e13, dl, hfma2u(e13, dh, hneg2u(hi[2 * i + 1])));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<uint4 *>(base + (2 * k + i) * 128) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                *reinterpret_cast<uint4 *>(base + kLow + (2 * k + i) * 128) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
            }
        }
        // the high pieces of s, the low ones, and both again: four blocks' beside their chunks, or all eight's
        const uint32_t sh = pack2(high[2], high[3]), sl = pack2(v[2] - high[2], v[3] - high[3]);
        if constexpr (C::kStack) {
            uint8_t *m = to + quarter / 2 * C::kSlotB + C::kBytesB + (c >> 3) * 256 + row * 16 + quarter % 2 * 4;
            *reinterpret_cast<uint32_t *>(m) = sh;
            *reinterpret_cast<uint32_t *>(m + 8) = sl;
            *reinterpret_cast<uint32_t *>(m + 128) = sh;
            *reinterpret_cast<uint32_t *>(m + 136) = sl;
        } else {
            uint8_t *m = to + (c >> 3) * 512 + row * 16 + quarter * 4;
            *reinterpret_cast<uint32_t *>(m) = sh;
            *reinterpret_cast<uint32_t *>(m + 128) = sl;
            *reinterpret_cast<uint32_t *>(m + 256) = sh;
            *reinterpret_cast<uint32_t *>(m + 384) = sl;
        }
        if (quarter == 0) col_scale[cell * N + c] = __uint_as_float((e2 + 1u) << 23);
    }
}

// silu(g) u without branches: e^-|g| <= 1 and a divisor of 1 .. 2, where the fast division is within 2 ulp.  Off by 11 half-ulps at most: 4 of
// expf, 4 of the division, the roundings of g e, 1 + e and the product with u.  (g / (1 + e^-g), whose division has branches: 3145 instead of 2992 us,
// 4096 tokens of 2 in 8 experts, 4096 > 14336; 89 instead of 77 us, 256 of 8 in 64, 2048 > 1024.)
__device__ __forceinline__ float silu_mul_straight(float g, float u)
{
    const float e = expf(-fabsf(g));
    return __fdividef(g >= 0.0f ? g : g * e, 1.0f + e) * u;
}

// A place in a ring of R slots and the parity of its phase.  kFew, where registers are short (tiles of 128 rows): one counter where
// R is a power of two.  With barriers by 32-bit address 3198 to 3002 us (gate and up, 4096 tokens, 8 experts of 14336 x 4096, top 2);
// tiles of 16 rows would lose 2% by the counter.
template <int R, bool kFew>
struct Ring {
    static constexpr bool kCount = kFew && (R & (R - 1)) == 0;
    unsigned n, phase;
    __device__ __forceinline__ explicit Ring(int first) : n(first), phase(0) {}
    __device__ __forceinline__ unsigned slot() const { return kCount ? n & (R - 1) : n; }
    __device__ __forceinline__ unsigned par() const { return kCount ? (n / R) & 1u : phase; }
    __device__ __forceinline__ void add(unsigned by)
    {
        n += by;
        if (!kCount && n >= R) {
            n -= R;
            phase ^= 1u;
        }
    }
};

// Two low codes, v = 1024 + q: sc q = v sc - 1024 sc, or centred sc (q - 8) = (v - 1032) sc (1032 sc is not exact in f16)
template <bool kPlain>
__device__ __forceinline__ uint32_t low_codes(uint32_t v, uint32_t sc, uint32_t add)
{
    return kPlain ? hfma2u(v, sc, add) : hmul2u(hsub2u(v, 0x64086408u), sc);
}

// A slot's codes times 2^-p, of the rows whose mins ask for it: read back and written again.  Rare, and so apart: beside each store it took
// 6 to 7% of the time of all tiles of 16 and 32 rows (instructions that are fetched and not executed).  In two factors, as 2^-25 is none in f16.
template <int kCols>
__device__ __forceinline__ void shrink_codes(uint32_t at, float by)
{
    const float first = fmaxf(by, 0x1p-14f), second = by < 0x1p-14f ? by * 0x1p14f : 1.0f;
    const uint32_t first2 = pack2(first, first), second2 = pack2(second, second);
    tm_store_wait();
#pragma unroll 1
    for (int c = 0; c < kCols; c += 8) {
        float v[16];
        tm_load8(at + c, v);
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = hmul2u(hmul2u(__float_as_uint(v[i]), first2), second2);
        tm_store8(at + c, o);
    }
}

// What a super-block's mins are multiplied by, what the scales that centred codes leave out, and the scale of its row.
struct Mins {
    float by, f, g;
    Mins() = default;
    __device__ __forceinline__ Mins(const uint4 &hd, bool any_wide)
    {
        const Head head = head_of(hd.x);
        float ratio = head.d == 0.0f ? 0.0f : __fdiv_rn(head.dmin, head.d);
        f = 1.0f;
        g = head.d;
        if (any_wide && head.wide) {
            f = head.shrink();
            ratio = head.d == 0.0f ? 1.0f : ratio * f;
            g = head.d == 0.0f ? head.dmin : __fdiv_rn(head.d, f);
        }
        by = head.fine ? -0.125f * ratio : 0.0f;
        g = head.fine ? g : NAN;
    }
    // six-bit mins of sub-blocks 0-3 and 4-7
    static __device__ __forceinline__ uint32_t low(const uint4 &hd) { return hd.z & 0x3f3f3f3fu; }
    static __device__ __forceinline__ uint32_t high(const uint4 &hd) { return ((hd.w >> 4) & 0x0f0f0f0fu) | ((hd.z >> 2) & 0x30303030u); }
};

// Items in parts of in_dim, where whole ones leave SMs without work: the fewest super-blocks on an SM, with three more for each item's
// start and end.  65 tokens of 4 in 16 experts, 4864 > 896: 39.8 to 30.6 us; 33 tokens of 2 in 8, 5632 > 2048: 39.3 to 27.7 us.
__device__ __forceinline__ int parts_of(int64_t items, int nsb, int max_parts)
{
    int best = 1;
    int64_t least = INT64_MAX;
    for (int p = 1; p <= max_parts; ++p) {
        const int per = (nsb + p - 1) / p;
        if ((p - 1) * per >= nsb) continue;  // the last would be empty
        const int64_t t = (items * p + gridDim.x - 1) / gridDim.x * (per + 3);
        if (t < least) {
            least = t;
            best = p;
        }
    }
    return best;
}

template <int N, bool kSwiglu>
__global__ void __launch_bounds__(Cfg<N>::kThreads, 1) moe_gemm_tc_kernel(const __grid_constant__ TcArgs a)
{
    using C = Cfg<N>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    Bars &b = *reinterpret_cast<Bars *>(sm + C::off_bars);
    int *cum = reinterpret_cast<int *>(sm + C::off_cum);
    const uint32_t sm32 = smem_u32(sm), bars = sm32 + C::off_bars;
    const MoeGemvArgs &g = a.g;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int nsb = g.in_dim / 256;
    const int row_tiles = static_cast<int>((g.out_dim + (kSwiglu ? 127 : 255)) / (kSwiglu ? 128 : 256));

    if (tid == 0) {
        for (int i = 0; i < 2 * C::kSlotsA; ++i) {
            mbar_init(&b.a_full[i & 1][i >> 1], 4);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&b.a_empty[i & 1][i >> 1], 1);
        for (int i = 0; i < C::kRingB; ++i) {
            mbar_init(&b.b_full[i], 1);
            mbar_init(&b.b_empty[i], 2);
        }
        for (int i = 0; i < C::kRingRaw; ++i) {
            mbar_init(&b.raw_full[i], 1);
            mbar_init(&b.raw_empty[i], C::kStack ? 4 : 4 * 2);
        }
        for (int i = 0; i < C::kBufD; ++i) {
            mbar_init(&b.d_full[i], 1);
            mbar_init(&b.d_empty[i], 8);
        }
        for (int i = 0; i < kHdr; ++i) {
            mbar_init(&b.h_full[i], 8);
            mbar_init(&b.cs_full[i], 1);
        }
        mbar_init(&b.done[0], 1);
        mbar_init(&b.done[1], 1);
        b.limit = a.stall && blockIdx.x == 0 ? a.stall : kWaitLimit / 8;
        fence_mbar_init();
        tma_prefetch_desc(&a.map1);
        if (kSwiglu) tma_prefetch_desc(&a.map2);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&b.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 1) {
        tiles_before<N>(g, cum, lane);
        if constexpr (!kSwiglu) {
            __syncwarp();
            if (lane == 0) {
                b.parts = parts_of(static_cast<int64_t>(cum[g.n_experts]) * row_tiles, nsb, g.max_parts);
                if (g.max_parts > 1 && blockIdx.x == 0) *g.parts = b.parts;
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    constexpr uint32_t tmem = 0;  // all 512 columns are allocated
    const int64_t whole = static_cast<int64_t>(cum[g.n_experts]) * row_tiles;
    const int parts = kSwiglu ? 1 : b.parts, per = (nsb + parts - 1) / parts;
    const int64_t items = b.tmem == tmem ? whole * parts : 0;
    // this CTA's items, and super-blocks, one after another; the last part's items may be shorter, and come last
    const int my_items = items > blockIdx.x ? static_cast<int>((items - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
    const int64_t full = items > 0 ? items - whole : 0;
    const int my_full = full > blockIdx.x ? static_cast<int>((full - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
    const int rest = nsb - (parts - 1) * per;
    const int64_t blocks = static_cast<int64_t>(my_full) * per + static_cast<int64_t>(my_items - my_full) * rest;

    if (warp < 4) {
        if constexpr (C::kRegsIssue) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsIssue ? C::kRegsIssue : 24));
        if (warp < 2) {
            // -------------------------------------------------------- products of matrix `warp`
            const int mt = warp;
            const uint32_t elected = elect();
            Ring<C::kSlotsA, N == 128> pa(0);
            Ring<C::kRingB, N == 128> pb(0);
            Ring<C::kBufD, N == 128> pd(mt);
            bool ok = true;
            for (int64_t k = 0; k < blocks && ok; ++k) {
                const uint32_t d = tmem + pd.slot() * C::kColsD;
                const Ring<C::kSlotsA, N == 128> first = pa;
#pragma unroll (C::kStack ? 4 : 1)
                for (int entry = 0; entry < C::kEntries; ++entry) {
                    // of A: the next slot, but for the high pieces, which go over the chunks' slots again
                    const bool again = !C::kStack && entry > 4, last = entry == C::kEntries - 1;
                    Ring<C::kSlotsA, N == 128> at = pa;
                    if (again) {
                        at = first;
                        at.add(entry - 4);
                    }
                    // the phases tested together, one latency; what is not complete is waited for
                    const bool ra = again || test_phase(RZ_BAR(a_full) + 32 * mt + 8 * at.slot(), at.par());
                    const bool rb = test_phase(RZ_BAR(b_full) + 8 * pb.slot(), pb.par());
                    const bool rd = entry > 0 || test_phase(RZ_BAR(d_empty) + 8 * pd.slot(), pd.par() ^ 1u);
                    if (!__all_sync(0xffffffffu, ra && rb && rd)) {
                        if (entry == 0 && !(ok = wait_warp(RZ_BAR(d_empty) + 8 * pd.slot(), pd.par() ^ 1u, bars))) break;
                        if (!(ok = wait_warp(RZ_BAR(b_full) + 8 * pb.slot(), pb.par(), bars))) break;
                        if (!again && !(ok = wait_warp(RZ_BAR(a_full) + 32 * mt + 8 * at.slot(), at.par(), bars))) break;
                    }
                    fence_after();
                    const uint32_t ta = tmem + C::kColA + (mt * C::kSlotsA + at.slot()) * C::kWidthA;
                    const uint32_t tb = operand_low(sm32 + C::off_b + pb.slot() * C::kSlotB);
                    if constexpr (C::kStack) {
                        // the mins early: the codes' sums cancel against them as they grow
                        mma_ts(elected, d, ta, tb, operand_high(2048), idesc_f16(2 * N), entry > 0);
                        mma_ts(elected, d, ta + 64, tb + C::kBytesB / 16, operand_high(256), idesc_f16(N), true);
#pragma unroll
                        for (int i = 1; i < 8; ++i) mma_ts(elected, d, ta + 8 * i, tb + 16 * i, operand_high(2048), idesc_f16(2 * N), true);
                    } else if (entry == 0) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) mma_ts(elected, d, ta + 8 * i, tb + 16 * i, operand_high(512), idesc_f16(N), i > 0);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma_ts(elected, d, ta + 8 * i, tb + 16 * i, operand_high(1024), idesc_f16(N), true);
                    }
                    // side by side: the other group writes this slot next, and waits at a barrier of its own
                    const unsigned next = C::kStack ? at.slot() + (k & 1 ? 0 : 2) : at.slot();
                    if (C::kStack || entry == 0 || again) commit(elected, RZ_BAR(a_empty) + 32 * mt + 8 * next);
                    commit(elected, RZ_BAR(b_empty) + 8 * pb.slot());
                    if (last) commit(elected, RZ_BAR(d_full) + 8 * pd.slot());
                    if (!again) pa.add(1);
                    pb.add(1);
                }
                pd.add(2);
            }
            commit(elected, RZ_BAR(done) + 8 * mt);  // every product issued has completed once this arrives
            wait_landed(RZ_BAR(done) + 8 * mt, 0);
        } else if (lane == 0) {
            // -------------------------------------------------------- copies: warp 2 B and the columns' exponents, warp 3 the raw weights
            const uint64_t pol = l2_evict_first_policy();
            const bool weights = warp == 3, stalled = weights && a.stall && blockIdx.x == 0;  // the first weights are not copied
            RingPos p{0, 0}, ph{0, 0};
            int64_t issued = 0, issued_h = 0;
            bool ok = true;
            for (int i = 0; i < my_items && ok; ++i) {
                int64_t it = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
                const int part = parts > 1 ? static_cast<int>(it / whole) : 0;
                it -= part * whole;
                const int first = part * per, end = min(nsb, first + per);
                const MoeItem item = moe_item(it, row_tiles, cum, g.n_experts);
                const int e = item.expert, rt = item.row_tile, tile = item.tile;
                if (weights) {
                    const int row = g.offsets[e] + tile * N;
                    sts4(sm32 + C::off_item + 16 * (i % kItems), row, min(N, g.offsets[e + 1] - row), rt, part);
                    const int y0 = static_cast<int>(e * g.out_dim + static_cast<int64_t>(rt) * (kSwiglu ? 128 : 256));
                    for (int sb = first; sb < end && ok; ++sb) {
                        for (int mt = 0; mt < 2; ++mt) {
                            if (!(ok = wait_one(RZ_BAR(raw_empty) + 8 * p.s, p.par ^ 1u, bars))) break;
                            if (!stalled || issued > 0) {
                                expect_tx(RZ_BAR(raw_full) + 8 * p.s, kRawBytes);
                                copy_box(sm32 + C::off_raw + p.s * kRawBytes, kSwiglu && mt ? &a.map2 : &a.map1, sb * 144,
                                         y0 + (kSwiglu ? 0 : 128 * mt), RZ_BAR(raw_full) + 8 * p.s, pol);
                            }
                            ++issued;
                            ring_next(p, C::kRingRaw);
                        }
                    }
                } else {
                    const int64_t cell0 = static_cast<int64_t>(cum[e] + tile) * nsb;
                    for (int sb = first; sb < end && ok; ++sb) {
                        const uint8_t *from = a.pack + (cell0 + sb) * C::kCellB;
                        for (int entry = 0; entry < C::kEntries; ++entry) {
                            if (!(ok = wait_one(RZ_BAR(b_empty) + 8 * p.s, p.par ^ 1u, bars))) break;
                            const uint32_t bytes = C::kStack ? C::kSlotB : entry == 0 ? C::kMinsB : C::kBytesB;
                            expect_tx(RZ_BAR(b_full) + 8 * p.s, bytes);
                            copy_bulk(sm32 + C::off_b + p.s * C::kSlotB, from, bytes, RZ_BAR(b_full) + 8 * p.s);
                            from += bytes;
                            ++issued;
                            ring_next(p, C::kRingB);
                        }
                        if (!ok) break;
                        expect_tx(RZ_BAR(cs_full) + 8 * ph.s, N * 4);
                        copy_bulk(sm32 + C::off_cs + ph.s * N * 4, a.col_scale + (cell0 + sb) * N, N * 4, RZ_BAR(cs_full) + 8 * ph.s);
                        ++issued_h;
                        ring_next(ph, kHdr);
                    }
                }
            }
            // copies in flight land before the CTA ends
            const int ring = weights ? C::kRingRaw : C::kRingB;
            for (int64_t k = max(static_cast<int64_t>(stalled), issued - ring); k < issued; ++k) {
                const RingPos q = ring_pos(k, ring);
                wait_landed(weights ? RZ_BAR(raw_full) + 8 * q.s : RZ_BAR(b_full) + 8 * q.s, q.par);
            }
            for (int64_t k = max(static_cast<int64_t>(0), issued_h - kHdr); k < issued_h; ++k) {
                const RingPos q = ring_pos(k, kHdr);
                wait_landed(RZ_BAR(cs_full) + 8 * q.s, q.par);
            }
        }
    } else if (warp < C::kFirstSum) {
        // ------------------------------------------------------------ unpacking
        if constexpr (C::kRegsUnpack) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsUnpack ? C::kRegsUnpack : 24));
        // group: matrix, and which of its steps
        const int cw = warp - C::kFirstUnpack, wrow = 32 * (cw & 3) + lane, mt = (cw >> 2) & 1, turn = cw >> 3;
        const uint32_t ta0 = tmem + (static_cast<uint32_t>(32 * (cw & 3)) << 16) + C::kColA + mt * C::kSlotsA * C::kWidthA;
        Ring<C::kRingRaw, N == 128> praw(C::kStack ? mt + 2 * turn : mt);
        Ring<C::kSlotsA, N == 128> pa(C::kStack ? 0 : turn);
        Ring<kHdr, N == 128> ph(C::kStack ? turn : 0);
        // Side by side, a group has every other super-block; else every other slot, over the super-blocks' ends.
        int use = C::kStack ? 0 : turn;
        unsigned before = turn;  // side by side: parity of the phase in which the other group's use of a slot is read
        bool ok = true;
        for (int64_t k = C::kStack ? turn : 0; k < blocks && ok; k += C::kStack ? 2 : 1) {
            if (!(ok = wait_warp(RZ_BAR(raw_full) + 8 * praw.slot(), praw.par(), bars))) break;
            const uint32_t raw = sm32 + C::off_raw + praw.slot() * kRawBytes + wrow * 144;
            const uint4 hd = lds4(raw);
            const bool any_wide = __any_sync(0xffffffffu, mins_are_unit(hd.x));
            // six-bit scales, four to a word: sub-blocks 0-3 and 4-7
            const uint32_t sc0 = hd.y & 0x3f3f3f3fu, sc1 = (hd.w & 0x0f0f0f0fu) | ((hd.y >> 2) & 0x30303030u);
            Mins mins_of;
            if constexpr (C::kStack) mins_of = Mins(hd, any_wide);
#pragma unroll 1
            for (; use < C::kUses; use += C::kStack ? 1 : 2) {
                const bool mins = !C::kStack && use == 0;  // the mins alone
                if constexpr (C::kStack) {
                    if (!(ok = wait_warp(RZ_BAR(a_empty) + 32 * mt + 8 * (use + 2 * turn), before ^ 1u, bars))) break;
                } else {
                    if (!(ok = wait_warp(RZ_BAR(a_empty) + 32 * mt + 8 * pa.slot(), pa.par() ^ 1u, bars))) break;
                }
                fence_after();
                const unsigned slot = C::kStack ? use : pa.slot();
                const uint32_t ta = ta0 + slot * C::kWidthA;
                if (!mins) {
#pragma unroll
                    for (int cc = 0; cc < C::kChunks; ++cc) {
                        const int c = C::kStack ? 2 * use + cc : use - 1;
                        const uint32_t six = (c < 2 ? sc0 : sc1) >> (16 * (c & 1));
                        // the high codes (1024 + 16 q) (sc / 16) - 72 sc = sc (q - 8): one rounding of an exact small integer
                        const uint32_t s0 = hsub2u(__byte_perm(six, 0x64646464u, 0x4040), 0x64006400u);
                        const uint32_t s1 = hsub2u(__byte_perm(six, 0x64646464u, 0x4141), 0x64006400u);
                        const uint32_t add0 = hmul2u(s0, 0xe400e400u);  // * -1024
                        const uint32_t mul1 = hmul2u(s1, 0x2c002c00u), add1 = hmul2u(s1, 0xd480d480u);  // / 16, * -72
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint4 q = lds4(raw + 16 + 32 * c + 16 * half);
                            const uint32_t words[4] = {q.x, q.y, q.z, q.w};
                            uint32_t lo[8], hi[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t w8 = words[i] >> 8;
                                lo[2 * i] = low_codes<C::kStack>(lop_and_or(words[i], 0x000f000fu, 0x64006400u), s0, add0);
                                lo[2 * i + 1] = low_codes<C::kStack>(lop_and_or(w8, 0x000f000fu, 0x64006400u), s0, add0);
                                hi[2 * i] = hfma2u(lop_and_or(words[i], 0x00f000f0u, 0x64006400u), mul1, add1);
                                hi[2 * i + 1] = hfma2u(lop_and_or(w8, 0x00f000f0u, 0x64006400u), mul1, add1);
                            }
                            tm_store8(ta + 32 * cc + 8 * half, lo);
                            tm_store8(ta + 32 * cc + 16 + 8 * half, hi);
                        }
                    }
                    if (any_wide) shrink_codes<32 * C::kChunks>(ta, C::kStack ? mins_of.f : head_of(lds4(raw).x).shrink());
                }
                if (C::kStack || mins) {
                    const uint4 h = C::kStack ? hd : lds4(raw);
                    const Mins of = C::kStack ? mins_of : Mins(h, any_wide);
                    constexpr int kWords = C::kStack ? 2 : 4;  // of two sub-blocks: this slot's, or all
                    uint32_t hi[2 * kWords], lo[2 * kWords];   // high pieces, twice; low ones, twice
#pragma unroll
                    for (int i = 0; i < kWords; ++i) {
                        // two mins, and the scales 8 of which centred codes leave out, as f16 (1024 + m is 0x64 m)
                        const int quad = C::kStack ? use : i >> 1;
                        const uint32_t mm = quad ? Mins::high(h) : Mins::low(h), ss = quad ? sc1 : sc0;
                        const float2 m = unpack2(hsub2u(__byte_perm(mm, 0x64646464u, i & 1 ? 0x4342 : 0x4140), 0x64006400u));
                        const float2 sc = unpack2(hsub2u(__byte_perm(ss, 0x64646464u, i & 1 ? 0x4342 : 0x4140), 0x64006400u));
                        const float r0 = C::kStack ? of.by * m.x : fmaf(of.by, m.x, of.f * sc.x), r1 = fmaf(of.by, m.y, of.f * sc.y);
                        hi[i] = hi[kWords + i] = pack2(r0, r1);
                        const float2 t = unpack2(hi[i]);
                        lo[i] = lo[kWords + i] = pack2(r0 - t.x, r1 - t.y);
                    }
                    if constexpr (C::kStack) {
                        const uint32_t o[8] = {hi[0], hi[1], hi[2], hi[3], lo[0], lo[1], lo[2], lo[3]};
                        tm_store8(ta + 64, o);
                    } else {
                        tm_store8(ta, hi);
                        tm_store8(ta + 8, lo);
                    }
                    if (!C::kStack || use == 1) sts1(sm32 + C::off_g + 4 * ((ph.slot() * 2 + mt) * 128 + wrow), __float_as_uint(of.g));
                }
                tm_store_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive(RZ_BAR(a_full) + 32 * mt + 8 * slot);
                    if (C::kStack ? use == 1 : mins) arrive(RZ_BAR(h_full) + 8 * ph.slot());
                }
                if constexpr (!C::kStack) pa.add(2);
            }
            if (!ok) break;
            if (lane == 0) arrive(RZ_BAR(raw_empty) + 8 * praw.slot());
            use -= C::kUses;
            before ^= 1u;
            ph.add(C::kStack ? 2 : 1);
            praw.add(C::kStack ? 4 : 2);
        }
    } else {
        // ------------------------------------------------------------ sums
        if constexpr (C::kRegsSum) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSum ? C::kRegsSum : 24));
        const int dw = warp - C::kFirstSum, col0 = (dw >> 2) * C::kHalf, wrow = 32 * (dw & 3) + lane;
        const uint32_t at = tmem + (static_cast<uint32_t>(32 * (dw & 3)) << 16) + col0;
        Ring<C::kBufD, N == 128> pd(0);
        Ring<kHdr, N == 128> ph(0);
        bool ok = true;
        for (int item = 0; item < my_items && ok; ++item) {
            float sum[2][C::kHalf];
#pragma unroll
            for (int i = 0; i < C::kHalf; ++i) sum[0][i] = sum[1][i] = 0.0f;
            for (int left = item < my_full ? per : rest; left > 0 && ok; --left) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    if (mt == 0) {
                        ok = wait_warp(RZ_BAR(h_full) + 8 * ph.slot(), ph.par(), bars) &&
                             wait_warp(RZ_BAR(cs_full) + 8 * ph.slot(), ph.par(), bars);
                        if (!ok) break;
                    }
                    if (!(ok = wait_warp(RZ_BAR(d_full) + 8 * pd.slot(), pd.par(), bars))) break;
                    fence_after();
                    const float gs = lds1f(sm32 + C::off_g + 4 * ((ph.slot() * 2 + mt) * 128 + wrow));
                    const uint32_t cs = sm32 + C::off_cs + 4 * (ph.slot() * N + col0);
                    const uint32_t from = at + pd.slot() * C::kColsD;
#pragma unroll
                    for (int i = 0; i < C::kHalf; i += 8) {
                        float v[16];
                        if constexpr (C::kStack) {
                            tm_load8x2(from + i, from + N + i, v);
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] += v[8 + j];
                        } else {
                            tm_load8(from + i, v);
                        }
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            const float4 c = lds4f(cs + 4 * (i + j));
                            add_scaled(sum[mt][i + j], sum[mt][i + j + 1], v[j], v[j + 1], c.x, c.y, gs);
                            add_scaled(sum[mt][i + j + 2], sum[mt][i + j + 3], v[j + 2], v[j + 3], c.z, c.w, gs);
                        }
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(RZ_BAR(d_empty) + 8 * pd.slot());
                    pd.add(1);
                }
                ph.add(1);
            }
            if (!ok) break;  // the same for the warp, as its lanes wait for one another below; else the sums are whole, whatever gave up since
            // ---- outputs: a warp's 32 rows lie side by side in each column's row of y
            struct {
                int row, m, rt, part;
            } w;
            {
                const uint4 t = lds4(sm32 + C::off_item + 16 * (item % kItems));
                w.row = t.x;
                w.m = t.y;
                w.rt = t.z;
                w.part = t.w;
            }
            const int64_t o = static_cast<int64_t>(w.rt) * (kSwiglu ? 128 : 256) + wrow;
            const bool in = o < g.out_dim;
            const int m = w.m - col0;
            int64_t to = static_cast<int64_t>(w.row + col0) * g.out_dim + o;
            if constexpr (kSwiglu) {
                // in place first: half of the registers are free for what follows
#pragma unroll
                for (int i = 0; i < C::kHalf; ++i) sum[0][i] = in ? silu_mul_straight(sum[0][i], sum[1][i]) : 0.0f;
                if (g.y && in) {
                    float *y = g.y + to;
#pragma unroll
                    for (int i = 0; i < C::kHalf; ++i, y += g.out_dim)
                        if (i < m) *y = sum[0][i];
                }
                if (g.yq && in) {  // out_dim is a multiple of 32: all of the warp or none
                    // eight columns in straight code, then the others move up
#pragma unroll 1
                    for (int i0 = 0; i0 < C::kHalf && i0 < m; i0 += 8) {
#pragma unroll
                        for (int i = 0; i < 8; ++i, to += g.out_dim) {
                            if (i0 + i >= m) break;
                            const float v = sum[0][i];
                            // as in moe_gemv.cu: a block with a NaN has the scale NaN
                            const float d = __fdiv_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v)))), 127.0f);
                            const int code = q8_code(v, q8_scale(d));
                            const int total = __reduce_add_sync(0xffffffffu, code);
                            g.yq[to] = static_cast<int8_t>(code);
                            if (lane == 0) {
                                g.yd[to / 32] = d;
                                g.ys[to / 32] = __fmul_rn(d, static_cast<float>(total));
                            }
                        }
#pragma unroll
                        for (int i = 0; i + 8 < C::kHalf; ++i) sum[0][i] = sum[0][i + 8];
                    }
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    float *y = g.y + w.part * static_cast<int64_t>(g.n_pairs) * g.out_dim + to + 128 * mt;
                    if (o + 128 * mt < g.out_dim) {
#pragma unroll
                        for (int i = 0; i < C::kHalf; ++i, y += g.out_dim)
                            if (i < m) *y = sum[mt][i];
                    }
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    if (tid == 0 && gave_up(bars)) set_error(g.err, DEV_TIMEOUT_MOE);
    if (warp == 0) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(b.tmem) : "memory");
    }
}

template <int N, bool kSwiglu>
cudaError_t launch(const TcArgs &a, cudaStream_t s)
{
    using C = Cfg<N>;
    cudaError_t e = cudaFuncSetAttribute(moe_gemm_tc_kernel<N, kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(dev_info().sm_count));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, moe_gemm_tc_kernel<N, kSwiglu>, a);
}

}  // namespace

namespace {
template <int N>
int64_t pack_bytes(int64_t n_pairs, int n_experts, int64_t in_dim)
{
    return moe_most_tiles(n_pairs, n_experts, N) * (in_dim / 256) * (Cfg<N>::kCellB + N * 4);
}

template <int N>
cudaError_t launch_all(const MoeGemvArgs &g, void *workspace, cudaStream_t s)
{
    using C = Cfg<N>;
    TcArgs a{};
    a.g = g;
    const int nsb = g.in_dim / 256;
    const int64_t tiles = moe_most_tiles(g.n_pairs, g.n_experts, N);
    uint8_t *pack = static_cast<uint8_t *>(workspace);
    float *col_scale = reinterpret_cast<float *>(pack + tiles * nsb * C::kCellB);
    a.pack = pack;
    a.col_scale = col_scale;
    a.stall = g_stall_next_moe;
    g_stall_next_moe = 0;  // one product only
    const uint64_t row_bytes = static_cast<uint64_t>(nsb) * 144, rows = static_cast<uint64_t>(g.n_experts) * g.out_dim;
    cudaError_t e = encode_tensor_map_2d(&a.map1, g.w1, 1, row_bytes, rows, row_bytes, 144, 128);
    if (e == cudaSuccess && g.w2) e = encode_tensor_map_2d(&a.map2, g.w2, 1, row_bytes, rows, row_bytes, 144, 128);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(std::min<int64_t>(nsb, std::max<int64_t>(1, 2048 / tiles))));
    cfg.blockDim = dim3(kPackThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_use_pdl ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, moe_pack_kernel<N>, g, pack, col_scale);
    if (e != cudaSuccess) return e;
    return g.w2 ? launch<N, true>(a, s) : launch<N, false>(a, s);
}
}  // namespace

int64_t moe_pack_bytes(int columns, int64_t n_pairs, int n_experts, int64_t in_dim)
{
    switch (columns) {
        case 16: return pack_bytes<16>(n_pairs, n_experts, in_dim);
        case 32: return pack_bytes<32>(n_pairs, n_experts, in_dim);
        case 128: return pack_bytes<128>(n_pairs, n_experts, in_dim);
        default: return 0;
    }
}

cudaError_t launch_moe_gemm_tc(const MoeGemvArgs &g, int columns, void *workspace, cudaStream_t s)
{
    switch (columns) {
        case 16: return launch_all<16>(g, workspace, s);
        case 32: return launch_all<32>(g, workspace, s);
        default: return launch_all<128>(g, workspace, s);
    }
}

// Tiles by the rows that an expert has on average (us in a graph, tiles of 16 | 32 | 128 rows; experts chosen evenly, and unevenly: logits
// with a normal part of their own for each expert).  0: fewer rows than experts, which are for the integer dots.
//   gate and up, 2 of 8 experts of 4096 > 14336
//      6 rows: 114, 114 | 127, 126;   8 rows: 115, 123 | 127, 126;   10 rows: 123, 140 | 127, 127
//      75 rows: 354, 346 | 372, 482;  100 rows: 434, 444 | 375, 513;  128 rows: 533, 526 | 519, 547
//   gate and up, 8 of 64 experts of 2048 > 1024
//      8 rows: 49, 48 | 56, 44;  12 rows: 49, 58 | 57, 56;  80 rows: 132, 132 | 149, 184;  96 rows: 147, 147 | 151, 186;  128 rows: 187, 191 | 198, 221
//   down, 8 of 64, 1024 > 2048, half unevenly:  8 rows: 33 | 38;  64 rows: 67 | 90;  128 rows: 113 | 128;  160 rows: 137 | 146;  512 rows: 393 | 357
// Which of the two a batch is, only the device knows: few large experts of some 100 rows, met evenly, would be 14% faster in tiles of 128; met
// unevenly they are 13 to 16% faster as it is.
int moe_tiles(int64_t n_pairs, int n_experts, bool gate_up)
{
    const int64_t rows = n_pairs / n_experts;
    return rows < 1 ? 0 : rows <= 10 ? 16 : rows < (gate_up ? 128 : 192) ? 32 : 128;
}

// The tiles, or 0, integer dots, where they would be tiles of 16 and rows and weights are so few that their time is less.  In us, of 304 CTAs side
// by side, each a round of 8 super-blocks after the other; and of 152, by super-block, of the experts that are met if all
// are as likely, after some 17 us for B's pieces, starts and ends.  152 (and 304) are GB300's SMs: constants, as the queries of workspaces
// make the same choice and ask no device.  Measured (dots | tiles of 16):
//   gate and up, 2 of 8, 4096 > 14336:  1 row 86 | 70;  1.5 rows 126 | 88;  2 rows 165 | 97;   8 of 64, 2048 > 1024:  1 row 32 | 33;
//   1.5 rows 46 | 38;  2 rows 59 | 38;   8 of 128, 2048 > 768:  1 row 46 | 42;  1.5 rows 67 | 51
//   down, 2 of 8, 14336 > 4096:  1 row 46 | 46;  1.5 rows 66 | 57;  2 rows 83 | 57;   8 of 64, 1024 > 2048:  1 row 37 | 27;
//   4 of 16, 4864 > 896:  1 row 12 | 22;  2 rows 18 | 25;  3 rows 26 | 26;   2 of 8, 512 > 1024:  2 rows 6 | 11;   1 of 4, 768 > 512:  3 rows 3 | 11
int moe_columns(int64_t n_pairs, int n_experts, int top_k, int64_t out_dim, int64_t in_dim, bool gate_up)
{
    const int columns = moe_tiles(n_pairs, n_experts, gate_up);
    if (columns != 16) return columns;
    const double nsb = in_dim / 256, met = n_experts * (1.0 - pow(1.0 - 1.0 / n_experts, static_cast<double>(n_pairs)));
    const int of_cta = gate_up ? 32 : 4 * moe_down_quads(top_k);
    const double ctas = static_cast<double>(gate_up ? n_pairs : n_pairs / top_k) * ((out_dim + of_cta - 1) / of_cta);
    const double dots = 3.0 + std::max(1.0, ctas / 304) * (gate_up ? 2 : 1) * (0.8 + 1.5 * ceil(nsb / 8));
    const double items = met * ((out_dim + (gate_up ? 127 : 255)) / (gate_up ? 128 : 256));
    return dots <= 17.0 + nsb * std::max(gate_up ? 1.0 : 0.25, items / 152) ? 0 : columns;
}

// Parts of in_dim are for products that may come to fewer than two items an SM.
int moe_max_parts(int columns, int64_t n_pairs, int64_t out_dim, int64_t in_dim)
{
    if (columns == 0) return 1;
    const int64_t least = (n_pairs + columns - 1) / columns * ((out_dim + 255) / 256);
    return static_cast<int>(std::max<int64_t>(1, std::min({int64_t(8), in_dim / 512, 2 * 152 / least})));
}

}  // namespace rz
