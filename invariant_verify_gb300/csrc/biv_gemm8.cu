// No-split-K GEMM of e4m3 operands with a scale for every 128 terms, on the
// 5th-generation tensor cores (tcgen05 + TMEM), fed by TMA:
//   C[m][n] = act(sum_b sa[b][m] sb[n / 128][b] sum_{k in block b} A[m][k] B[n][k] + bias[n]) + residual[m][n]
//
// The tensor core sums one k-block of 128 terms (four MMAs of K = 32) into an
// accumulator in TMEM that starts at zero; the epilogue warps read it, multiply it by the
// two scales and add it to fp32 sums in their registers, block by block in increasing k.
// That order, and a row's bits, do not depend on M or on the tile.  So the work of the CUDA
// cores goes with the tensor core's: 128 x 256 a CTA and k-block are 128 fused multiply-adds
// a thread (in pairs, fma.rn.f32x2, they take nearly twice as long), some 360 cycles with
// the reads of TMEM, beside 517 of the MMAs.
//
// A row of A is a lane of the accumulator, so that a thread's scale is one number for 128
// columns.  (With the weights along the lanes M need not be a multiple of 128, but every column
// has its own scale, from shared memory: 840 cycles a k-block instead of 590.)
//
// What it comes to, and what is left of it without the copies, without the MMAs, without the sums; copies alone, MMAs
// alone, the hand-overs of stages and sets alone (us; these three without the stores):
//   1024 x 4096 x 14336 (1.91 PFLOP/s)    62.9; 57.1, 55.4, 45.3; 32.6, 35.6, 25.1
//   320 x 128256 x 4096, fp32 C          236.1; 215.5, 196.1, 200.5; 120.5, 103.5, 66.4
//   64 x 4096 x 14336                     20.8; 18.8, 18.7, 18.4; 16.0, 16.2, 9.1
//   8 x 6144 x 4096                        9.4; 7.6, 8.3, 8.0; 6.1, 6.1, 3.7
// So no part alone bounds it.  Wide tiles: an accumulator's way from the MMAs to the sums and back is hidden only by the
// other one.  The head: that, stages of 96 KB of which two fit, and the stores.  Few rows: a CTA's copies (56 boxes of some
// 280 ns for 64 x 4096 x 14336) and its narrow MMAs take three quarters of the time each, on the same hand-overs.
//
// Kernel layout (384 threads, one CTA per SM, persistent over tiles):
//   warp 0      TMA producer: boxes of NB k-blocks, 128-byte swizzle
//   warps 1, 2  MMA issuers, which take the stages in turn: one warp's waits and commits take some 300
//               cycles a k-block, in which the MMAs that it has queued run out.  Stages and sets are even
//               in number, so that each has its own, and every wait is for the phase after one that the
//               same warp has seen: a parity cannot tell phases apart that are two away
//   warps 4..   sums and stores: two warps per TMEM lane quarter, which share the columns
// TMEM holds kSets sets of NB k-blocks' accumulators: one is read while others are filled.
// CG = 1: a CTA per tile of 128 rows.  CG = 2: a pair per tile of 256 (cta_group::2): each CTA copies its
// 128 rows of A and half of the BN rows of B, the even one issues the MMAs.
#include <algorithm>
#include <type_traits>

#include "biv_act.cuh"
#include "biv_e4m3.cuh"

namespace biv {
namespace {

BIV_DEFINE_ERR_WORD(g_gemm8_err)

constexpr int kLanes = 128;                   // rows of an accumulator in one CTA
constexpr int kBK = 128;                      // a k-block: 128 e4m3, one swizzle row and one scale
constexpr int kMaxStages = 16;
constexpr int kIssuers = 2;
constexpr int kEpilogue = 256;                // epilogue threads
constexpr int kThreads = 128 + kEpilogue;
// Registers of a thread after the start, where each has the 168 that 384 threads leave: the first
// warpgroup gives up what the sums need (128 x 40 + 256 x 232 = 384 x 168).
constexpr int kRegsStart = 168, kRegsFew = 40, kRegsMany = 232;
static_assert(128 * kRegsFew + kEpilogue * kRegsMany <= kThreads * kRegsStart, "more registers than the CTA holds");
constexpr int kBarBytes = 512;
constexpr int kPageBlocks = 16;               // k-blocks whose scales are copied at once
constexpr int kPageFloats = kPageBlocks * (kLanes + 4);
// A scale that, times the quantiser's least, is a normal number: 2^-26.
constexpr float kMuchLarger = 1.4901161193847656e-08f;
constexpr int kSlack = kLanes * kBK;          // an MMA may read 128 rows past the last stage
constexpr int kMaxSmem = 227 * 1024 - 1024;
constexpr int kRing = kMaxSmem - 1024 - kBarBytes - 2 * kPageFloats * 4;

struct Gemm8Args {
    const float* sa;                          // [KB][M]
    const float* sb;                          // [ceil(N / 128)][KB]
    void* C;
    BiasActArgs ba;
    int M, N, K, KB;                          // k-blocks
    int f32;
    int wide;                                 // C's rows are 32-byte aligned
    int BN, stages;                           // tile width, stages
    int xr, yr;                               // rows of a CTA's boxes of A and of B
    int m_tiles, tiles;
    int boxes;                                // of a stage and operand: 1, or all where K % 128 != 0
    uint32_t idesc;
};

// PARTS: 16-column parts of a thread (half of BN, rounded up).  DEEP: sets of one k-block, four of them, where two of two
// would fit as well.
template <int PARTS, bool DEEP>
struct Form {
    static constexpr int kCols = 32 * PARTS;  // the widest BN
    // K-blocks of a set of accumulators; the sets are taken in turn.  Where a set is one k-block a stage holds two
    // sets, since a box costs the TMA unit some 280 ns whatever its size (1024 x 4096 x 14336: with boxes of one k-block
    // 79 us where this took 65).
    static constexpr int kBlocks = kCols <= 64 ? 4 : kCols <= 128 && !DEEP ? 2 : 1;
    static constexpr int kStageSets = kBlocks == 1 ? 2 : 1, kStage = kBlocks * kStageSets;
    static constexpr int kSets = kCols <= 32 || DEEP ? 4 : 2;
    static constexpr int kSetCols = 512 / kSets;
    // A barrier of the summing threads and a vote: true if every one says so.
    BIV_DEV static bool all_say(bool ok) {
        uint32_t r;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(r)
                     : "r"(ok ? 1u : 0u), "n"(kEpilogue)
                     : "memory");
        return r != 0;
    }
};

// The four MMAs of a k-block into an accumulator that starts at zero, by one elected lane of a converged warp
// (one election for the four: 7 % of a small product's time).  +32 bytes along K inside the swizzle
// row are +2 in the descriptors' 16-byte units.
#define BIV_MMA_BLOCK(CG)                                                                                       \
    "{\n\t.reg .pred e, pt, pf;\n\t.reg .b64 x1, x2, x3, y1, y2, y3;\n\t"                                        \
    "setp.eq.u32 pt, 0, 0;\n\tsetp.ne.u32 pf, 0, 0;\n\t"                                                        \
    "add.s64 x1, %1, 2;\n\tadd.s64 y1, %2, 2;\n\tadd.s64 x2, %1, 4;\n\tadd.s64 y2, %2, 4;\n\t"                   \
    "add.s64 x3, %1, 6;\n\tadd.s64 y3, %2, 6;\n\telect.sync _|e, 0xffffffff;\n\t"                               \
    "@e tcgen05.mma.cta_group::" CG ".kind::f8f6f4 [%0], %1, %2, %3, pf;\n\t"                                   \
    "@e tcgen05.mma.cta_group::" CG ".kind::f8f6f4 [%0], x1, y1, %3, pt;\n\t"                                   \
    "@e tcgen05.mma.cta_group::" CG ".kind::f8f6f4 [%0], x2, y2, %3, pt;\n\t"                                   \
    "@e tcgen05.mma.cta_group::" CG ".kind::f8f6f4 [%0], x3, y3, %3, pt;\n\t}\n"
template <int CG>
BIV_DEV void mma_block(uint32_t d, uint64_t x, uint64_t y, uint32_t idesc) {
    if constexpr (CG == 2)
        asm volatile(BIV_MMA_BLOCK("2")::"r"(d), "l"(x), "l"(y), "r"(idesc) : "memory");
    else
        asm volatile(BIV_MMA_BLOCK("1")::"r"(d), "l"(x), "l"(y), "r"(idesc) : "memory");
}

// Arrive once on `bar` (of both CTAs of a pair) when the MMAs issued so far by the elected lane complete.
template <int CG>
BIV_DEV void commit(uint64_t* bar) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred e;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        umma_commit_elect(bar);
}

// A bounded wait of a whole warp (shared-memory address).  The loop holds nothing but the poll: a k-block takes
// some 600 cycles, and what stands between a phase and the work behind it is seen in each (a vote on the
// outcome: 100).  Where the wait runs out it sets the CTA's abort flag and returns all the same; each loop
// reads the flag before its wait, which costs nothing, and leaves after it: all lanes together, and at most one
// block of work later than they could.
BIV_DEV void warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    int polls = kFastPolls;
    uint32_t ok;
#pragma unroll 1
    do {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    } while (!ok && --polls);
    if (!ok) mbar_wait(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(bar)), parity, abort_flag, &g_gemm8_err);
}
BIV_DEV float ld_shared(uint32_t at) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
}

// Four bytes to shared memory, zero where there are none to read.
BIV_DEV void copy_4(float* dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// What a block's sums are multiplied by: scale * lift is the product a * b of its two scales.  lift is 1, and scale
// a * b itself, where that is a normal number; a product below them (down to 2^-200) loses bits, one above is infinite
// (and times a sum of zero NaN), though the sums, of 2^-18 to 2^25, may bring the result back.  There lift is a power of
// two, by which a sum is multiplied first: 2^-80 exactly, and 2^112 exactly or, if that is infinite, the result is too.
struct BlockScale {
    float scale, lift;
    BIV_DEV BlockScale(float a, float b) : scale(a * b), lift(1.0f) {
        const uint32_t bits = __float_as_uint(scale) << 1;
        if (bits - 0x01000000u >= 0xfe000000u) {
            const bool small = fabsf(scale) < 1.0f;
            lift = small ? 8.271806125530277e-25f : 5.192296858534828e+33f;                    // 2^-80, 2^112
            const float part = small ? 1.099511627776e+12f : 1.3877787807814457e-17f;          // 2^40, 2^-56
            scale = (a * part) * (b * part);
            // both the quantiser's least: sums times 2^-200 are less than half of the smallest number, and their sign is
            // not to turn a sum of 0 to -0 on such a page and not on another
            if (small && fabsf(scale) < 1.504632769052528e-36f) scale = 0.0f;                  // 2^-119
        }
    }
};

// The smallest and the largest of the scales above `skip`, which lie in the order of their bits; zeros (rows and columns
// that there are none of) aside, and what is below zero, or not finite, counts as too large.
struct ScaleRange {
    uint32_t skip;                           // its bits
    uint32_t over = 0xffffffffu, hi = 0u;    // by how much the smallest lies over skip, less one; the largest
    BIV_DEV void add(float x) {
        over = min(over, __float_as_uint(x) - skip - 1u);
        hi = max(hi, __float_as_uint(x));
    }
    BIV_DEV bool within(float least) const { return over >= __float_as_uint(least) - skip - 1u && hi < __float_as_uint(9.223372036854775808e18f); }      // 2^63
};

// Eight words to memory, 32-byte aligned: a thread has a row, so that a warp's store meets 32 lines whatever its
// width (16 bytes: 320 x 128256 x 4096 271 us, 237 so; through shared memory to 64 bytes a row 247 where this took 234).
BIV_DEV void st_global_32(void* p, const uint32_t (&x)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]),
                 "r"(x[6]), "r"(x[7])
                 : "memory");
}

// A thread's row: PARTS x 16 columns from col0 on (the first `cols` of them) to C.
template <bool F32, int PARTS>
BIV_DEV void put_row(const float (&acc)[PARTS][16], int row, int col0, int cols, const Gemm8Args& g) {
    if (row >= g.M) return;
    const bool plain = !g.ba.bias && !g.ba.residual && g.ba.act == BIV_ACT_NONE;
    uint8_t* dst = static_cast<uint8_t*>(g.C) + (static_cast<long long>(row) * g.N + col0) * (F32 ? 4 : 2);
    const int n = min(cols, g.N - col0);       // columns that there are: a multiple of 8
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        if (16 * i >= n) break;
        float x[2][8];
        if (plain) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e >> 3][e & 7] = acc[i][e];
        } else {
            const BiasActRow operands(true, row, col0 + 16 * i, g.N, g.ba);
            operands.values([&](int e) { return acc[i][e]; }, g.ba, x);
        }
        uint8_t* at = dst + 16 * i * (F32 ? 4 : 2);
        if constexpr (F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (16 * i + 8 * h >= n) break;
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(x[h][e]);
                if (g.wide) {
                    st_global_32(at + 32 * h, y);
                } else {
                    *reinterpret_cast<uint4*>(at + 32 * h) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(at + 32 * h + 16) = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
        } else {
            const uint4 a = BiasActRow::pack8(x[0]), b = BiasActRow::pack8(x[1]);
            if (g.wide && 16 * i + 8 < n) {
                const uint32_t y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                st_global_32(at, y);
            } else {
                *reinterpret_cast<uint4*>(at) = a;
                if (16 * i + 8 < n) *reinterpret_cast<uint4*>(at + 16) = b;
            }
        }
    }
}

// WHOLE: BN = 256, so that a warp's columns lie in one 128-column block of weights.
template <int CG, int PARTS, bool WHOLE, bool DEEP>
__global__ void __launch_bounds__(kThreads, 1) gemm_e4m3_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                                                                const Gemm8Args g) {
    using Q = Form<PARTS, DEEP>;
    constexpr int NB = Q::kBlocks, KS = Q::kStage;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int A_BYTES = KS * g.xr * kBK, STAGE = A_BYTES + KS * g.yr * kBK, S = g.stages;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * STAGE + (g.xr < kLanes ? kSlack : 0));
    uint64_t* empty = full + kMaxStages;
    uint64_t* tfull = empty + kMaxStages;     // [kSets]
    uint64_t* tempty = tfull + Q::kSets;      // [kSets]
    uint64_t* drain = tempty + Q::kSets;      // [kIssuers]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + kIssuers);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float(*s_page)[kPageFloats] = reinterpret_cast<float(*)[kPageFloats]>(reinterpret_cast<uint8_t*>(full) + kBarBytes);   // [2]

    const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / CG, n_units = static_cast<int>(gridDim.x) / CG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_stages = (g.KB + KS - 1) / KS;                   // of a tile
    // epilogue warps with rows to read: all, or those of the quarters that M reaches
    const int readers = CG == 2 ? 16 : 2 * min(4, (g.M + 31) / 32);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], Q::kStageSets);      // commits of the issuers that read it
        }
        for (int a = 0; a < Q::kSets; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], readers);
        }
        for (int i = 0; i < kIssuers; ++i) mbar_init(&drain[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(tmem_slot, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // weights: read once, or by the CTAs of all rows at about the same time; activations: by every CTA
    const uint64_t pol_w = g.m_tiles == 1 ? policy_evict_first() : policy_evict_normal(), pol_a = policy_evict_last();
    auto load = [&](const CUtensorMap* map, uint8_t* dst, int stage, int row, int rows, int sb, uint64_t pol) {
        const bool whole = g.K % kBK == 0;
        for (int j = 0; j < g.boxes; ++j) {
            const int c0 = whole ? 0 : (sb * KS + j) * kBK, c2 = whole ? sb * KS : 0;
            if constexpr (CG == 2)
                tma_load_3d_pair(dst + j * rows * kBK, map, mapa_shared(&full[stage], 0), c0, row, c2, pol);
            else
                tma_load_3d(dst + j * rows * kBK, map, &full[stage], c0, row, c2, pol);
        }
    };
    // tile t: rows (t % m_tiles), columns (t / m_tiles)
    auto load_a = [&](int t, int sb, int stage) {
        load(&tmA, smem + stage * STAGE, stage, (t % g.m_tiles) * (kLanes * CG) + rank * kLanes, g.xr, sb, pol_a);
    };
    auto load_b = [&](int t, int sb, int stage) {
        load(&tmB, smem + stage * STAGE + A_BYTES, stage, (t / g.m_tiles) * g.BN + rank * g.yr, g.yr, sb, pol_w);
    };
    auto expect = [&](int stage) {            // a pair's copies all complete on the even CTA's barrier
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(CG * STAGE));
    };
    // The weights are no output of the previous kernel: the first stages' are asked for before waiting for it.
    int early = 0;
    if (warp == 0 && lane == 0 && unit < g.tiles) {
        early = min(S, n_stages);
        for (int sb = 0; sb < early; ++sb) {
            expect(sb);
            load_b(unit, sb, sb);
        }
    }
    pdl_wait();
    pdl_trigger();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int t = unit; t < g.tiles && ok; t += n_units)
                for (int sb = 0; sb < n_stages; ++sb) {
                    ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_gemm8_err);
                    if (!ok) break;
                    if (t != unit || sb >= early) {
                        expect(stage);
                        load_b(t, sb, stage);
                    }
                    load_a(t, sb, stage);
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            if (!ok) {
                // let the copies that may still be in flight land before the CTA exits
                if (rank == 0) {
                    for (long long i = issued > S ? issued - S : 0; i < issued; ++i)
                        mbar_wait_drain(&full[i % S], static_cast<uint32_t>((i / S) & 1));
                } else {
                    // the odd CTA's complete on the even CTA's barriers: give them time
                    const uint64_t t0 = globaltimer();
                    while (globaltimer() - t0 < 50000ull) {
                    }
                }
            }
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // -------------------------------------------------- MMA issuers
            // Stages and sets taken in turn: issuer 0 the even ones, 1 the odd ones; or of every stage's two sets one each.
            const int me = warp - 1;
            constexpr int kStep = Q::kStageSets == 2 ? 1 : kIssuers;
            const int first = Q::kStageSets == 2 ? 0 : me, j0 = Q::kStageSets == 2 ? me * NB : 0;
            const int unit_tiles = unit < g.tiles ? (g.tiles - unit + n_units - 1) / n_units : 0;
            const long long all = static_cast<long long>(unit_tiles) * n_stages;
            int stage = first, set = me, sb = first % n_stages;      // sb: the stage's place in its tile
            uint32_t phase = 0, set_phase = 0;
            bool ok = true, any = false;
            const uint32_t full0 = smem_u32(full), tempty0 = smem_u32(tempty);
            const uint32_t a_step = static_cast<uint32_t>(g.xr * kBK / 16), b_step = static_cast<uint32_t>(g.yr * kBK / 16);      // of a k-block
            const uint64_t a0 = sw128_kmajor_desc(smem_u32(smem)) + j0 * a_step, b0 = sw128_kmajor_desc(smem_u32(smem + A_BYTES)) + j0 * b_step;
            for (long long c = first; c < all; c += kStep) {
                const int nkb = min(NB, g.KB - sb * KS - j0);        // none: the second set of a last stage that is not full
                const bool stop = *abort_flag;
                warp_wait(full0 + 8u * stage, phase, abort_flag);
                if (nkb > 0) warp_wait(tempty0 + 8u * set, set_phase ^ 1u, abort_flag);
                if (stop) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = static_cast<uint32_t>(stage * (STAGE / 16)), d = tmem_base + static_cast<uint32_t>(set * Q::kSetCols);
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    if (j < nkb) mma_block<CG>(d + static_cast<uint32_t>(j * g.BN), a0 + at + j * a_step, b0 + at + j * b_step, g.idesc);
                if (nkb > 0) {
                    commit<CG>(&tfull[set]);
                    if ((set += kIssuers) >= Q::kSets) {
                        set = me;
                        set_phase ^= 1u;
                    }
                }
                commit<CG>(&empty[stage]);
                any = true;
                if ((stage += kStep) >= S) {
                    stage = first;
                    phase ^= 1u;
                }
                for (sb += kStep; sb >= n_stages;) sb -= n_stages;
            }
            if (!ok && any) {                 // all MMAs issued so far have finished
                commit<CG>(&drain[me]);
                if (lane == 0) mbar_wait_drain(&drain[me], 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------- sums and stores
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        const int q = warp & 3, tid = static_cast<int>(threadIdx.x) - 128;
        const int cb = (warp / 4 - 1) * 16 * PARTS;                     // this warp's first column of the tile
        const bool reads = CG == 2 || q * 32 < g.M;
        const int sets = (g.KB + NB - 1) / NB, pages = (g.KB + kPageBlocks - 1) / kPageBlocks;
        constexpr int kPageSets = kPageBlocks / NB;
        // Scales of a page of tile t: [k-block][row] sa, then [k-block][4] sb of the tile's 128-column blocks.
        auto fetch = [&](int t, int page, float* dst) {
            const int row = (t % g.m_tiles) * (kLanes * CG) + rank * kLanes + (tid & (kLanes - 1)), kb0 = page * kPageBlocks;
            int kb = kb0 + tid / kLanes;
            const float* src = g.sa + static_cast<long long>(kb) * g.M + row;
#pragma unroll
            for (int i = 0; i < kPageBlocks / 2; ++i, kb += 2, src += 2LL * g.M) {
                const bool in = kb < g.KB && row < g.M;
                copy_4(dst + i * kEpilogue + tid, in ? src : g.sa, in);
            }
            if (tid < 4 * kPageBlocks) {
                const int nblk = (t / g.m_tiles) * g.BN / 128 + (tid & 3);
                kb = kb0 + tid / 4;
                const bool in = kb < g.KB && nblk < (g.N + 127) / 128;
                copy_4(dst + kPageBlocks * kLanes + tid, in ? g.sb + static_cast<long long>(nblk) * g.KB + kb : g.sb, in);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const uint32_t tfull0 = smem_u32(tfull), pages0 = smem_u32(&s_page[0][0]);
        uint32_t freed = smem_u32(tempty);    // the sets' barriers where the MMAs are issued
        if constexpr (CG == 2) freed = mapa_shared(tempty, 0);
        // The set of a tile's next k-blocks: in turn, or where a stage holds two, in turn among the even ones for its
        // first and among the odd ones for its second, which a tile's last stage may lack.
        int next[2] = {0, 1}, buf = 0;
        uint32_t phases = 0;                  // bit a: the phase of set a
        bool ok = true;                       // a wait ran out: the warps leave together, at the next vote
        if (unit < g.tiles) fetch(unit, 0, s_page[0]);
        for (int t = unit; t < g.tiles; t += n_units) {
            const int n0 = (t / g.m_tiles) * g.BN;
            float acc[PARTS][16];
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
            // the warp's columns lie in two 128-column blocks of weights at most: the first one, and its parts
            const int blk = (n0 + cb) / 128 - n0 / 128, turn = (128 - (n0 + cb) % 128) / 16;         // the first one, and its parts
            auto set_read = [&](int set) {    // the MMAs may have it again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_remote(freed + 8u * set);
                    else
                        mbar_arrive(&tempty[set]);
                }
            };
            // The sets [s0, s1) of a page.  lifted: products of its scales lie outside the normal numbers; then the sums go
            // through memory, so that the other loop has the registers as if it were alone (1023 x 14336 x 4096: 59.6 us; one
            // loop with a branch in it 67.2, two that share the sums' registers 61.7, without the check 58.9; 625
            // with far scales everywhere).
            auto page_sets = [&](auto lifted, int s0, int s1) {
#pragma unroll 1
                for (int s = s0; s < s1; ++s) {
                    const int in_page = s - s0, nkb = min(NB, g.KB - s * NB);
                    const int second = Q::kStageSets == 2 ? s & 1 : 0, set = second ? next[1] : next[0];
                    if (reads) {
                        const uint32_t row_scale = pages0 + static_cast<uint32_t>((buf ^ 1) * kPageFloats + in_page * NB * kLanes + q * 32 + lane) * 4u;
                        const uint32_t col_scale = pages0 + static_cast<uint32_t>((buf ^ 1) * kPageFloats + kPageBlocks * kLanes + in_page * NB * 4 + blk) * 4u;
                        ok = !*abort_flag;
                        warp_wait(tfull0 + 8u * set, (phases >> set) & 1u, abort_flag);
                        tc_fence_after();
                        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(set * Q::kSetCols + cb);
                        if constexpr (lifted) {
                            float4 sums[4 * PARTS];
#pragma unroll
                            for (int i = 0; i < 4 * PARTS; ++i) {
                                const float* x = &acc[i / 4][i % 4 * 4];
                                sums[i] = make_float4(x[0], x[1], x[2], x[3]);
                            }
#pragma unroll 1
                            for (int kl = 0; kl < nkb; ++kl) {
                                const float mine = ld_shared(row_scale + kl * kLanes * 4u);
                                const BlockScale x0(mine, ld_shared(col_scale + kl * 16u)), x1(mine, ld_shared(col_scale + kl * 16u + (WHOLE ? 0u : 4u)));
#pragma unroll 1
                                for (int i = 0; i < PARTS; ++i) {
                                    uint32_t r[16];
                                    tmem_ld16_sync(taddr + static_cast<uint32_t>(kl * g.BN + 16 * i), r);
                                    const float x = i < turn ? x0.scale : x1.scale, lift = i < turn ? x0.lift : x1.lift;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        float4& y = sums[4 * i + e];
                                        y.x = fmaf(__uint_as_float(r[4 * e]) * lift, x, y.x);
                                        y.y = fmaf(__uint_as_float(r[4 * e + 1]) * lift, x, y.y);
                                        y.z = fmaf(__uint_as_float(r[4 * e + 2]) * lift, x, y.z);
                                        y.w = fmaf(__uint_as_float(r[4 * e + 3]) * lift, x, y.w);
                                    }
                                }
                            }
                            set_read(set);
#pragma unroll
                            for (int i = 0; i < 4 * PARTS; ++i) {
                                float* x = &acc[i / 4][i % 4 * 4];
                                x[0] = sums[i].x, x[1] = sums[i].y, x[2] = sums[i].z, x[3] = sums[i].w;
                            }
                        } else {
#pragma unroll
                            for (int kl = 0; kl < NB; ++kl)
                                if (kl < nkb) {
                                    const float mine = ld_shared(row_scale + kl * kLanes * 4u);
                                    const float x0 = mine * ld_shared(col_scale + kl * 16u), x1 = WHOLE ? x0 : mine * ld_shared(col_scale + kl * 16u + 4u);
#pragma unroll
                                    for (int i = 0; i < PARTS; i += 2) {
                                        const uint32_t at = taddr + static_cast<uint32_t>(kl * g.BN + 16 * i);
                                        uint32_t r[32];
                                        if (i + 1 < PARTS) {
                                            tmem_ld32_sync(at, r);
                                        } else {
                                            uint32_t h[16];
                                            tmem_ld16_sync(at, h);
#pragma unroll
                                            for (int e = 0; e < 16; ++e) r[e] = h[e];
                                        }
                                        if (i + 2 >= PARTS && (NB == 1 || kl + 1 == nkb)) set_read(set);
#pragma unroll
                                        for (int h = 0; h < 2; ++h)
                                            if (i + h < PARTS) {
                                                const float x = WHOLE || i + h < turn ? x0 : x1;
#pragma unroll
                                                for (int e = 0; e < 16; ++e)
                                                    acc[i + h < PARTS ? i + h : 0][e] = fmaf(__uint_as_float(r[16 * h + e]), x, acc[i + h < PARTS ? i + h : 0][e]);
                                            }
                                    }
                                }
                        }
                    }
                    phases ^= 1u << set;
                    const int after = (set + Q::kStageSets) & (Q::kSets - 1);
                    if (second) next[1] = after;
                    else next[0] = after;
                }
            };
            for (int s = 0; s < sets; s += kPageSets) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                // The vote: this page has landed, and the one before it is read.  And its products of scales are normal, as those of
                // most pages are: the scales of rows are the quantiser's least (rows of zeros have it) or above, and those of
                // weights are not small.  (Or the other way round; or the least of both meet, whose product makes nothing, and
                // the others are not small: blocks of zeros among the weights.)
                const float* landed = s_page[buf];            // this thread's own copies
                auto ranges = [&](float skip, auto&& fits) {
                    ScaleRange ra{__float_as_uint(skip)}, rb = ra;
#pragma unroll
                    for (int i = 0; i < kPageBlocks / 2; ++i) ra.add(landed[i * kEpilogue + tid]);
                    if (tid < 4 * kPageBlocks) rb.add(landed[kPageBlocks * kLanes + tid]);
                    return fits(ra, rb);
                };
                bool plain = Q::all_say(ok && ranges(0.0f, [](auto& ra, auto& rb) { return ra.within(kLeastScale) && rb.within(kMuchLarger); }));
                if (!plain) {
                    const bool least = ok && ranges(0.0f, [](auto& ra, auto& rb) { return ra.within(kLeastScale) && rb.within(kLeastScale); });
                    plain = Q::all_say(least && ranges(kLeastScale, [](auto& ra, auto& rb) { return ra.within(kMuchLarger) && rb.within(kMuchLarger); })) ||
                            Q::all_say(least && ranges(0.0f, [](auto& ra, auto&) { return ra.within(kMuchLarger); }));
                    if (!plain && !(ok = Q::all_say(ok))) break;
                }
                const int page = s / kPageSets + 1;
                buf ^= 1;
                if (page < pages)
                    fetch(t, page, s_page[buf]);
                else if (t + n_units < g.tiles)
                    fetch(t + n_units, 0, s_page[buf]);
                if (plain) page_sets(std::false_type{}, s, min(s + kPageSets, sets));
                else page_sets(std::true_type{}, s, min(s + kPageSets, sets));
            }
            if (!ok || !reads) continue;      // to the vote, or to the end
            const int row = (t % g.m_tiles) * (kLanes * CG) + rank * kLanes + q * 32 + lane;
            if (g.f32)
                put_row<true, PARTS>(acc, row, n0 + cb, g.BN - cb, g);
            else
                put_row<false, PARTS>(acc, row, n0 + cb, g.BN - cb, g);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }

    tc_fence_before();
    if constexpr (CG == 2) {
        // neither CTA leaves while the other may still read its shared memory or signal its barriers
        cluster_sync();
        tc_fence_after();
        if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
    } else {
        __syncthreads();
        tc_fence_after();
        if (warp == 1) tmem_dealloc(tmem_base, 512);
    }
}

// ---------------------------------------------------------------- host side
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// e4m3 [rows, K] in boxes [ks][box_rows][128 bytes], 128-byte swizzle; zeros past the ends.  Where K is no
// multiple of 128 a box holds one k-block.
bool encode_e4m3(CUtensorMap* map, const void* base, int rows, int K, int box_rows, int ks) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool whole = K % kBK == 0;
    const cuuint64_t ld = static_cast<cuuint64_t>(K);
    const cuuint64_t dims[3] = {whole ? kBK : ld, static_cast<cuuint64_t>(rows), whole ? ld / kBK : 1};
    const cuuint64_t strides[2] = {ld, kBK};
    const cuuint32_t box[3] = {kBK, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(whole ? ks : 1)}, estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Once per device and kernel: its opt-in shared memory, the registers it starts with (those that the sums'
// warps take are the ones that the others give up), and how many units (CTAs, or pairs) run at once.
template <int CG, int PARTS, bool WHOLE, bool DEEP>
int setup_e4m3(int* out) {
    static std::mutex mu;
    static int units[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    if (dev < 0 || dev >= kMaxDevices) return BIV_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(mu);
    if (units[dev] == 0) {
        auto kern = gemm_e4m3_kernel<CG, PARTS, WHOLE, DEEP>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return cuda_status(e);
        cudaFuncAttributes attrs;
        e = cudaFuncGetAttributes(&attrs, kern);
        if (e != cudaSuccess) return cuda_status(e);
        if (attrs.numRegs != kRegsStart) return BIV_ERR_DEVICE;
        int n = num_sms();
        if (CG == 2) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(2 * num_sms()));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = static_cast<size_t>(kMaxSmem);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) return cuda_status(e);
            if (n <= 0) return BIV_ERR_DEVICE;
        }
        units[dev] = n;
    }
    *out = units[dev];
    return BIV_OK;
}

template <int CG, int PARTS, bool WHOLE = false, bool DEEP = false>
int launch_e4m3(const void* A, const void* B, Gemm8Args g, cudaStream_t s) {
    int units = 0;
    const int st = setup_e4m3<CG, PARTS, WHOLE, DEEP>(&units);
    if (st != BIV_OK) return st;
    using Q = Form<PARTS, DEEP>;
    g.xr = CG == 2 ? kLanes : std::min(kLanes, (g.M + 7) / 8 * 8);
    g.yr = g.BN / CG;
    g.idesc = idesc_e4m3_f32(CG * kLanes, g.BN);
    const int per_kb = (g.xr + g.yr) * kBK, slack = g.xr < kLanes ? kSlack : 0;
    g.boxes = g.K % kBK == 0 ? 1 : Q::kStage;
    g.stages = std::min(kMaxStages, (kRing - slack) / (Q::kStage * per_kb) / (kIssuers / Q::kStageSets) * (kIssuers / Q::kStageSets));      // two at least
    g.m_tiles = static_cast<int>(ceil_div(g.M, CG * kLanes));
    const long long tiles = ceil_div(g.N, g.BN) * g.m_tiles;
    if (tiles > 0x3fffffffLL) return BIV_ERR_SHAPE;
    g.tiles = static_cast<int>(tiles);
    CUtensorMap ta, tb;
    if (!encode_e4m3(&ta, A, g.M, g.K, g.xr, Q::kStage) || !encode_e4m3(&tb, B, g.N, g.K, g.yr, Q::kStage)) {
        set_cuda_error(cudaErrorInvalidValue);
        return BIV_ERR_CUDA;
    }
    const size_t smem = 1024 + static_cast<size_t>(g.stages) * Q::kStage * per_kb + slack + kBarBytes + 2 * kPageFloats * 4;
    const unsigned grid = static_cast<unsigned>(std::min(g.tiles, units));
    if (CG == 2) return launch_cluster_pdl(gemm_e4m3_kernel<CG, PARTS, WHOLE, DEEP>, dim3(2 * grid), dim3(kThreads), smem, s, 2, ta, tb, g);
    return launch_pdl(gemm_e4m3_kernel<CG, PARTS, WHOLE, DEEP>, dim3(grid), dim3(kThreads), smem, s, ta, tb, g);
}

// The kernel for a tile width.
int launch_single(const void* A, const void* B, const Gemm8Args& g, cudaStream_t s) {
    if (g.BN <= 32) return launch_e4m3<1, 1>(A, B, g, s);
    if (g.BN <= 64) return launch_e4m3<1, 2>(A, B, g, s);
    // four sets of one k-block hide an accumulator's way to the sums and back better, two of two cost fewer steps on it:
    // 14336 x 4096 (two of two in brackets) 8 rows 15.5 us (14.6), 80: 15.3 (15.3), 96: 15.4 (15.5), 128: 15.6 (17.4);
    // 256 x 8192 x 4096 15.8 (17.9); 16384 x 14336 8 rows 43.9 (43.3), 80: 44.9 (44.5), 128: 46.2 (56.2), but also 96:
    // 45.2 (55.5), and 80 x 19200 x 4096 17.0 (19.3): between 65 and 96 rows it goes by N as well
    if (g.BN <= 128) return g.M <= 96 ? launch_e4m3<1, 4>(A, B, g, s) : launch_e4m3<1, 4, false, true>(A, B, g, s);
    if (g.BN <= 192) return launch_e4m3<1, 6>(A, B, g, s);
    return g.BN == 256 ? launch_e4m3<1, 8, true>(A, B, g, s) : launch_e4m3<1, 8>(A, B, g, s);
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" int biv_gemm_e4m3(const void* A, const float* a_scales, const void* B, const float* b_scales, const void* bias,
                             const void* residual, void* C, int out_dtype, int act, int M, int N, int K, biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (M < 0 || N <= 0 || K <= 0 || N % 8 != 0 || K % 16 != 0) return BIV_ERR_SHAPE;
    // rows, columns and terms are rounded up to whole tiles and stages in 32 bits
    constexpr int kMost = 0x7fffffff - 255;
    if (M > kMost || N > kMost || K > kMost) return BIV_ERR_SHAPE;
    if ((out_dtype != BIV_BF16 && out_dtype != BIV_F32) || act < BIV_ACT_NONE || act > BIV_ACT_SILU) return BIV_ERR_VALUE;
    if (M == 0) return BIV_OK;
    if (!A || !a_scales || !B || !b_scales || !C) return BIV_ERR_NULL;
    for (const void* p : {A, static_cast<const void*>(a_scales), B, static_cast<const void*>(b_scales), static_cast<const void*>(C), bias, residual})
        if (!aligned16(p)) return BIV_ERR_ALIGN;
    // an fp32 C over a bf16 residual would overwrite rows that are still to be read
    if (C == A || C == B || C == bias || C == a_scales || C == b_scales || (C == residual && out_dtype == BIV_F32)) return BIV_ERR_VALUE;
    Gemm8Args g = {};
    g.sa = a_scales;
    g.sb = b_scales;
    g.C = C;
    g.ba.bias = static_cast<const __nv_bfloat16*>(bias);
    g.ba.residual = static_cast<const __nv_bfloat16*>(residual);
    g.ba.act = act;
    g.M = M;
    g.N = N;
    g.K = K;
    g.KB = static_cast<int>(ceil_div(K, kBK));
    g.f32 = out_dtype == BIV_F32;
    g.wide = reinterpret_cast<uintptr_t>(C) % 32 == 0 && (g.f32 || N % 16 == 0);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sms = num_sms();
    const long long m_tiles = ceil_div(M, kLanes);
    const long long bn = std::max<long long>(16, ceil_div(ceil_div(N, sms), 16) * 16);
    if (m_tiles == 1 && bn <= 256) {
        g.BN = static_cast<int>(bn);
        return launch_single(A, B, g, s);
    }
    // several waves, or several row tiles: the width that fills whole waves, rather a wide one.  (64, 128, 160, 192, 256)
    // columns, us, and which is taken: 320 x 14336 x 4096 44.7, 40.6, 36.4, 38.5, 44.9 (160); 256 x 8192 x 4096 20.2, 15.7,
    // 19.8, 21.1, 23.3 (128); 160 x 4096 x 4096 11.5, 14.9, 19.3, 20.4, 22.6 (64); 513 x 14336 x 4096 69.2, 53.4, 52.7, 55.3,
    // 44.8 (256); 128 x 128256 x 4096 128, 100, 113, 104, 105 (256)
    double least = 1e30;
    for (int w : {64, 128, 160, 192, 256}) {
        const double cost = static_cast<double>(ceil_div(m_tiles * ceil_div(N, w), sms)) * (w + 96);
        if (cost <= least) {
            least = cost;
            g.BN = w;
        }
    }
    // Pairs take B out of L2 once for 256 rows, where that pads M no further: 1023 x 14336 x 4096 59.8 us (single CTAs:
    // 67.0), 1024 x 4096 x 14336 63.0 (71.5); but 320 x 128256 x 4096, with 512 rows for 384: 294 (237), and 513 x 14336 x
    // 4096 56.8 (44.8).
    return g.BN == 256 && m_tiles % 2 == 0 ? launch_e4m3<2, 8, true>(A, B, g, s) : launch_single(A, B, g, s);
}
