// No-split-K GEMM of e4m3 operands with a scale for every 128 terms, on the
// 5th-generation tensor cores (tcgen05 + TMEM), fed by TMA:
//   C[m][n] = act(sum_b sa[b][m] sb[n / 128][b] sum_{k in block b} A[m][k] B[n][k] + bias[n]) + residual[m][n]
//
// The tensor core sums one k-block of 128 terms (four MMAs of K = 32) into an
// accumulator in TMEM that starts at zero; the epilogue warps read it, multiply it by the
// two scales and add it to fp32 sums in their registers, block by block in increasing k.
// That order, and a row's bits, do not depend on M, on the tile or on which operand lies
// along the accumulator's lanes.  So the work of the CUDA cores goes with the tensor
// core's: 256 x 256 a pair and k-block are 128 fused multiply-adds a thread.
//
// Kernel layout (320 threads, one CTA per SM, persistent over tiles), as in biv_gemm.cu:
//   warp 0      TMA producer: boxes of KS k-blocks, 128-byte swizzle
//   warp 1      TMEM allocator + MMA issuer
//   warps 2..9  sums and stores, two warps per TMEM lane quarter (half of the columns each)
// TMEM holds two sets of 256 columns, each of `nb` k-blocks' accumulators (nb BN <= 256):
// while the epilogue reads one, the other is filled.
//
// Two forms:
//   rows    (M <= 128, and N small enough for one wave) one CTA per tile: the rows of A along
//           the lanes, BN columns of C: the weights stream once, as many CTAs as SMs.
//   columns a pair of CTAs per tile (cta_group::2): 256 rows of the WEIGHTS along the lanes
//           (one scale for a CTA and k-block), BN rows of A as the tile's columns: M is cut into
//           multiples of 32 instead of 128 (320 rows are two tiles of 160, not 512), and a
//           warp's lanes are consecutive n of one row of C, so that it stores whole lines.
#include <algorithm>

#include "biv_act.cuh"

namespace biv {
namespace {

BIV_DEFINE_ERR_WORD(g_gemm8_err)

constexpr int kLanes = 128;                   // rows of an accumulator in one CTA
constexpr int kBK = 128;                      // a k-block: 128 e4m3, one swizzle row and one scale
constexpr int kSetCols = 256;
constexpr int kMaxStages = 16;
constexpr int kEpilogue = 256;                // epilogue threads
constexpr int kRowSets = 4;                   // k-blocks of a set, at most, in the rows form
constexpr int kBarBytes = 512;
constexpr int kScaleFloats = kRowSets * kLanes + kRowSets * 4;        // of a set: see Scales
constexpr int kRing = 227 * 1024 - 1024 - kBarBytes - 2 * kScaleFloats * 4 - 1024;
constexpr int kSlack = kLanes * kBK;          // an MMA may read 128 rows past the last stage
constexpr int kParts = 8;                     // 16 columns each: a thread's half of 256

struct Gemm8Args {
    int M, N, K, KB;                          // k-blocks
    int BN, KS, stages, nb;
    int xr, yr;                               // rows of a CTA's boxes: along the lanes, along the columns
    int y_tiles, work;
    int three_d;                              // K % 128 == 0: a box may hold several k-blocks
    uint32_t idesc;
    const float* sa;                          // [KB][M]
    const float* sb;                          // [ceil(N / 128)][KB]
};

// A barrier of the epilogue threads and a vote: true if every one says so.
BIV_DEV bool set_all(bool ok) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(ok ? 1u : 0u)
                 : "memory");
    return r != 0;
}

template <bool COLS, bool F32>
__global__ void __launch_bounds__(64 + kEpilogue, 1)
gemm_e4m3_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY, void* __restrict__ C,
                 const Gemm8Args g, const BiasActArgs ba) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int CG = COLS ? 2 : 1;
    const int X_BYTES = g.KS * g.xr * kBK, STAGE = X_BYTES + g.KS * g.yr * kBK, S = g.stages;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * STAGE + (g.xr < kLanes ? kSlack : 0));
    uint64_t* empty = full + kMaxStages;
    uint64_t* tfull = empty + kMaxStages;     // [2]
    uint64_t* tempty = tfull + 2;             // [2]
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float(*s_scale)[kScaleFloats] = reinterpret_cast<float(*)[kScaleFloats]>(reinterpret_cast<uint8_t*>(full) + kBarBytes);   // [2]

    const int rank = COLS ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / CG, n_units = static_cast<int>(gridDim.x) / CG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_stages = (g.KB + g.KS - 1) / g.KS;                   // of a tile
    // epilogue warps with rows to read: all, or those of the quarters that M reaches
    const int readers = COLS ? 16 : 2 * min(4, (g.M + 31) / 32);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], readers);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmY);
    }
    if (warp == 1) {
        if constexpr (COLS) {
            tmem_alloc_pair(tmem_slot, 2 * kSetCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, 2 * kSetCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if constexpr (COLS)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const uint64_t pol_w = !COLS || g.y_tiles == 1 ? policy_evict_first() : policy_evict_normal();   // weights: read once
    const uint64_t pol_a = policy_evict_last();                                                      // activations: by every CTA
    const uint32_t tx = static_cast<uint32_t>(STAGE);
    // the X or Y box of a stage of tile t
    auto load = [&](const CUtensorMap* map, uint8_t* dst, int stage, int row, int sb, uint64_t pol) {
        const int c0 = g.three_d ? 0 : sb * kBK, c2 = g.three_d ? sb * g.KS : 0;
        if constexpr (COLS)
            tma_load_3d_pair(dst, map, mapa_shared(&full[stage], 0), c0, row, c2, pol);
        else
            tma_load_3d(dst, map, &full[stage], c0, row, c2, pol);
    };
    auto load_x = [&](int t, int sb, int stage) {
        load(&tmX, smem + stage * STAGE, stage, (t / g.y_tiles) * (kLanes * CG) + rank * kLanes, sb, COLS ? pol_w : pol_a);
    };
    auto load_y = [&](int t, int sb, int stage) {
        load(&tmY, smem + stage * STAGE + X_BYTES, stage, (t % g.y_tiles) * g.BN + rank * g.yr, sb, COLS ? pol_a : pol_w);
    };
    auto expect = [&](int stage) {            // a pair's copies all complete on the even CTA's barrier
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * tx);
    };
    // The weights are no output of the previous kernel: the first stages' are asked for before waiting for it.
    int early = 0;
    if (warp == 0 && lane == 0 && unit < g.work) {
        early = min(S, n_stages);
        for (int sb = 0; sb < early; ++sb) {
            expect(sb);
            if constexpr (COLS)
                load_x(unit, sb, sb);
            else
                load_y(unit, sb, sb);
        }
    }
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int t = unit; t < g.work && ok; t += n_units)
                for (int sb = 0; sb < n_stages; ++sb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_gemm8_err, true, COLS)) {
                        ok = false;
                        break;
                    }
                    const bool asked = t == unit && sb < early;
                    if (!asked) expect(stage);
                    if (!(COLS && asked)) load_x(t, sb, stage);
                    if (!(!COLS && asked)) load_y(t, sb, stage);
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
        }
    } else if (warp == 1) {
        // --------------------------------------------------- MMA issuer
        if (rank == 0) {
            int stage = 0, set = 0;
            uint32_t phase = 0, set_phase = 0;
            bool ok = true, any = false;
            auto commit_set = [&]() {
                if constexpr (COLS) {
                    umma_commit_pair_elect(mapa_shared(&tfull[set], 0));
                    umma_commit_pair_elect(mapa_shared(&tfull[set], 1));
                } else {
                    umma_commit_elect(&tfull[set]);
                }
                set ^= 1;
                if (set == 0) set_phase ^= 1u;
            };
            for (int t = unit; t < g.work && ok; t += n_units) {
                int in_set = 0;                                      // k-blocks of the present set
                for (int sb = 0; sb < n_stages && ok; ++sb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, &g_gemm8_err, true, COLS));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t x_addr = smem_u32(smem + stage * STAGE), y_addr = x_addr + static_cast<uint32_t>(X_BYTES);
                    const int nkb = min(g.KS, g.KB - sb * g.KS);
                    for (int j = 0; j < nkb; ++j) {
                        if (in_set == 0) {
                            ok = __all_sync(0xffffffffu, mbar_wait(&tempty[set], set_phase ^ 1u, abort_flag, &g_gemm8_err, true, COLS));
                            if (!ok) break;
                            tc_fence_after();
                        }
                        const uint32_t d = tmem_base + static_cast<uint32_t>(set * kSetCols + in_set * g.BN);
                        const uint64_t x = sw128_kmajor_desc(x_addr + static_cast<uint32_t>(j * g.xr * kBK));
                        const uint64_t y = sw128_kmajor_desc(y_addr + static_cast<uint32_t>(j * g.yr * kBK));
#pragma unroll
                        for (int k = 0; k < kBK / 32; ++k) {
                            // +32 bytes along K inside the swizzle row = +2 in 16-byte units
                            if constexpr (COLS)
                                umma_f8_pair_elect(d, x + 2u * k, y + 2u * k, g.idesc, k > 0 ? 1u : 0u);
                            else
                                umma_f8_elect(d, x + 2u * k, y + 2u * k, g.idesc, k > 0 ? 1u : 0u);
                        }
                        any = true;
                        if (++in_set == g.nb || sb * g.KS + j + 1 == g.KB) {
                            commit_set();
                            in_set = 0;
                        }
                    }
                    if (!ok) break;
                    if constexpr (COLS) {
                        umma_commit_pair_elect(mapa_shared(&empty[stage], 0));
                        umma_commit_pair_elect(mapa_shared(&empty[stage], 1));
                    } else {
                        umma_commit_elect(&empty[stage]);
                    }
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && any) {
                // all MMAs issued so far have finished
                if constexpr (COLS)
                    umma_commit_pair_elect(mapa_shared(drain, 0));
                else
                    umma_commit_elect(drain);
                if (lane == 0) mbar_wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------- sums and stores
        const int q = warp & 3, half = (warp - 2) >> 2, tid = static_cast<int>(threadIdx.x) - 64;
        const int hc = (g.BN / 2 + 15) / 16 * 16;
        const int cb = half ? hc : 0, ce = half ? g.BN : hc;           // this warp's columns of the tile
        const bool reads = COLS || q * 32 < g.M;
        const int parts = reads ? (ce - cb + 15) / 16 : 0;
        const int sets = (g.KB + g.nb - 1) / g.nb;
        // Scales of set s of tile t, one to three numbers a thread.  Columns form: [k-block][column]
        // sa times the CTA's sb.  Rows form: [k-block][row] sa, then [k-block][4] sb of the tile's 128-column blocks.
        float pre[3];
        auto fetch = [&](int t, int s) {
            pre[0] = pre[1] = pre[2] = 0.0f;
            if constexpr (COLS) {
                const int kb = s * g.nb + tid / g.BN, col = tid % g.BN;
                const int m = (t % g.y_tiles) * g.BN + col, n0 = (t / g.y_tiles) * (2 * kLanes) + rank * kLanes;
                if (tid / g.BN < g.nb && kb < g.KB && m < g.M && n0 < g.N)
                    pre[0] = g.sa[static_cast<long long>(kb) * g.M + m] * __ldg(g.sb + static_cast<long long>(n0 / 128) * g.KB + kb);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int kl = (tid + i * kEpilogue) / kLanes, row = tid % kLanes, kb = s * g.nb + kl;
                    if (kl < g.nb && kb < g.KB && row < g.M) pre[i] = g.sa[static_cast<long long>(kb) * g.M + row];
                }
                const int kl = tid / 4, kb = s * g.nb + kl, nblk = t * g.BN / 128 + tid % 4;
                if (kl < g.nb && kb < g.KB && nblk < (g.N + 127) / 128) pre[2] = __ldg(g.sb + static_cast<long long>(nblk) * g.KB + kb);
            }
        };
        auto put = [&](float* dst) {
            if constexpr (COLS) {
                dst[tid] = pre[0];
            } else {
                dst[tid] = pre[0];
                dst[tid + kEpilogue] = pre[1];
                if (tid < 4 * kRowSets) dst[kRowSets * kLanes + tid] = pre[2];
            }
        };
        int set = 0;
        uint32_t set_phase = 0;
        bool ok = true;                       // a wait ran out: the warps leave together, at the next vote
        if (unit < g.work) fetch(unit, 0);
        for (int t = unit; t < g.work; t += n_units) {
            const int col0 = (t % g.y_tiles) * g.BN;
            float acc[kParts][16];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
            for (int s = 0; s < sets; ++s) {
                float* scale = s_scale[set];
                put(scale);
                if (!(ok = set_all(ok))) break;
                if (s + 1 < sets)
                    fetch(t, s + 1);
                else if (t + n_units < g.work)
                    fetch(t + n_units, 0);
                if (reads) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&tfull[set], set_phase, abort_flag, &g_gemm8_err, false, COLS));
                    tc_fence_after();
                    const int nkb = ok ? min(g.nb, g.KB - s * g.nb) : 0;
                    for (int kl = 0; kl < nkb; ++kl) {
                        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(set * kSetCols + kl * g.BN + cb);
                        const float row_scale = COLS ? 0.0f : scale[kl * kLanes + q * 32 + lane];
#pragma unroll
                        for (int i = 0; i < kParts; ++i)
                            if (i < parts) {
                                uint32_t r[16];
                                tmem_ld16_sync(taddr + static_cast<uint32_t>(16 * i), r);
                                if constexpr (COLS) {
                                    const float4* sc = reinterpret_cast<const float4*>(scale + kl * g.BN + cb + 16 * i);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float4 x = sc[e];
                                        acc[i][4 * e] = fmaf(__uint_as_float(r[4 * e]), x.x, acc[i][4 * e]);
                                        acc[i][4 * e + 1] = fmaf(__uint_as_float(r[4 * e + 1]), x.y, acc[i][4 * e + 1]);
                                        acc[i][4 * e + 2] = fmaf(__uint_as_float(r[4 * e + 2]), x.z, acc[i][4 * e + 2]);
                                        acc[i][4 * e + 3] = fmaf(__uint_as_float(r[4 * e + 3]), x.w, acc[i][4 * e + 3]);
                                    }
                                } else {
                                    const float x = row_scale * scale[kRowSets * kLanes + kl * 4 + (col0 + cb + 16 * i) / 128 - col0 / 128];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) acc[i][e] = fmaf(__uint_as_float(r[e]), x, acc[i][e]);
                                }
                            }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (COLS)
                            mbar_arrive_cluster(mapa_shared(&tempty[set], 0));
                        else
                            mbar_arrive(&tempty[set]);
                    }
                }
                set ^= 1;
                if (set == 0) set_phase ^= 1u;
            }
            if (!ok) continue;                // to the vote, or to the end
            if constexpr (COLS) {
                // lane: n; columns: rows m of C
                const int n = (t / g.y_tiles) * (2 * kLanes) + rank * kLanes + q * 32 + lane;
                const float bias = ba.bias && n < g.N ? __bfloat162float(ba.bias[n]) : 0.0f;
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    if (i < parts) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const int m = col0 + cb + 16 * i + e;
                            float v0 = acc[i][e] + bias, v1 = acc[i][e + 1] + bias;
                            if (ba.act != BIV_ACT_NONE) {
                                v0 = activate(v0, ba.act);
                                v1 = activate(v1, ba.act);
                            }
                            if constexpr (F32) {
                                if (n < g.N) {
                                    const long long at = static_cast<long long>(m) * g.N + n;
                                    if (m < g.M) static_cast<float*>(C)[at] = v0 + (ba.residual ? __bfloat162float(ba.residual[at]) : 0.0f);
                                    if (m + 1 < g.M)
                                        static_cast<float*>(C)[at + g.N] = v1 + (ba.residual ? __bfloat162float(ba.residual[at + g.N]) : 0.0f);
                                }
                            } else {
                                // even lanes store n, n + 1 of row m, odd lanes n - 1, n of row m + 1
                                const bool odd = lane & 1;
                                const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
                                float lo = odd ? other : v0, hi = odd ? v1 : other;
                                const int row = m + (odd ? 1 : 0), n2 = n & ~1;
                                if (row < g.M && n2 < g.N) {
                                    uint32_t* at = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(C) + static_cast<long long>(row) * g.N + n2);
                                    if (ba.residual) {
                                        const uint32_t x = *reinterpret_cast<const volatile uint32_t*>(ba.residual + static_cast<long long>(row) * g.N + n2);
                                        lo += bf16lo(x);
                                        hi += bf16hi(x);
                                    }
                                    *at = pack_bf16x2(lo, hi);
                                }
                            }
                        }
                    }
            } else {
                const int row = q * 32 + lane;
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    if (i < parts) {
                        const BiasActRow operands(row < g.M, row, col0 + cb + 16 * i, g.N, ba);
                        operands.template store<F32>([&](int e) { return acc[i][e]; }, C, ba);
                    }
            }
        }
    }

    tc_fence_before();
    if constexpr (COLS) {
        // neither CTA leaves while the other may still read its shared memory or signal its barriers
        cluster_sync();
        tc_fence_after();
        if (warp == 1) tmem_dealloc_pair(tmem_base, 2 * kSetCols);
    } else {
        __syncthreads();
        tc_fence_after();
        if (warp == 1) tmem_dealloc(tmem_base, 2 * kSetCols);
    }
}

// ---------------------------------------------------------------- host side
// e4m3 [rows, K] in boxes [KS][box_rows][128 bytes], 128-byte swizzle; zeros past the ends.
bool encode_e4m3(CUtensorMap* map, const void* base, int rows, int K, int box_rows, int ks, bool three_d) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t ld = static_cast<cuuint64_t>(K);
    const cuuint64_t dims[3] = {three_d ? kBK : ld, static_cast<cuuint64_t>(rows), three_d ? ld / kBK : 1};
    const cuuint64_t strides[2] = {ld, kBK};
    const cuuint32_t box[3] = {kBK, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(ks)}, estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// The kernel's opt-in shared memory and how many of its CTAs (pairs) run at once.
template <bool COLS, bool F32>
int setup_e4m3(int dev, int* units) {
    static std::mutex mu;
    static int known[kMaxDevices] = {};
    if (dev < 0 || dev >= kMaxDevices) return BIV_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        auto kern = gemm_e4m3_kernel<COLS, F32>;
        const int smem = 227 * 1024 - 1024;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_status(e);
        int n = num_sms();
        if (COLS) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(2 * num_sms()));
            cfg.blockDim = dim3(64 + kEpilogue);
            cfg.dynamicSmemBytes = static_cast<size_t>(smem);
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
        known[dev] = n;
    }
    *units = known[dev];
    return BIV_OK;
}

template <bool COLS, bool F32>
int launch_e4m3(const void* A, const void* B, void* C, Gemm8Args g, const BiasActArgs& ba, cudaStream_t s) {
    int dev = 0, units = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    const int st = setup_e4m3<COLS, F32>(dev, &units);
    if (st != BIV_OK) return st;
    g.xr = COLS ? kLanes : std::min(kLanes, (g.M + 7) / 8 * 8);
    g.yr = COLS ? g.BN / 2 : g.BN;
    g.nb = std::min(kRowSets, kSetCols / g.BN);
    g.three_d = g.K % kBK == 0 ? 1 : 0;
    g.idesc = idesc_e4m3_f32(COLS ? 2 * kLanes : kLanes, g.BN);
    const int per_kb = (g.xr + g.yr) * kBK, ring = kRing - (g.xr < kLanes ? kSlack : 0);
    // A box costs the TMA unit a fixed time: several k-blocks each, as long as four stages fit.
    g.KS = g.three_d ? std::min(g.KB, std::max(1, ring / (COLS ? 3 : 4) / per_kb)) : 1;
    if (COLS) g.KS = std::min(g.KS, 2);
    g.stages = std::min(kMaxStages, ring / (g.KS * per_kb));
    const long long x_tiles = COLS ? ceil_div(g.N, 2 * kLanes) : 1;
    g.y_tiles = static_cast<int>(ceil_div(COLS ? g.M : g.N, g.BN));
    if (x_tiles * g.y_tiles > 0x3fffffffLL) return BIV_ERR_SHAPE;
    g.work = static_cast<int>(x_tiles * g.y_tiles);
    CUtensorMap tx, ty;
    if (!encode_e4m3(&tx, COLS ? B : A, COLS ? g.N : g.M, g.K, g.xr, g.KS, g.three_d) ||
        !encode_e4m3(&ty, COLS ? A : B, COLS ? g.M : g.N, g.K, g.yr, g.KS, g.three_d)) {
        set_cuda_error(cudaErrorInvalidValue);
        return BIV_ERR_CUDA;
    }
    const size_t smem = 1024 + static_cast<size_t>(g.stages) * g.KS * per_kb + (g.xr < kLanes ? kSlack : 0) + kBarBytes + 2 * kScaleFloats * 4;
    const unsigned grid = static_cast<unsigned>(std::min(g.work, units));
    if (COLS) return launch_cluster_pdl(gemm_e4m3_kernel<COLS, F32>, dim3(2 * grid), dim3(64 + kEpilogue), smem, s, 2, tx, ty, C, g, ba);
    return launch_pdl(gemm_e4m3_kernel<COLS, F32>, dim3(grid), dim3(64 + kEpilogue), smem, s, tx, ty, C, g, ba);
}

// Columns form: M in tiles of equal width, a multiple of 32 up to 256, so that the waves of
// pairs are full and the tiles wide.
int columns_tile(int M, int N, int pairs) {
    int best = 256;
    double least = 1e30;
    for (int bn = 32; bn <= 256; bn += 32) {
        const double cost = static_cast<double>(ceil_div(ceil_div(N, 2 * kLanes) * ceil_div(M, bn), pairs)) * (bn + 32);
        if (cost <= least) {
            least = cost;
            best = bn;
        }
    }
    return best;
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" int biv_gemm_e4m3(const void* A, const float* a_scales, const void* B, const float* b_scales, const void* bias,
                             const void* residual, void* C, int out_dtype, int act, int M, int N, int K, biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (M < 0 || N <= 0 || K <= 0 || N % 8 != 0 || K % 16 != 0) return BIV_ERR_SHAPE;
    if ((out_dtype != BIV_BF16 && out_dtype != BIV_F32) || act < BIV_ACT_NONE || act > BIV_ACT_SILU) return BIV_ERR_VALUE;
    if (M == 0) return BIV_OK;
    if (!A || !a_scales || !B || !b_scales || !C) return BIV_ERR_NULL;
    for (const void* p : {A, static_cast<const void*>(a_scales), B, static_cast<const void*>(b_scales), static_cast<const void*>(C), bias, residual})
        if (!aligned16(p)) return BIV_ERR_ALIGN;
    // an fp32 C over a bf16 residual would overwrite rows that are still to be read
    if (C == A || C == B || C == bias || C == a_scales || C == b_scales || (C == residual && out_dtype == BIV_F32)) return BIV_ERR_VALUE;
    Gemm8Args g = {};
    g.M = M;
    g.N = N;
    g.K = K;
    g.KB = static_cast<int>(ceil_div(K, kBK));
    g.sa = a_scales;
    g.sb = b_scales;
    BiasActArgs ba;
    ba.bias = static_cast<const __nv_bfloat16*>(bias);
    ba.residual = static_cast<const __nv_bfloat16*>(residual);
    ba.act = act;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sms = num_sms();
    const long long bn = std::max<long long>(16, ceil_div(ceil_div(N, sms), 16) * 16);
    if (M <= kLanes && bn <= kSetCols) {
        g.BN = static_cast<int>(bn);
        return out_dtype == BIV_F32 ? launch_e4m3<false, true>(A, B, C, g, ba, s) : launch_e4m3<false, false>(A, B, C, g, ba, s);
    }
    g.BN = columns_tile(M, N, sms / 2);
    return out_dtype == BIV_F32 ? launch_e4m3<true, true>(A, B, C, g, ba, s) : launch_e4m3<true, false>(A, B, C, g, ba, s);
}
