// The paged key-value cache: rotation and write of new rows into pages, and
// fixed-split decode attention over them.
#include <algorithm>
#include <cmath>

#include "biv_common.cuh"

namespace biv {
namespace {

BIV_DEFINE_ERR_WORD(g_paged_err)

constexpr int kSplit = BIV_KV_SPLIT;

// Where a pool's rows lie: page p, KV head h, offset t is row (p * Hkv + h) *
// page_size + t of hd elements.
struct PageTable {
    const int32_t* table;      // [n_slots, max_pages]
    int n_slots, max_pages, n_pages, page_size, page_shift;
};

// --------------------------------------------------- RoPE + paged write
// Turns per position of each rotation pair, theta^(-2i/hd) / 2 pi, as 64-bit
// fractions of a turn: position times this, modulo 2^64, is the angle modulo a
// full turn with an error of pos * 2^-65 turns.
struct RopeTurns {
    uint64_t per_pos[128];     // hd / 2 <= 128
};

constexpr int kRopeThreads = 256;

// One CTA per `rows` consecutive rows.  Its threads first take the sines and
// cosines of the rows' angles (one each, in shared memory), then rotate: an
// item is eight pairs of one head, two 16-byte loads and two 16-byte stores, so
// every sector that is touched is used whole.  Bound by memory: 2 x (Hq + 2 Hkv)
// hd x 2 bytes per row.
__global__ void __launch_bounds__(kRopeThreads)
rope_kv_write_paged_kernel(const __nv_bfloat16* __restrict__ qkv, __nv_bfloat16* __restrict__ q_out,
                           __nv_bfloat16* __restrict__ kp, __nv_bfloat16* __restrict__ vp, const PageTable pt,
                           const int32_t* __restrict__ row_slot, const int32_t* __restrict__ row_pos,
                           const int32_t* __restrict__ rows_keep, int W, int K, int Hq, int Hkv, int hd, int rows,
                           const __grid_constant__ RopeTurns turns) {
    extern __shared__ float s_cs[];                     // [rows][2][hd / 2]: cosines, then sines
    __shared__ long long s_dst[8];                      // first element of the row's place for KV head 0, or -1
    const int half = hd / 2;
    const int w0 = blockIdx.x * rows;
    const int nr = min(rows, W - w0);
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(threadIdx.x) < nr) {
        const int w = w0 + threadIdx.x;
        const int pos = row_pos[w];
        const bool keep = !rows_keep || (w % K) < rows_keep[w / K];
        long long dst = -1;
        if (keep && pos != -1) {
            const int slot = row_slot[w];
            int page = -1;
            if (slot >= 0 && slot < pt.n_slots && pos >= 0 && (pos >> pt.page_shift) < pt.max_pages)
                page = pt.table[static_cast<long long>(slot) * pt.max_pages + (pos >> pt.page_shift)];
            if (page >= 0 && page < pt.n_pages)
                dst = (static_cast<long long>(page) * Hkv * pt.page_size + (pos & (pt.page_size - 1))) * hd;
            else
                atomicOr(&g_paged_err, BIV_DEVERR_INDEX);
        }
        s_dst[threadIdx.x] = dst;
    }
    for (int e = threadIdx.x; e < nr * half; e += kRopeThreads) {
        const int r = e / half, i = e - r * half;
        const uint64_t phase = static_cast<uint64_t>(static_cast<long long>(row_pos[w0 + r])) * turns.per_pos[i];
        // the top 32 bits as a signed fraction of half a turn
        const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;
        float sn, cs;
        sincospif(x, &sn, &cs);
        s_cs[r * hd + i] = cs;
        s_cs[r * hd + half + i] = sn;
    }
    __syncthreads();
    const int per_head = half / 8;                      // rotation items of one head
    const int heads = Hq + 2 * Hkv;
    const int items = heads * per_head;
    for (int it = threadIdx.x; it < nr * items; it += kRopeThreads) {
        const int r = it / items, u = it - r * items;
        const int h = u / per_head, i = (u - h * per_head) * 8;
        const int w = w0 + r;
        __nv_bfloat16* dst;
        if (h < Hq) {
            dst = q_out + (static_cast<long long>(w) * Hq + h) * hd;
        } else {
            if (s_dst[r] < 0) continue;
            const int kh = h < Hq + Hkv ? h - Hq : h - Hq - Hkv;
            dst = (h < Hq + Hkv ? kp : vp) + s_dst[r] + static_cast<long long>(kh) * pt.page_size * hd;
        }
        const __nv_bfloat16* src = qkv + (static_cast<long long>(w) * heads + h) * hd;
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(src + i));
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(src + half + i));
        if (h >= Hq + Hkv) {
            *reinterpret_cast<uint4*>(dst + i) = a;
            *reinterpret_cast<uint4*>(dst + half + i) = b;
            continue;
        }
        const uint32_t a4[4] = {a.x, a.y, a.z, a.w}, b4[4] = {b.x, b.y, b.z, b.w};
        const float* cs = s_cs + r * hd + i;
        const float* sn = cs + half;
        uint32_t o1[4], o2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float al = bf16lo(a4[e]), ah = bf16hi(a4[e]), bl = bf16lo(b4[e]), bh = bf16hi(b4[e]);
            const float cl = cs[2 * e], ch = cs[2 * e + 1], sl = sn[2 * e], sh = sn[2 * e + 1];
            o1[e] = pack_bf16x2(al * cl - bl * sl, ah * ch - bh * sh);
            o2[e] = pack_bf16x2(bl * cl + al * sl, bh * ch + ah * sh);
        }
        *reinterpret_cast<uint4*>(dst + i) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
        *reinterpret_cast<uint4*>(dst + half + i) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
    }
}

// ------------------------------------------------------ paged attention
struct PagedAttnParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kp;
    const __nv_bfloat16* vp;
    const int32_t* row_slot;
    const int32_t* row_pos;
    __nv_bfloat16* o;
    float* ws_o;               // [W][Hq][s_max][hd] unnormalised outputs of a split
    float2* ws_ml;             // [W][Hq][s_max] (maximum in units of log 2, sum); sum -1: a page id out of range
    PageTable pt;
    int W, rpg, G, Hq, Hkv, s_max, cap;
    float scale_log2;          // log2(e) / sqrt(hd)
};

// Position of row w if the row is to be computed, else -1; the first row's slot
// decides the group's.  flag: raise the error bits (one thread of a grid).
BIV_DEV int usable_pos(const PagedAttnParams& P, int w, bool flag) {
    const int pos = P.row_pos[w];
    if (pos == -1) return -1;
    const int slot = P.row_slot[w], first = P.row_slot[w - w % P.rpg];
    unsigned int bits = 0;
    if (pos < 0 || pos >= P.cap || slot < 0 || slot >= P.pt.n_slots) bits = BIV_DEVERR_INDEX;
    else if (slot != first) bits = BIV_DEVERR_GROUP;
    if (bits && flag) atomicOr(&g_paged_err, bits);
    return bits ? -1 : pos;
}

// ---- the split kernel
// One item is (request, KV head, 256-key split, tile of 8 NT query rows), where
// the query rows are the request's window rows times the G heads of the KV
// head.  Keys go along the M side of the tensor core's tile and query rows along
// N (mma.m16n8k16): S^T = K Q^T and O^T = V^T P^T, so eight rows fill a tile and
// the four rows of a single token waste half of it instead of the 60 of 64 that
// a rows-by-keys tile would.  The permutation of the dims inside a product is
// free, and chosen so that every operand comes straight from global memory in
// 32-byte loads, a whole 128-byte line per four (K) or eight (V) lanes: no
// shared memory, no barrier and no address arithmetic between HBM and the
// tensor core.  Four warps take the 16-key steps of the split in turn, each with
// its own running maximum and sum, and meet once at the end.
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kStep = 16;
constexpr int kStepsPerWarp = kSplit / kStep / kAttnWarps;
constexpr int kMaxGroups = 1024;       // entries of the table of live splits; more groups share entries

// 32 bytes of a row of keys or values: read once, so not kept in L1.
BIV_DEV void ld_row32(const __nv_bfloat16* p, uint32_t (&r)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
BIV_DEV void ld_row16(const __nv_bfloat16* p, uint32_t (&r)[4]) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
}

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 with fp32 sums.
BIV_DEV void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 tile of bf16 held two to a lane.
BIV_DEV uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Largest usable position of group g, -1 if it has none.
BIV_DEV int group_pos(const PagedAttnParams& P, int g, bool flag) {
    int best = -1;
    const int w1 = min(P.W, (g + 1) * P.rpg);
    for (int w = g * P.rpg; w < w1; ++w) best = max(best, usable_pos(P, w, flag));
    return best;
}

template <int HD, int NT>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? 3 : 2)
paged_attn_kernel(const PagedAttnParams P) {
    constexpr int KS = HD / 16;            // k-steps of S^T; also the 16-dim tiles of O^T
    constexpr int KC = HD / 64;            // 64-dim chunks of a key: one 32-byte load per lane each
    constexpr int TR = 8 * NT;             // query rows of a tile
    constexpr int HDP = HD + 4;            // padded row of the warps' outputs
    __shared__ int s_pre[kMaxGroups + 1];  // live splits before each entry
    __shared__ int s_pos[kMaxGroups];      // largest usable position of each group (one group per entry)
    __shared__ int s_scan[kAttnWarps];
    __shared__ __align__(16) float s_o[kAttnWarps][TR][HDP];
    __shared__ float2 s_ml[kAttnWarps][TR];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;       // row of an 8-row fragment, column pair

    // Live splits of every group: computed by each CTA from the positions, which
    // are not an output of the previous kernel.
    const int n_groups = (P.W + P.rpg - 1) / P.rpg;
    const int chunk = (n_groups + kMaxGroups - 1) / kMaxGroups;
    const int entries = (n_groups + chunk - 1) / chunk;
    const bool flag = blockIdx.x == 0;
    if (chunk == 1) {
        for (int e = tid; e < entries; e += kAttnThreads) s_pos[e] = -1;
        __syncthreads();
        for (int w = tid; w < P.W; w += kAttnThreads) {
            const int pos = usable_pos(P, w, flag);
            if (pos >= 0) atomicMax(&s_pos[w / P.rpg], pos);
        }
        __syncthreads();
    }
    constexpr int EPT = kMaxGroups / kAttnThreads;         // entries of a thread
    int mine[EPT], sum = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int e = tid * EPT + i;
        int n = 0;
        if (e < entries) {
            if (chunk == 1) n = s_pos[e] / kSplit + (s_pos[e] >= 0);
            else
                for (int g = e * chunk; g < min(n_groups, (e + 1) * chunk); ++g) {
                    const int pos = group_pos(P, g, flag);
                    n += pos / kSplit + (pos >= 0);
                }
        }
        mine[i] = sum;
        sum += n;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int before = incl - sum, units = 0;
    for (int k = 0; k < kAttnWarps; ++k) {
        if (k < warp) before += s_scan[k];
        units += s_scan[k];
    }
#pragma unroll
    for (int i = 0; i < EPT; ++i)
        if (tid * EPT + i < entries) s_pre[tid * EPT + i] = before + mine[i];
    __syncthreads();

    pdl_wait();
    pdl_trigger();

    // rows that are not computed come back as zeros
    for (int w = blockIdx.x; w < P.W; w += gridDim.x) {
        const int pos = chunk == 1 && P.rpg == 1 ? s_pos[w] : usable_pos(P, w, false);
        if (pos < 0)
            for (int e = tid; e < P.Hq * HD / 8; e += kAttnThreads)
                reinterpret_cast<uint4*>(P.o + static_cast<long long>(w) * P.Hq * HD)[e] = make_uint4(0, 0, 0, 0);
    }

    const int tiles = (P.rpg * P.G + TR - 1) / TR;
    const int per_unit = P.Hkv * tiles;
    const long long items = static_cast<long long>(units) * per_unit;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int unit = static_cast<int>(item / per_unit), sub = static_cast<int>(item - static_cast<long long>(unit) * per_unit);
        const int kvh = sub / tiles, tile = sub - kvh * tiles;
        int lo = 0, hi = entries - 1;              // the last entry with s_pre <= unit
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_pre[mid] <= unit) lo = mid;
            else hi = mid - 1;
        }
        int grp = lo, split = unit - s_pre[lo];
        if (chunk > 1) {
            for (grp = lo * chunk;; ++grp) {
                const int pos = group_pos(P, grp, false);
                const int n = pos / kSplit + (pos >= 0);
                if (split < n) break;
                split -= n;
            }
        }
        const int w0 = grp * P.rpg;
        const int rows = min(P.rpg, P.W - w0) * P.G;       // query rows of the group
        // positions of this thread's columns of S^T (rows 2 c4 and 2 c4 + 1 of each n-tile)
        int pos2[NT][2], tmax = -1, tmin = 0x7fffffff;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = tile * TR + t * 8 + 2 * c4 + e;
                int pos = -1;
                if (i < rows) pos = chunk == 1 && P.rpg == 1 ? s_pos[grp] : usable_pos(P, w0 + i / P.G, false);
                pos2[t][e] = pos;
                tmax = max(tmax, pos);
                tmin = min(tmin, pos);
            }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, d));
            tmin = min(tmin, __shfl_xor_sync(0xffffffffu, tmin, d));
        }
        const int key_lo = split * kSplit;
        if (tmax < key_lo) continue;                       // the same in every warp
        const int nsteps = min(kSplit / kStep, (tmax - key_lo) / kStep + 1);

        // pages of this warp's steps (lane i: step warp + 4 i)
        int page = 0;
        const int slot = P.row_slot[w0];
        if (lane < kStepsPerWarp && warp + kAttnWarps * lane < nsteps)
            page = P.pt.table[static_cast<long long>(slot) * P.pt.max_pages +
                              ((key_lo + kStep * (warp + kAttnWarps * lane)) >> P.pt.page_shift)];
        const bool page_ok = page >= 0 && page < P.pt.n_pages;
        const uint32_t bad_pages = __ballot_sync(0xffffffffu, !page_ok);
        if (!page_ok) {
            atomicOr(&g_paged_err, BIV_DEVERR_INDEX);
            page = 0;
        }

        uint32_t qf[NT][KS][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int i = tile * TR + t * 8 + g8;
            const bool live = i < rows;
            const __nv_bfloat16* qr = P.q + (static_cast<long long>(w0 + (live ? i / P.G : 0)) * P.Hq + kvh * P.G +
                                             (live ? i % P.G : 0)) * HD + 16 * c4;
#pragma unroll
            for (int b = 0; b < KC; ++b) {
                uint32_t r[8];
                ld_row32(qr + 64 * b, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    qf[t][4 * b + k][0] = live ? r[2 * k] : 0u;
                    qf[t][4 * b + k][1] = live ? r[2 * k + 1] : 0u;
                }
            }
        }

        float acc[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][k][e] = 0.0f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
        }
        uint32_t bad_rows = 0;                             // bit 2 t + e: the row met a page id out of range
        uint32_t kr[2][KC][8];                             // keys g8 and g8 + 8 of the step
        uint32_t vr[4][KS];                                // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9: dims [KS * 2 g8, ..)
        const int in_page = P.pt.page_size - 1;
        auto row_at = [&](int i) {                         // element offset of this warp's i-th step
            const int pg = __shfl_sync(0xffffffffu, page, i);
            const int off = (key_lo + kStep * (warp + kAttnWarps * i)) & in_page;
            return ((static_cast<long long>(pg) * P.Hkv + kvh) * P.pt.page_size + off) * HD;
        };
        auto load_k = [&](long long at) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < KC; ++b) ld_row32(P.kp + at + (g8 + 8 * r) * HD + 64 * b + 16 * c4, kr[r][b]);
        };
        auto load_v = [&](long long at) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat16* src = P.vp + at + (2 * c4 + (k & 1) + 8 * (k >> 1)) * HD + 2 * KS * g8;
                if constexpr (KS == 8) ld_row32(src, vr[k]);
                else ld_row16(src, vr[k]);
            }
        };
        const int my_steps = (nsteps - warp + kAttnWarps - 1) / kAttnWarps;
        long long at = 0;
        if (my_steps > 0) {
            at = row_at(0);
            load_k(at);
            load_v(at);
        }
#pragma unroll 1
        for (int i = 0; i < my_steps; ++i) {
            const int key0 = key_lo + kStep * (warp + kAttnWarps * i);
            float st[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 4; ++e) st[t][e] = 0.0f;
                // two chains, so that an MMA does not wait for the one before it
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    const int b = k >> 2, r = 2 * (k & 3);
                    mma_16816(st[t], kr[0][b][r], kr[1][b][r], kr[0][b][r + 1], kr[1][b][r + 1], qf[t][k][0], qf[t][k][1]);
                    mma_16816(s1, kr[0][b][r + 2], kr[1][b][r + 2], kr[0][b][r + 3], kr[1][b][r + 3], qf[t][k + 1][0],
                              qf[t][k + 1][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) st[t][e] += s1[e];
            }
            long long next = 0;
            if (i + 1 < my_steps) {
                next = row_at(i + 1);
                load_k(next);
            }
            if ((bad_pages >> i) & 1u) {                   // a row that reaches this step cannot be computed
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (pos2[t][e] >= key0) bad_rows |= 1u << (2 * t + e);
            }
            if (key0 + kStep - 1 > tmin) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + g8 + 8 * (e >> 1) > pos2[t][e & 1]) st[t][e] = -INFINITY;
                if (key0 + kStep - 1 > tmax) {             // what lies behind the last key may hold anything
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (key0 + 2 * c4 + (k & 1) + 8 * (k >> 1) > tmax) {
#pragma unroll
                            for (int d = 0; d < KS; ++d) vr[k][d] = 0u;
                        }
                }
            }
            uint32_t hi[NT][2], low[NT][2];                // P^T of the step: keys 0-7 and 8-15, transposed to B fragments
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float f[2];
                bool grew = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(st[t][e], st[t][e + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    const float mn = fmaxf(m[t][e], x * P.scale_log2);
                    const float mu = mn == -INFINITY ? 0.0f : mn;
                    f[e] = ex2_approx(m[t][e] - mu);
                    grew |= mn > m[t][e];
                    m[t][e] = mn;
                    const float p0 = ex2_approx(fmaf(st[t][e], P.scale_log2, -mu));
                    const float p1 = ex2_approx(fmaf(st[t][e + 2], P.scale_log2, -mu));
                    st[t][e] = p0;
                    st[t][e + 2] = p1;
                    l[t][e] = fmaf(l[t][e], f[e], p0 + p1);
                }
                if (__any_sync(0xffffffffu, grew)) {       // a factor of a row that did not grow is exactly 1
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[t][k][e] *= f[e & 1];
                }
                // each weight as the sum of two bf16 values: 16 of its bits meet V
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t h = pack_bf16x2(st[t][2 * r], st[t][2 * r + 1]);
                    hi[t][r] = transpose8(h);
                    low[t][r] = transpose8(pack_bf16x2(st[t][2 * r] - bf16lo(h), st[t][2 * r + 1] - bf16hi(h)));
                }
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint32_t a0 = __byte_perm(vr[0][k], vr[1][k], 0x5410), a1 = __byte_perm(vr[0][k], vr[1][k], 0x7632);
                const uint32_t a2 = __byte_perm(vr[2][k], vr[3][k], 0x5410), a3 = __byte_perm(vr[2][k], vr[3][k], 0x7632);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma_16816(acc[t][k], a0, a1, a2, a3, hi[t][0], hi[t][1]);
                    mma_16816(acc[t][k], a0, a1, a2, a3, low[t][0], low[t][1]);
                }
            }
            if (i + 1 < my_steps) load_v(next);
        }

        // the warps' shares of each row, joined in warp order
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], d);
                const int row = t * 8 + 2 * c4 + e;
                if (g8 == 0)
                    s_ml[warp][row] = make_float2(m[t][e], (bad_rows >> (2 * t + e)) & 1u ? -INFINITY : l[t][e]);
                // acc[k][e], acc[k][e + 2]: dims 2 KS g8 + 2 k and + 1 of the row
#pragma unroll
                for (int k = 0; k < KS; k += 2)
                    *reinterpret_cast<float4*>(&s_o[warp][row][2 * KS * g8 + 2 * k]) =
                        make_float4(acc[t][k][e], acc[t][k][e + 2], acc[t][k + 1][e], acc[t][k + 1][e + 2]);
            }
        }
        __syncthreads();
        {
            constexpr int TPR = kAttnThreads / TR;         // threads of a row
            constexpr int DPT = HD / TPR;                  // dims of a thread
            const int row = tid / TPR, d0 = (tid % TPR) * 4;
            const int i = tile * TR + row;
            const int w = w0 + i / P.G;
            int pos = -1;
            if (i < rows) pos = chunk == 1 && P.rpg == 1 ? s_pos[grp] : usable_pos(P, w, false);
            if (pos >= key_lo) {
                float mx = -INFINITY, f[kAttnWarps], sum_l = 0.0f;
#pragma unroll
                for (int k = 0; k < kAttnWarps; ++k) mx = fmaxf(mx, s_ml[k][row].x);
                bool bad = false;
#pragma unroll
                for (int k = 0; k < kAttnWarps; ++k) {
                    const float2 ml = s_ml[k][row];
                    bad |= ml.y == -INFINITY;
                    f[k] = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - mx);
                    sum_l = fmaf(ml.y, f[k], sum_l);
                }
                const long long pair = static_cast<long long>(w) * P.Hq + kvh * P.G + i % P.G;
                const bool whole = pos < kSplit;           // the row's only split
                const float scale = !whole ? 1.0f : bad ? 0.0f : 1.0f / sum_l;
                const long long part = pair * P.s_max + split;
                if (!whole && tid % TPR == 0) P.ws_ml[part] = make_float2(mx, bad ? -1.0f : sum_l);
#pragma unroll
                for (int j = 0; j < DPT / 4; ++j) {
                    const int d = d0 + 4 * TPR * j;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < kAttnWarps; ++k) {
                        const float4 y = *reinterpret_cast<const float4*>(&s_o[k][row][d]);
                        x.x = fmaf(y.x, f[k], x.x);
                        x.y = fmaf(y.y, f[k], x.y);
                        x.z = fmaf(y.z, f[k], x.z);
                        x.w = fmaf(y.w, f[k], x.w);
                    }
                    if (whole) {
                        if (bad) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        *reinterpret_cast<uint2*>(P.o + pair * HD + d) =
                            make_uint2(pack_bf16x2(x.x * scale, x.y * scale), pack_bf16x2(x.z * scale, x.w * scale));
                    } else {
                        *reinterpret_cast<float4*>(P.ws_o + part * HD + d) = x;
                    }
                }
            }
        }
        __syncthreads();
    }
}

// Joins the splits of one (row, head), in an order that goes by their number
// alone: warp k takes splits k, k + 8, ..., and the warps' sums are added in warp
// order.  Rows of a single split were finished by the split kernel.
constexpr int kCombineWarps = 8;

template <int HD>
__global__ void __launch_bounds__(32 * kCombineWarps) paged_combine_kernel(const PagedAttnParams P) {
    constexpr int E = HD / 32;
    __shared__ float s_acc[kCombineWarps][HD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long pair = blockIdx.x;
    const int pos = usable_pos(P, static_cast<int>(pair / P.Hq), false);
    pdl_wait();
    pdl_trigger();
    if (pos < kSplit) return;
    const int ns = pos / kSplit + 1;
    const float2* ml = P.ws_ml + pair * P.s_max;
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int s = lane; s < ns; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int s = lane; s < ns; s += 32) {
        const float2 x = ml[s];
        bad |= x.y == -1.0f;
        l = fmaf(x.y, ex2_approx(x.x - m), l);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    bad = __any_sync(0xffffffffu, bad);
    float acc[E] = {};
    const float* o = P.ws_o + pair * P.s_max * HD + lane * E;
#pragma unroll 8
    for (int s = warp; s < ns; s += kCombineWarps) {
        const float f = ex2_approx(ml[s].x - m);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(o[static_cast<long long>(s) * HD + e], f, acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
    __syncthreads();
    const int d = threadIdx.x;
    if (d < HD) {
        float x = 0.0f;
#pragma unroll
        for (int k = 0; k < kCombineWarps; ++k) x += s_acc[k][d];
        P.o[pair * HD + d] = __float2bfloat16_rn(bad ? 0.0f : x / l);
    }
}

int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Sizes of a paged call; fills pt.
int check_pages(int n_slots, int max_pages, int n_pages, int page_size, PageTable* pt) {
    if (n_slots <= 0 || max_pages <= 0 || n_pages <= 0 || page_size <= 0) return BIV_ERR_SHAPE;
    pt->page_shift = page_shift_of(page_size);
    if (pt->page_shift < 0) return BIV_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_pages) * page_size > 0x7fffffffLL) return BIV_ERR_SHAPE;
    pt->n_slots = n_slots;
    pt->max_pages = max_pages;
    pt->n_pages = n_pages;
    pt->page_size = page_size;
    return BIV_OK;
}

template <int HD, int NT>
int launch_paged_attn(const PagedAttnParams& P, cudaStream_t s) {
    const long long n_groups = (P.W + P.rpg - 1) / P.rpg;
    const long long tiles = (static_cast<long long>(P.rpg) * P.G + 8 * NT - 1) / (8 * NT);
    const long long most = n_groups * P.Hkv * tiles * P.s_max;
    const long long grid = std::min<long long>(most, static_cast<long long>(num_sms()) * (NT == 1 ? 3 : 2));
    int st = launch_pdl(paged_attn_kernel<HD, NT>, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), 0, s, P);
    if (st != BIV_OK || P.s_max == 1) return st;
    const long long pairs = static_cast<long long>(P.W) * P.Hq;
    return launch_pdl(paged_combine_kernel<HD>, dim3(static_cast<unsigned>(pairs)), dim3(32 * kCombineWarps), 0, s, P);
}

template <int HD>
int launch_paged_attn(const PagedAttnParams& P, cudaStream_t s) {
    return static_cast<long long>(P.rpg) * P.G <= 8 ? launch_paged_attn<HD, 1>(P, s) : launch_paged_attn<HD, 2>(P, s);
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" int biv_rope_kv_write_paged(const void* qkv, void* q_out, void* k_pages, void* v_pages,
                                       const int32_t* page_table, const int32_t* row_slot, const int32_t* row_pos,
                                       const int32_t* rows_keep, int W, int K, int Hq, int Hkv, int hd, int n_slots,
                                       int max_pages, int n_pages, int page_size, float theta, biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (W < 0 || K < 1 || Hq <= 0 || Hkv <= 0 || hd <= 0 || hd % 16 != 0 || hd > 256) return BIV_ERR_SHAPE;
    if (W % K != 0 || static_cast<long long>(Hq) + 2LL * Hkv > (1 << 20)) return BIV_ERR_SHAPE;
    PageTable pt;
    const int st = check_pages(n_slots, max_pages, n_pages, page_size, &pt);
    if (st != BIV_OK) return st;
    if (!(theta > 1.0f) || !std::isfinite(theta)) return BIV_ERR_VALUE;
    if (W == 0) return BIV_OK;
    if (!qkv || !q_out || !k_pages || !v_pages || !page_table || !row_slot || !row_pos) return BIV_ERR_NULL;
    if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_pages) || !aligned16(v_pages)) return BIV_ERR_ALIGN;
    pt.table = page_table;
    RopeTurns turns = {};
    for (int i = 0; i < hd / 2; ++i) {
        const double t = std::pow(static_cast<double>(theta), -2.0 * i / hd) * 0.15915494309189533577;   // 1 / 2 pi
        turns.per_pos[i] = static_cast<uint64_t>(std::ldexp(t, 64));
    }
    // few rows: one per CTA, so that all SMs work; many: four, so that the
    // sines of a CTA's rows are one round of its threads
    const int rows = W <= 4 * num_sms() ? 1 : 4;
    return launch_pdl(rope_kv_write_paged_kernel, dim3(static_cast<unsigned>((W + rows - 1) / rows)),
                      dim3(kRopeThreads), static_cast<size_t>(rows) * hd * sizeof(float),
                      reinterpret_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(qkv),
                      static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_pages),
                      static_cast<__nv_bfloat16*>(v_pages), pt, row_slot, row_pos, rows_keep, W, K, Hq, Hkv, hd, rows,
                      turns);
}

extern "C" size_t biv_decode_attn_paged_workspace_size(int W, int Hq, int hd, int max_pages, int page_size) {
    if (W <= 0 || Hq <= 0 || hd <= 0 || max_pages <= 0 || page_size <= 0) return 0;
    const long long splits = (static_cast<long long>(max_pages) * page_size + kSplit - 1) / kSplit;
    return static_cast<size_t>(W) * Hq * static_cast<size_t>(splits) * (hd + 2) * sizeof(float) + 16;
}

extern "C" int biv_decode_attn_paged(const void* q, const void* k_pages, const void* v_pages,
                                     const int32_t* page_table, const int32_t* row_slot, const int32_t* row_pos,
                                     void* o, int W, int rows_per_group, int Hq, int Hkv, int hd, int n_slots,
                                     int max_pages, int n_pages, int page_size, void* workspace, size_t ws_bytes,
                                     biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (W < 0 || rows_per_group <= 0 || Hq <= 0 || Hkv <= 0 || hd <= 0 || Hq % Hkv != 0) return BIV_ERR_SHAPE;
    PagedAttnParams P;
    const int st = check_pages(n_slots, max_pages, n_pages, page_size, &P.pt);
    if (st != BIV_OK) return st;
    if (hd != 64 && hd != 128) return BIV_ERR_UNSUPPORTED;
    if (static_cast<long long>(W) * Hq > 0x7fffffffLL) return BIV_ERR_SHAPE;
    if (W == 0) return BIV_OK;
    if (!q || !k_pages || !v_pages || !page_table || !row_slot || !row_pos || !o || !workspace) return BIV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned16(workspace))
        return BIV_ERR_ALIGN;
    if (ws_bytes < biv_decode_attn_paged_workspace_size(W, Hq, hd, max_pages, page_size)) return BIV_ERR_SHAPE;
    if (o == q) return BIV_ERR_VALUE;
    P.q = static_cast<const __nv_bfloat16*>(q);
    P.kp = static_cast<const __nv_bfloat16*>(k_pages);
    P.vp = static_cast<const __nv_bfloat16*>(v_pages);
    P.pt.table = page_table;
    P.row_slot = row_slot;
    P.row_pos = row_pos;
    P.o = static_cast<__nv_bfloat16*>(o);
    P.W = W;
    P.rpg = std::min(rows_per_group, W);
    P.G = Hq / Hkv;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.cap = max_pages * page_size;
    P.s_max = (P.cap + kSplit - 1) / kSplit;
    P.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(hd)));
    const long long parts = static_cast<long long>(W) * Hq * P.s_max;
    // partial outputs 32-byte aligned
    P.ws_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~static_cast<uintptr_t>(31));
    P.ws_ml = reinterpret_cast<float2*>(P.ws_o + parts * hd);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return hd == 128 ? launch_paged_attn<128>(P, s) : launch_paged_attn<64>(P, s);
}
