// What the attention and the writes over pages share, whatever type the pages hold:
// the page table, the positions' angles, the items of a call and the joins of the
// splits.  Each translation unit that includes it has its own error word.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "biv_common.cuh"

namespace biv {
namespace {

BIV_DEFINE_ERR_WORD(g_paged_err)

constexpr int kSplit = BIV_PAGED_SPLIT;                // keys of a split: the including file says

// Where a pool's rows lie: page p, KV head h, offset t is row (p * Hkv + h) *
// page_size + t of hd elements.
struct PageTable {
    const int32_t* table;      // [n_slots, max_pages]
    int n_slots, max_pages, n_pages, page_size, page_shift;
};

// ---- rotation
// Turns per position of each rotation pair, theta^(-2i/hd) / 2 pi, as 64-bit
// fractions of a turn: position times this, modulo 2^64, is the angle modulo a
// full turn with an error of about pos * 2^-56 turns (the table's doubles: 53 bits
// of at most 1 / 2 pi, below 2^-65 for pairs that turn slowly).
struct RopeTurns {
    uint64_t per_pos[128];     // hd / 2 <= 128
};

// The table of (theta, hd); a thread keeps its last one (64 powers are 2 us of host time).
inline const RopeTurns& rope_turns(float theta, int hd) {
    static thread_local RopeTurns turns;
    static thread_local float of_theta = 0.0f;
    static thread_local int of_hd = 0;
    if (of_theta != theta || of_hd != hd) {
        for (int i = 0; i < hd / 2; ++i) {
            const double t = std::pow(static_cast<double>(theta), -2.0 * i / hd) * 0.15915494309189533577;   // 1 / 2 pi
            turns.per_pos[i] = static_cast<uint64_t>(std::ldexp(t, 64));
        }
        of_theta = theta;
        of_hd = hd;
    }
    return turns;
}

// ---- attention: what every kernel of it shares
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
    uint32_t g_magic;          // ceil(2^32 / G) where that divides every query row's number exactly, else 0
    float scale_log2;          // log2(e) / sqrt(hd)
};

// Window row and head of query row i of a group (i = row * G + head).
BIV_DEV void row_head(const PagedAttnParams& P, int i, int& row, int& head) {
    row = P.g_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), P.g_magic)) : P.G == 1 ? i : i / P.G;
    head = i - row * P.G;
}

// Position of row w if the row is to be computed, else -1; the first row's slot
// decides the group's.  flag: raise the error bits (one thread of a grid).
BIV_DEV int usable_pos(const PagedAttnParams& P, int w, bool flag) {
    const int pos = P.row_pos[w], slot = P.row_slot[w], first = P.row_slot[w - w % P.rpg];
    unsigned int bits = 0;
    if (pos < 0 || pos >= P.cap || slot < 0 || slot >= P.pt.n_slots) bits = BIV_DEVERR_INDEX;
    else if (slot != first) bits = BIV_DEVERR_GROUP;
    if (bits && pos != -1 && flag) atomicOr(&g_paged_err, bits);
    return bits ? -1 : pos;
}

// A split's 16-key steps are taken in turn by four classes of warps (class k: steps k, k + 4, ...).
constexpr int kClasses = 4;
constexpr int kStep = 16;
constexpr int kSteps = kSplit / kStep;                 // steps of a split
constexpr int kStepsPerClass = kSteps / kClasses;
constexpr int kDirectThreads = 32 * kClasses;
constexpr int kMaxGroups = 1024;       // entries of the table of live splits; more groups share entries
constexpr int kMaxRows = BIV_PAGED_ROWS;     // rows whose positions are kept in shared memory; with more they are read again

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

BIV_DEV void cp_async16(void* smem, const void* gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}

// One warp's running softmax over eight query rows: this lane's columns are rows
// 2 (lane % 4) and the next; acc holds HD / 16 tiles of O^T.
template <int HD>
struct RowState {
    static constexpr int KS = HD / 16;
    float acc[KS][4];
    float m[2], l[2];
    float mu[2];               // m, or 0 while no key has counted

    BIV_DEV void clear() {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[k][e] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = mu[0] = mu[1] = 0.0f;
    }

    // Scores of a step (S^T fragment: keys g8 and g8 + 8) to weights: each weight leaves
    // as the sum of two bf16 values, transposed to the B fragments of O^T += V^T P^T.
    // A row's reference m follows its running maximum only when a score passes it by
    // more than kSlack (weights of up to 2^kSlack are as exact as those up to 1), so that
    // most steps need one vote and no exchange of maxima or scaling of the output (32
    // windows of 5 rows: 71.4 -> 68.3 us, one request of 700 keys: 5.8 -> 5.4).
    // Whether a row moves on depends on that row's scores alone (the factor of a row that
    // does not is exactly 1).
    static constexpr float kSlack = 8.0f;
    BIV_DEV void step(float (&st)[4], float scale_log2, uint32_t (&hi)[2], uint32_t (&low)[2]) {
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = fmaxf(st[e], st[e + 2]) * scale_log2;
        if (__any_sync(0xffffffffu, x[0] > m[0] + kSlack || x[1] > m[1] + kSlack)) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                const float y0 = __shfl_xor_sync(0xffffffffu, x[0], d), y1 = __shfl_xor_sync(0xffffffffu, x[1], d);
                x[0] = fmaxf(x[0], y0);
                x[1] = fmaxf(x[1], y1);
            }
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[e] = 1.0f;
                if (x[e] > m[e] + kSlack) {
                    f[e] = ex2_approx(m[e] - x[e]);
                    m[e] = mu[e] = x[e];
                }
                l[e] *= f[e];
            }
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[k][e] *= f[e & 1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st[e] = ex2_approx(fmaf(st[e], scale_log2, -mu[e]));
            st[e + 2] = ex2_approx(fmaf(st[e + 2], scale_log2, -mu[e]));
            l[e] += st[e] + st[e + 2];
        }
        const uint32_t h0 = pack_bf16x2(st[0], st[1]), h1 = pack_bf16x2(st[2], st[3]);
        const uint32_t l0 = pack_bf16x2(st[0] - bf16lo(h0), st[1] - bf16hi(h0));
        const uint32_t l1 = pack_bf16x2(st[2] - bf16lo(h1), st[3] - bf16hi(h1));
        hi[0] = transpose8(h0);
        hi[1] = transpose8(h1);
        low[0] = transpose8(l0);
        low[1] = transpose8(l1);
    }

    // O^T += V^T (hi + low); frag(k, a) gives the A fragment of dims tile k.  The
    // two products of a tile stand kSkew tiles apart, so that the second does not
    // wait for the first.
    template <typename F>
    BIV_DEV void add(const uint32_t (&hi)[2], const uint32_t (&low)[2], F&& frag) {
        constexpr int kSkew = 2;
        uint32_t a[KS][4];
#pragma unroll
        for (int k = 0; k < KS + kSkew; ++k) {
            if (k < KS) {
                frag(k, a[k]);
                mma_16816(acc[k], a[k][0], a[k][1], a[k][2], a[k][3], hi[0], hi[1]);
            }
            if (k >= kSkew) {
                const int j = k - kSkew;
                mma_16816(acc[j], a[j][0], a[j][1], a[j][2], a[j][3], low[0], low[1]);
            }
        }
    }

    // Maximum and sum of every row to ml[row]; a row whose bit e is set in bad met a
    // page id out of range.
    BIV_DEV void put_ml(float2* ml, uint32_t bad, int g8, int c4) const {
        float s0 = l[0], s1 = l[1];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            const float y0 = __shfl_xor_sync(0xffffffffu, s0, d), y1 = __shfl_xor_sync(0xffffffffu, s1, d);
            s0 += y0;
            s1 += y1;
        }
        if (g8 == 0) {
            ml[2 * c4] = make_float2(m[0], bad & 1u ? -INFINITY : s0);
            ml[2 * c4 + 1] = make_float2(m[1], bad & 2u ? -INFINITY : s1);
        }
    }
};

// The last key that every row of an 8-row tile with keys in the split sees: up to there
// nothing needs a mask.  (Rows without keys there are not used.)
BIV_DEV int all_see(const int (&pos)[2], int key_lo) {
    int x = min(pos[0] >= key_lo ? pos[0] : 0x7fffffff, pos[1] >= key_lo ? pos[1] : 0x7fffffff);
    x = min(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return min(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// Scores of keys past a row's position count as -infinity.
BIV_DEV void mask_step(float (&st)[4], const int (&pos)[2], int key0, int g8) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (key0 + g8 + 8 * (e >> 1) > pos[e & 1]) st[e] = -INFINITY;
}

// One item; unit counts (request, split) pairs, sub (KV head, tile).
struct AttnItem {
    int unit, sub;
    int w0, rows;              // first row of the group; its query rows (window rows x G)
    int kvh, tile, split;
};

// Shared memory of both kernels: the positions and the live splits of every group.
struct LiveTable {
    int pre[kMaxGroups + 1];   // live splits before each entry
    int pos[kMaxRows];         // usable position of every row, -1: none
    int slot[kMaxRows];
    int scan[32];
};

// Finds the items of a call: every CTA forms the same table from the rows'
// positions (not an output of the previous kernel, so before the wait).
struct Items {
    const PagedAttnParams& P;
    LiveTable& t;
    int n_groups, chunk, entries, tiles, per_unit;
    bool kept;
    int units, step_unit, step_sub;        // live splits of all groups; a grid's stride in items

    BIV_DEV Items(const PagedAttnParams& p, LiveTable& table, int tile_rows) : P(p), t(table) {
        n_groups = (P.W + P.rpg - 1) / P.rpg;
        chunk = (n_groups + kMaxGroups - 1) / kMaxGroups;
        entries = (n_groups + chunk - 1) / chunk;
        kept = P.W <= kMaxRows;
        tiles = (P.rpg * P.G + tile_rows - 1) / tile_rows;
        per_unit = P.Hkv * tiles;
        step_unit = gridDim.x / per_unit;
        step_sub = gridDim.x - step_unit * per_unit;
        const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        if (kept)
            for (int w = tid; w < P.W; w += threads) {
                t.slot[w] = P.row_slot[w];
                t.pos[w] = usable_pos(P, w, blockIdx.x == 0);
            }
        else if (blockIdx.x == 0)
            for (int w = tid; w < P.W; w += threads) usable_pos(P, w, true);
        __syncthreads();
        const int ept = (entries + threads - 1) / threads;               // entries of a thread
        const int e0 = min(entries, tid * ept), e1 = min(entries, e0 + ept);
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += live_of(e);
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) t.scan[warp] = incl;
        __syncthreads();
        int before = incl - sum;
        units = 0;
        for (int k = 0; k < threads / 32; ++k) {
            if (k < warp) before += t.scan[k];
            units += t.scan[k];
        }
        for (int e = e0; e < e1; ++e) {
            t.pre[e] = before;
            before += live_of(e);
        }
        __syncthreads();
    }

    BIV_DEV int pos_of(int w) const { return kept ? t.pos[w] : usable_pos(P, w, false); }
    BIV_DEV int slot_of(int w) const { return kept ? t.slot[w] : P.row_slot[w]; }
    BIV_DEV int splits_of(int g) const {
        int best = -1;
        const int w1 = min(P.W, (g + 1) * P.rpg);
        for (int w = g * P.rpg; w < w1; ++w) best = max(best, pos_of(w));
        return best / kSplit + (best >= 0);
    }
    BIV_DEV int live_of(int e) const {
        int k = 0;
        for (int g = e * chunk; g < min(n_groups, (e + 1) * chunk); ++g) k += splits_of(g);
        return k;
    }
    // The CTA's first item, and the one after an item; false: there is none.
    // Every lane of a warp asks together.
    BIV_DEV bool first(AttnItem& it) const {
        it.unit = blockIdx.x / per_unit;
        it.sub = blockIdx.x - it.unit * per_unit;
        return it.unit < units && (find(it), true);
    }
    BIV_DEV bool next(const AttnItem& it, AttnItem& nx) const {
        nx.unit = it.unit + step_unit;
        nx.sub = it.sub + step_sub;
        if (nx.sub >= per_unit) {
            nx.sub -= per_unit;
            ++nx.unit;
        }
        return nx.unit < units && (find(nx), true);
    }
    BIV_DEV void find(AttnItem& it) const {
        it.kvh = tiles == 1 ? it.sub : it.sub / tiles;
        it.tile = it.sub - it.kvh * tiles;
        // the last entry with pre <= unit, 32 at a time
        const int lane = threadIdx.x & 31;
        int e = 0;
        if (entries > 32) {
            const bool le = lane * 32 < entries && t.pre[lane * 32] <= it.unit;
            e = (__popc(__ballot_sync(0xffffffffu, le)) - 1) * 32;
        }
        const bool le = e + lane < entries && t.pre[e + lane] <= it.unit;
        e += __popc(__ballot_sync(0xffffffffu, le)) - 1;
        int grp = e;
        it.split = it.unit - t.pre[e];
        if (chunk > 1) {
            for (grp = e * chunk;; ++grp) {
                const int k = splits_of(grp);
                if (it.split < k) break;
                it.split -= k;
            }
        }
        it.w0 = grp * P.rpg;
        it.rows = min(P.rpg, P.W - it.w0) * P.G;
    }
    // Largest position of query rows r0 .. r0 + n - 1 of an item, by a whole warp.
    BIV_DEV int largest_pos(const AttnItem& it, int r0, int n) const {
        int a, b, h, best = -1;
        if (r0 >= it.rows) return -1;
        row_head(P, r0, a, h);
        row_head(P, min(it.rows, r0 + n) - 1, b, h);
        for (int w = it.w0 + a + (threadIdx.x & 31); w <= it.w0 + b; w += 32) best = max(best, pos_of(w));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
        return best;
    }
    BIV_DEV static int steps_to(int tmax, int split) {     // 16-key steps of a split that position tmax reaches
        return tmax < split * kSplit ? 0 : min(kSteps, (tmax - split * kSplit) / kStep + 1);
    }
    // Rows that are not computed come back as zeros.
    template <int HD>
    BIV_DEV void zero_rows() const {
        for (int w = blockIdx.x; w < P.W; w += gridDim.x)
            if (pos_of(w) < 0)
                for (int e = threadIdx.x; e < P.Hq * HD / 8; e += blockDim.x)
                    reinterpret_cast<uint4*>(P.o + static_cast<long long>(w) * P.Hq * HD)[e] = make_uint4(0, 0, 0, 0);
    }
};

// Positions of a lane's two query rows of an 8-row tile that starts at query row r0.
BIV_DEV void tile_pos(const Items& I, int w0, int rows, int r0, int c4, int (&pos)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = r0 + 2 * c4 + e;
        int row, head;
        row_head(I.P, i, row, head);
        pos[e] = i < rows ? I.pos_of(w0 + row) : -1;
    }
}

// Q of `rows` query rows from r0 on, 16 bytes a thread; rows past the group's
// read its first row and are never used.
template <int HD>
BIV_DEV void load_q(const PagedAttnParams& P, const AttnItem& it, int r0, int rows, __nv_bfloat16* dst, int pitch, int tid,
                    int threads) {
    for (int e = tid; e < rows * (HD / 8); e += threads) {
        const int row = e / (HD / 8), d = (e % (HD / 8)) * 8;
        const int i = r0 + row;
        int j, head;
        row_head(P, i < it.rows ? i : 0, j, head);
        cp_async16(dst + row * pitch + d,
                   P.q + (static_cast<long long>(it.w0 + j) * P.Hq + it.kvh * P.G + head) * HD + d);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// How the classes' shares of a row are joined: the row's maximum, the factor of a
// class, and the row's sum.  A sum of -infinity marks a class that met a page id out
// of range; the row's sum is then -1.
BIV_DEV float classes_max(const float2 (&ml)[kClasses]) {
    return fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
}
BIV_DEV float class_factor(const float2& ml, float mx) { return ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - mx); }
BIV_DEV float classes_sum(const float2 (&ml)[kClasses], float mx) {
    float sum = 0.0f;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kClasses; ++k) {
        bad |= ml[k].y == -INFINITY;
        sum = fmaf(ml[k].y, class_factor(ml[k], mx), sum);
    }
    return bad ? -1.0f : sum;
}

// Four classes' scaled outputs of one element, in the order both kernels use.
BIV_DEV float join4(float c0, float c1, float c2, float c3) { return __fadd_rn(__fadd_rn(c0, c2), __fadd_rn(c1, c3)); }

// Four dims of a row from the classes' shares o[class][row], ml[class][row]; the row's
// maximum and sum.
template <int HD, int R>
BIV_DEV float4 join_dims(const float (*o)[R][HD + 4], const float2 (*ml)[R], int row, int d, float& mx, float& sum) {
    float2 c[kClasses];
    float4 y[kClasses];
#pragma unroll
    for (int k = 0; k < kClasses; ++k) {
        c[k] = ml[k][row];
        y[k] = *reinterpret_cast<const float4*>(&o[k][row][d]);
    }
    mx = classes_max(c);
    sum = classes_sum(c, mx);
#pragma unroll
    for (int k = 0; k < kClasses; ++k) {
        const float f = class_factor(c[k], mx);
        y[k].x *= f;
        y[k].y *= f;
        y[k].z *= f;
        y[k].w *= f;
    }
    return make_float4(join4(y[0].x, y[1].x, y[2].x, y[3].x), join4(y[0].y, y[1].y, y[2].y, y[3].y),
                       join4(y[0].z, y[1].z, y[2].z, y[3].z), join4(y[0].w, y[1].w, y[2].w, y[3].w));
}

// Dims d .. d + 3 of one row of a split, joined: a row's only split is finished here,
// others go to the workspace.
template <int HD, int R>
BIV_DEV void join_row(const PagedAttnParams& P, const float (*o)[R][HD + 4], const float2 (*ml)[R], int row, int d, int pos,
                      long long pair, int split) {
    float mx, sum;
    const float4 x = join_dims<HD>(o, ml, row, d, mx, sum);
    if (pos < kSplit) {
        const float scale = 1.0f / sum;
        uint2 z = make_uint2(pack_bf16x2(x.x * scale, x.y * scale), pack_bf16x2(x.z * scale, x.w * scale));
        if (sum == -1.0f) z = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(P.o + pair * HD + d) = z;
    } else {
        const long long part = pair * P.s_max + split;
        if (d == 0) P.ws_ml[part] = make_float2(mx, sum);
        *reinterpret_cast<float4*>(P.ws_o + part * HD + d) = x;
    }
}

// Pages of steps that the lanes have looked up: bit i set where lane i's is out of
// range (flagged, and page 0 read in its place).
BIV_DEV uint32_t bad_pages(const PagedAttnParams& P, int& page) {
    const bool ok = page >= 0 && page < P.pt.n_pages;
    if (!ok) {
        atomicOr(&g_paged_err, BIV_DEVERR_INDEX);
        page = 0;
    }
    return ~__ballot_sync(0xffffffffu, ok);
}

template <typename T>
BIV_DEV T ld_cluster(const T* p, uint32_t rank);
template <>
BIV_DEV float ld_cluster<float>(const float* p, uint32_t rank) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(p, rank)) : "memory");
    return x;
}
template <>
BIV_DEV float2 ld_cluster<float2>(const float2* p, uint32_t rank) {
    float2 x;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(mapa_shared(p, rank)) : "memory");
    return x;
}

// Joins the splits of a (row, head) in an order that goes by their number alone:
// blocks of 16 splits are summed in split order, then the blocks in block order.
// A row of up to kAlone splits is one warp's work; a longer one is shared by all
// warps of its CTA, which take a block each, so that one very long row does not
// wait for one warp's loads.  Rows of a single split were finished by the split
// kernel.
constexpr int kCombineWarps = 16;
constexpr int kBlock = 16;
constexpr int kAlone = 4 * kBlock;
constexpr int kAsk = 32 * kCombineWarps;

// WARPS: 16 for a long row's sake; with more rows than 16 warps on every SM can take at
// once, half of that, so that an SM takes new rows more often (5120 rows of 1 to 32
// splits: 1 us less than with 16; 32 rows of 512 splits: 2 us more).
template <int HD, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, kCombineWarps / WARPS) paged_combine_kernel(const PagedAttnParams P, int per_cta) {
    constexpr int E = HD / 32;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    __shared__ float s_acc[WARPS][HD], s_red[WARPS], s_sum[kAsk / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long pairs = static_cast<long long>(P.W) * P.Hq;
    const long long first = static_cast<long long>(blockIdx.x) * per_cta;
    auto splits_of = [&](int p) {                          // of the CTA's p-th row
        const int pos = p < per_cta && first + p < pairs ? usable_pos(P, static_cast<int>((first + p) / P.Hq), false) : -1;
        return pos < 0 ? 0 : pos / kSplit + 1;
    };
    int ns = splits_of(warp);                              // a row a warp: per_cta <= WARPS
    pdl_wait();
    pdl_trigger();

    // a block's outputs, all under way at once, and their sum in split order
    auto load = [&](long long pair, int s0, int ns, Vec (&v)[kBlock]) {
        const float* o = P.ws_o + (pair * P.s_max + s0) * HD + lane * E;
#pragma unroll
        for (int k = 0; k < kBlock; ++k)
            if (s0 + k < ns) v[k] = *reinterpret_cast<const Vec*>(o + static_cast<long long>(k) * HD);
    };
    auto add = [&](const Vec (&v)[kBlock], int s0, int ns, float factors, int lane0, float (&acc)[E]) {     // lane lane0 + k: split k's factor
#pragma unroll
        for (int k = 0; k < kBlock; ++k) {
            const float f = __shfl_sync(0xffffffffu, factors, lane0 + k);
            if (s0 + k < ns) {
                const float* x = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(x[e], f, acc[e]);
            }
        }
    };
    auto store = [&](long long pair, const float (&x)[E], float inv_l, bool bad) {
        uint32_t y[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) y[e] = bad ? 0u : pack_bf16x2(x[2 * e] * inv_l, x[2 * e + 1] * inv_l);
        __nv_bfloat16* dst = P.o + pair * HD + lane * E;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        else *reinterpret_cast<uint32_t*>(dst) = y[0];
    };

    if (ns > 1 && ns <= kAlone) {
        const long long pair = first + warp;
        // (maximum, sum) of splits lane and lane + 32 and the first outputs, all under way at once
        const float2* ml = P.ws_ml + pair * P.s_max;
        const float2 none = make_float2(-INFINITY, 0.0f);
        const float2 ml0 = lane < ns ? ml[lane] : none, ml1 = lane + 32 < ns ? ml[lane + 32] : none;
        Vec v[kBlock];
        load(pair, 0, ns, v);
        float m = fmaxf(ml0.x, ml1.x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float f0 = lane < ns ? ex2_approx(ml0.x - m) : 0.0f, f1 = lane + 32 < ns ? ex2_approx(ml1.x - m) : 0.0f;
        float l = fmaf(ml1.y, f1, ml0.y * f0);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const bool bad = __any_sync(0xffffffffu, ml0.y == -1.0f || ml1.y == -1.0f);
        float total[E] = {};
        for (int s0 = 0; s0 < ns; s0 += kBlock) {
            float acc[E] = {};
            if (s0 > 0) load(pair, s0, ns, v);
            add(v, s0, ns, s0 < 32 ? f0 : f1, s0 & 31, acc);
#pragma unroll
            for (int e = 0; e < E; ++e) total[e] += acc[e];
        }
        store(pair, total, 1.0f / l, bad);
    }
    if (!__syncthreads_or(ns > kAlone)) return;
    for (int p = 0; p < per_cta && first + p < pairs; ++p) {
        const long long pair = first + p;
        ns = splits_of(p);
        if (ns <= kAlone) continue;
        // maximum and sum over the row's splits: kAsk threads ask for one each at a time,
        // whatever the CTA's size, so that the order of the sum goes by ns alone
        const float2* ml = P.ws_ml + pair * P.s_max;
        float m = -INFINITY;
        for (int s = threadIdx.x; s < ns; s += 32 * WARPS) m = fmaxf(m, ml[s].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (lane == 0) s_red[warp] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WARPS; ++k) m = fmaxf(m, s_red[k]);
        bool bad = false;
#pragma unroll
        for (int t = 0; t < kAsk; t += 32 * WARPS) {
            float l = 0.0f;
            for (int s = t + threadIdx.x; s < ns; s += kAsk) {
                const float2 x = ml[s];
                bad |= x.y == -1.0f;
                l = fmaf(x.y, ex2_approx(x.x - m), l);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            if (lane == 0) s_sum[t / 32 + warp] = l;
        }
        bad = __syncthreads_or(bad);
        float l = 0.0f;
#pragma unroll
        for (int k = 0; k < kAsk / 32; ++k) l += s_sum[k];
        float total[E] = {};
        for (int s0 = 0; s0 < ns; s0 += kBlock * WARPS) {          // a block of each warp
            const int mine = s0 + kBlock * warp;
            if (mine < ns) {
                const int at = mine + (lane & (kBlock - 1));
                const float f = at < ns ? ex2_approx(ml[at].x - m) : 0.0f;
                float acc[E] = {};
                Vec v[kBlock];
                load(pair, mine, ns, v);
                add(v, mine, ns, f, 0, acc);
#pragma unroll
                for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
            }
            __syncthreads();
            if (warp == 0)
                for (int k = 0; k < WARPS && s0 + kBlock * k < ns; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e) total[e] += s_acc[k][lane * E + e];
            __syncthreads();
        }
        if (warp == 0) store(pair, total, 1.0f / l, bad);
    }
}

inline int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Sizes of a paged call; fills pt.
inline int check_pages(int n_slots, int max_pages, int n_pages, int page_size, PageTable* pt) {
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

// The parameters of an attention call but for its pools; P.pt's sizes have been checked.
inline void fill_attn(PagedAttnParams& P, const void* q, void* o, const int32_t* page_table, const int32_t* row_slot,
                      const int32_t* row_pos, int W, int rows_per_group, int Hq, int Hkv, int hd, int max_pages, int page_size,
                      void* workspace) {
    P.q = static_cast<const __nv_bfloat16*>(q);
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
    // i / G by a multiplication: exact while i * G stays below 2^32
    P.g_magic = P.G > 1 && static_cast<double>(P.rpg) * P.G * P.G < 4294967296.0
                    ? static_cast<uint32_t>((4294967296ull + P.G - 1) / P.G)
                    : 0u;
    P.s_max = (P.cap - 1) / kSplit + 1;                    // no sum that passes 31 bits
    P.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(hd)));
    const long long parts = static_cast<long long>(W) * Hq * P.s_max;
    // partial outputs 32-byte aligned
    P.ws_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~static_cast<uintptr_t>(31));
    P.ws_ml = reinterpret_cast<float2*>(P.ws_o + parts * hd);
}

// The join of the splits, where a row may have several.
template <int HD>
int launch_combine(const PagedAttnParams& P, cudaStream_t s) {
    // few rows: a CTA each, so that a long row has the whole CTA
    const long long pairs = static_cast<long long>(P.W) * P.Hq;
    const bool few = pairs <= static_cast<long long>(kCombineWarps) * num_sms();
    const int per_cta = few ? static_cast<int>((pairs + num_sms() - 1) / num_sms()) : kCombineWarps / 2;
    return launch_pdl(few ? paged_combine_kernel<HD, kCombineWarps> : paged_combine_kernel<HD, kCombineWarps / 2>,
                      dim3(static_cast<unsigned>((pairs + per_cta - 1) / per_cta)),
                      dim3(32 * (few ? kCombineWarps : kCombineWarps / 2)), 0, s, P, per_cta);
}

}  // namespace
}  // namespace biv
