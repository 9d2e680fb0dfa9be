// The paged key-value cache: rotation and write of new rows into pages, and
// fixed-split decode attention over them.
#include <algorithm>
#include <cmath>
#include <type_traits>

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
// full turn with an error of about pos * 2^-56 turns (the table's doubles: 53 bits
// of at most 1 / 2 pi, below 2^-65 for pairs that turn slowly).
struct RopeTurns {
    uint64_t per_pos[128];     // hd / 2 <= 128
};

// The table of (theta, hd); a thread keeps its last one (64 powers are 2 us of host time).
const RopeTurns& rope_turns(float theta, int hd) {
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

constexpr int kRopeThreads = 256;

// One CTA per `rows` consecutive rows.  Its threads first take the sines and
// cosines of the rows' angles (one each, in shared memory), then rotate: an
// item is eight pairs of one head, two 16-byte loads and two 16-byte stores, so
// every sector that is touched is used whole.  Bound by memory: 2 x (Hq + 2 Hkv)
// hd x 2 bytes per row (4095 rows of 32 + 16 heads of 128: 19.8 us, 5.1 TB/s; all loads
// first, or the rows brought into L2 while the angles are computed, is not faster).
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

// ---- the split kernels
// One item is (request, KV head, 256-key split, tile of query rows), where the
// query rows are the request's window rows times the G heads of the KV head.
// Keys go along the M side of the tensor core's tile and query rows along N
// (mma.m16n8k16): S^T = K Q^T and O^T = V^T P^T, so eight rows fill a tile and
// the four rows of a single token waste half of it instead of the 60 of 64 that
// a rows-by-keys tile would.  Four classes of warps take the split's 16-key
// steps in turn (class k: steps k, k + 4, ...), each with its own running maximum
// and sum, and meet once at the end in class order.  These kernels run that same
// program, with the same bits for a row:
//   direct  up to 8 query rows (one new token): the permutation of the dims
//           inside a product is free, and chosen so that K and V come straight
//           from global memory in 32-byte loads, a whole 128-byte line per four
//           (K) or eight (V) lanes: no shared memory, no barrier and no address
//           arithmetic between HBM and the tensor core.  Bound by memory: 64
//           requests of 256 to 8192 keys 60.4 us, one of 131071 keys 90.3,
//           both 5.9 TB/s with the join (a plain copy: 6.8).
//   small   few tiles of eight rows and short tables: the same loads, in one launch.
//   staged  more rows (verify windows): K and V pass through a ring in shared
//           memory, filled by TMA, so that up to four tiles of 8 rows share one
//           read of the keys.
constexpr int kClasses = 4;
constexpr int kStep = 16;
constexpr int kSteps = kSplit / kStep;                 // steps of a split
constexpr int kStepsPerClass = kSteps / kClasses;
constexpr int kDirectThreads = 32 * kClasses;
constexpr int kMaxGroups = 1024;       // entries of the table of live splits; more groups share entries
constexpr int kMaxRows = 2048;         // rows whose positions are kept in shared memory; with more they are read again

// 32 or 16 bytes of a row of keys or values: read once, so not kept in L1, and first to
// leave L2 (the 32-byte form has that hint), where the splits' partials shall stay for
// the join (64 requests: 65.7 us without the hint, 61.2 with it).
BIV_DEV void ld_row(const __nv_bfloat16* p, uint32_t (&r)[8]) {
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
BIV_DEV void ld_row(const __nv_bfloat16* p, uint32_t (&r)[4]) {
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
template <int HD>
BIV_DEV float4 join_dims(const float (*o)[8][HD + 4], const float2 (*ml)[8], int row, int d, float& mx, float& sum) {
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
template <int HD>
BIV_DEV void join_row(const PagedAttnParams& P, const float (*o)[8][HD + 4], const float2 (*ml)[8], int row, int d, int pos,
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

// A warp of the direct kernels: the keys and values of one 16-key step in registers.
template <int HD>
struct DirectKeys {
    static constexpr int KS = HD / 16;             // k-steps of S^T; also the 16-dim tiles of O^T
    static constexpr int KC = HD / 64;             // 64-dim chunks of a key: one 32-byte load per lane each
    uint32_t kr[2][KC][8];                         // keys g8 and g8 + 8
    uint32_t vr[4][KS];                            // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9: dims [2 KS g8, ..)

    BIV_DEV void load_k(const PagedAttnParams& P, long long at, int g8, int c4) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < KC; ++b) ld_row(P.kp + at + (g8 + 8 * r) * HD + 64 * b + 16 * c4, kr[r][b]);
    }
    BIV_DEV void load_v(const PagedAttnParams& P, long long at, int g8, int c4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) ld_row(P.vp + at + (2 * c4 + (k & 1) + 8 * (k >> 1)) * HD + 2 * KS * g8, vr[k]);
    }
    // S^T of the step; q: this lane's query row g8 from dim 16 c4 on.  Two chains, so that
    // an MMA does not wait for the one before it.
    BIV_DEV void scores(const __nv_bfloat16* q, float (&st)[4]) const {
        float s2[2][4] = {};
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
            const int b = k >> 2, r = 2 * (k & 3);
            const uint4 qv = *reinterpret_cast<const uint4*>(q + 64 * b + 2 * r);
            mma_16816(s2[0], kr[0][b][r], kr[1][b][r], kr[0][b][r + 1], kr[1][b][r + 1], qv.x, qv.y);
            mma_16816(s2[1], kr[0][b][r + 2], kr[1][b][r + 2], kr[0][b][r + 3], kr[1][b][r + 3], qv.z, qv.w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) st[e] = s2[0][e] + s2[1][e];
    }
    // The step's weights and O^T; what lies behind the last key (tmax) may hold anything.
    // see: all_see of the rows.
    BIV_DEV void accumulate(RowState<HD>& rs, float (&st)[4], const int (&pos)[2], int see, int tmax, int key0, int g8, int c4,
                            float scale_log2) {
        if (key0 + kStep - 1 > see) {
            mask_step(st, pos, key0, g8);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (key0 + 2 * c4 + (k & 1) + 8 * (k >> 1) > tmax) {
#pragma unroll
                    for (int d = 0; d < KS; ++d) vr[k][d] = 0u;
                }
        }
        uint32_t hi[2], low[2];
        rs.step(st, scale_log2, hi, low);
        rs.add(hi, low, [&](int k, uint32_t (&a)[4]) {
            a[0] = __byte_perm(vr[0][k], vr[1][k], 0x5410);
            a[1] = __byte_perm(vr[0][k], vr[1][k], 0x7632);
            a[2] = __byte_perm(vr[2][k], vr[3][k], 0x5410);
            a[3] = __byte_perm(vr[2][k], vr[3][k], 0x7632);
        });
    }
    // acc[k][e], acc[k][e + 2]: dims 2 KS g8 + 2 k and + 1 of row 2 c4 + e
    BIV_DEV static void put(const RowState<HD>& rs, float (*o)[HD + 4], int g8, int c4) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < KS; k += 2)
                *reinterpret_cast<float4*>(&o[2 * c4 + e][2 * KS * g8 + 2 * k]) =
                    make_float4(rs.acc[k][e], rs.acc[k][e + 2], rs.acc[k + 1][e], rs.acc[k + 1][e + 2]);
    }
};

// Element offset of the row of a pool where a 16-key step starts.
template <int HD>
BIV_DEV long long step_at(const PagedAttnParams& P, int page, int kvh, int key0) {
    return ((static_cast<long long>(page) * P.Hkv + kvh) * P.pt.page_size + (key0 & (P.pt.page_size - 1))) * HD;
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

template <int HD>
struct __align__(16) DirectSmem {
    float o[kClasses][8][HD + 4];          // rows padded against bank conflicts
    __nv_bfloat16 q[2][8][HD + 8];
    float2 ml[kClasses][8];
    LiveTable table;
};

template <int HD>
__global__ void __launch_bounds__(kDirectThreads, 3) paged_attn_direct_kernel(const PagedAttnParams P) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DirectSmem<HD>& sm = *reinterpret_cast<DirectSmem<HD>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, cls = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;       // row of an 8-row fragment, column pair
    const Items I(P, sm.table, 8);
    pdl_wait();
    pdl_trigger();
    I.zero_rows<HD>();

    DirectKeys<HD> keys;
    auto page_of = [&](const AttnItem& it, int nsteps) {        // lane i: page of this class's i-th step
        int page = 0;
        if (lane < kStepsPerClass && cls + kClasses * lane < nsteps)
            page = P.pt.table[static_cast<long long>(I.slot_of(it.w0)) * P.pt.max_pages +
                              ((it.split * kSplit + kStep * (cls + kClasses * lane)) >> P.pt.page_shift)];
        return page;
    };
    auto row_at = [&](const AttnItem& it, int page, int i) {           // where this class's i-th step lies
        return step_at<HD>(P, __shfl_sync(0xffffffffu, page, i), it.kvh, it.split * kSplit + kStep * (cls + kClasses * i));
    };
    auto steps_of = [&](int nsteps) { return (nsteps - cls + kClasses - 1) / kClasses; };

    AttnItem cur, nxt;
    if (!I.first(cur)) return;
    load_q<HD>(P, cur, 0, 8, &sm.q[0][0][0], HD + 8, tid, kDirectThreads);
    // the group's largest position, each lane's rows' and the steps that some row reaches
    auto describe = [&](const AttnItem& it, int (&pos)[2], int& tmax) {
        tile_pos(I, it.w0, it.rows, 0, c4, pos);
        tmax = max(pos[0], pos[1]);
        if (P.rpg > 1) {
            tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
            tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
        } else {
            tmax = I.pos_of(it.w0);
        }
        return Items::steps_to(tmax, it.split);
    };
    int cur_pos[2], nxt_pos[2], cur_tmax, nxt_tmax = -1;
    int cur_steps = describe(cur, cur_pos, cur_tmax), nxt_steps = 0;
    int cur_page = page_of(cur, cur_steps), nxt_page = 0;
    uint32_t cur_bad = bad_pages(P, cur_page), nxt_bad = 0;
    if (steps_of(cur_steps) > 0) {
        const long long at = row_at(cur, cur_page, 0);
        keys.load_k(P, at, g8, c4);
        keys.load_v(P, at, g8, c4);
    }
    for (int buf = 0;; buf ^= 1) {
        // this item's Q has landed; every class has joined the item before
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        const bool more = I.next(cur, nxt);
        if (more) {
            load_q<HD>(P, nxt, 0, 8, &sm.q[buf ^ 1][0][0], HD + 8, tid, kDirectThreads);
            nxt_steps = describe(nxt, nxt_pos, nxt_tmax);
            nxt_page = page_of(nxt, nxt_steps);
        }
        RowState<HD> rs;
        rs.clear();
        uint32_t bad_rows = 0;                     // bit e: the row met a page id out of range
        const int my_steps = steps_of(cur_steps), see = all_see(cur_pos, cur.split * kSplit);
        long long next_at = 0;
        bool next = false;
#pragma unroll 1
        for (int i = 0; i < my_steps; ++i) {
            const int key0 = cur.split * kSplit + kStep * (cls + kClasses * i);
            float st[4];
            keys.scores(&sm.q[buf][g8][16 * c4], st);
            // the keys of this class's next step, or of its first step of the next item
            next = i + 1 < my_steps;
            if (next) {
                next_at = row_at(cur, cur_page, i + 1);
            } else if (more) {
                nxt_bad = bad_pages(P, nxt_page);
                next = steps_of(nxt_steps) > 0;
                if (next) next_at = row_at(nxt, nxt_page, 0);
            }
            if (next) keys.load_k(P, next_at, g8, c4);
            const bool bad = (cur_bad >> i) & 1u;  // a row that reaches this step cannot be computed; for the others its values are none
            if (bad) bad_rows |= (cur_pos[0] >= key0 ? 1u : 0u) | (cur_pos[1] >= key0 ? 2u : 0u);
            keys.accumulate(rs, st, cur_pos, see, bad ? -1 : cur_tmax, key0, g8, c4, P.scale_log2);
            if (next) keys.load_v(P, next_at, g8, c4);
        }
        if (my_steps == 0 && more) {
            nxt_bad = bad_pages(P, nxt_page);
            if (steps_of(nxt_steps) > 0) {
                next_at = row_at(nxt, nxt_page, 0);
                keys.load_k(P, next_at, g8, c4);
                keys.load_v(P, next_at, g8, c4);
            }
        }
        rs.put_ml(sm.ml[cls], bad_rows, g8, c4);
        DirectKeys<HD>::put(rs, sm.o[cls], g8, c4);
        __syncthreads();
        for (int x4 = tid; x4 < 8 * (HD / 4); x4 += kDirectThreads) {
            const int row = x4 / (HD / 4), d = (x4 % (HD / 4)) * 4;
            if (row >= cur.rows) break;
            int j, head;
            row_head(P, row, j, head);
            const int pos = I.pos_of(cur.w0 + j);
            if (pos >= cur.split * kSplit)
                join_row<HD>(P, sm.o, sm.ml, row, d, pos, static_cast<long long>(cur.w0 + j) * P.Hq + cur.kvh * P.G + head, cur.split);
        }
        if (!more) break;
        cur = nxt;
        cur_pos[0] = nxt_pos[0];
        cur_pos[1] = nxt_pos[1];
        cur_tmax = nxt_tmax;
        cur_steps = nxt_steps;
        cur_page = nxt_page;
        cur_bad = nxt_bad;
    }
}

// ---- small calls: a cluster of C CTAs per (request, KV head, 8 query rows), CTA c taking
// splits c and c + C; the partials stay in shared memory, and CTA c joins query rows c,
// c + C, ... of all splits.  One launch and no workspace traffic where the direct kernel
// and the combine kernel would mostly wait for one another (1 request of 700 keys: 7.9 us
// for the two, 5.5 so).  The same steps, joins and bits.
constexpr int kSmallTurns = 2;                     // splits a CTA takes at most

template <int HD, int C>
struct __align__(16) SmallSmem {
    float o[kClasses][8][HD + 4];
    float part[kSmallTurns][8][HD];        // this CTA's splits' outputs
    float2 part_ml[kSmallTurns][8];
    __nv_bfloat16 q[8][HD + 8];
    float2 ml[kClasses][8];
};

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

template <int HD, int C>
__global__ void __launch_bounds__(kDirectThreads, 2) paged_attn_small_kernel(const PagedAttnParams P) {
    __shared__ SmallSmem<HD, C> sm;
    const int tid = threadIdx.x, lane = tid & 31, cls = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;
    const int rank = static_cast<int>(cluster_ctarank());
    const int tiles = (P.rpg * P.G + 7) / 8, p = blockIdx.x / C / tiles, tile = blockIdx.x / C - p * tiles;
    const int grp = p / P.Hkv, kvh = p - grp * P.Hkv;
    const int w0 = grp * P.rpg, r0 = 8 * tile, rows = min(8, min(P.rpg, P.W - w0) * P.G - r0);   // none: a last group that is not full
    int pos[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * c4 + e;
        pos[e] = i < rows ? usable_pos(P, w0 + (r0 + i) / P.G, rank == 0 && kvh == 0) : -1;
    }
    int tmax = max(pos[0], pos[1]);
    tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
    tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
    // pages of this class's steps of both splits (lane kStepsPerClass j + i: step i of split rank + C j)
    int page = 0;
    {
        const int key0 = (rank + C * (lane / kStepsPerClass)) * kSplit + kStep * (cls + kClasses * (lane % kStepsPerClass));
        if (lane < kStepsPerClass * kSmallTurns && key0 <= tmax)
            page = P.pt.table[static_cast<long long>(P.row_slot[w0]) * P.pt.max_pages + (key0 >> P.pt.page_shift)];
    }
    const uint32_t bad = bad_pages(P, page);
    pdl_wait();
    pdl_trigger();
    for (int e = tid; e < 8 * (HD / 8); e += kDirectThreads) {         // rows past the group's read its first row and are never used
        const int row = e / (HD / 8), d = (e % (HD / 8)) * 8, i = row < rows ? r0 + row : 0;
        cp_async16(&sm.q[row][d], P.q + (static_cast<long long>(w0 + i / P.G) * P.Hq + kvh * P.G + i % P.G) * HD + d);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    DirectKeys<HD> keys;
    auto steps_of = [&](int j) {                           // of this class, of the j-th split; a later split has no more
        return j < kSmallTurns ? (Items::steps_to(tmax, rank + C * j) - cls + kClasses - 1) / kClasses : 0;
    };
    auto at = [&](int j, int i) {
        return step_at<HD>(P, __shfl_sync(0xffffffffu, page, kStepsPerClass * j + i), kvh,
                           (rank + C * j) * kSplit + kStep * (cls + kClasses * i));
    };
    if (steps_of(0) > 0) {
        const long long a = at(0, 0);
        keys.load_k(P, a, g8, c4);
        keys.load_v(P, a, g8, c4);
    }
    for (int j = 0; j < kSmallTurns; ++j) {
        const int split = rank + C * j, steps = steps_of(j);
        if (split * kSplit > tmax) break;                  // the same in every warp
        const int see = all_see(pos, split * kSplit);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                   // Q has landed; the split before is joined
        RowState<HD> rs;
        rs.clear();
        uint32_t bad_rows = 0;
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            const int key0 = split * kSplit + kStep * (cls + kClasses * i);
            float st[4];
            keys.scores(&sm.q[g8][16 * c4], st);
            // the next step, or the next split's first
            const bool here = i + 1 < steps, more = here || steps_of(j + 1) > 0;
            long long next = 0;
            if (more) {
                next = here ? at(j, i + 1) : at(j + 1, 0);
                keys.load_k(P, next, g8, c4);
            }
            const bool step_bad = (bad >> (kStepsPerClass * j + i)) & 1u;
            if (step_bad) bad_rows |= (pos[0] >= key0 ? 1u : 0u) | (pos[1] >= key0 ? 2u : 0u);
            keys.accumulate(rs, st, pos, see, step_bad ? -1 : tmax, key0, g8, c4, P.scale_log2);
            if (more) keys.load_v(P, next, g8, c4);
        }
        rs.put_ml(sm.ml[cls], bad_rows, g8, c4);
        DirectKeys<HD>::put(rs, sm.o[cls], g8, c4);
        __syncthreads();
        for (int x4 = tid; x4 < 8 * (HD / 4); x4 += kDirectThreads) {
            const int row = x4 / (HD / 4), d = (x4 % (HD / 4)) * 4;
            float mx, sum;
            const float4 x = join_dims<HD>(sm.o, sm.ml, row, d, mx, sum);
            *reinterpret_cast<float4*>(&sm.part[j][row][d]) = x;
            if (d == 0) sm.part_ml[j][row] = make_float2(mx, sum);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    cluster_sync();
    // query rows rank, rank + C, ..., joined as the combine kernel does (up to 16 splits: one block)
    for (int r = rank; r < rows; r += C) {
        const int w = w0 + (r0 + r) / P.G;
        const int row_pos = usable_pos(P, w, false), ns = row_pos < 0 ? 0 : row_pos / kSplit + 1;
        const long long pair = static_cast<long long>(w) * P.Hq + kvh * P.G + (r0 + r) % P.G;
        const float2 mine = lane < ns ? ld_cluster(&sm.part_ml[lane / C][r], lane % C)
                                      : make_float2(-INFINITY, 0.0f);
        float x[kSmallTurns * C] = {};
        if (tid < HD) {
#pragma unroll
            for (int k = 0; k < kSmallTurns * C; ++k)
                if (k < ns) x[k] = ld_cluster(&sm.part[k / C][r][tid], k % C);
        }
        float m = mine.x, l;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float f_lane = lane < ns ? ex2_approx(mine.x - m) : 0.0f;
        l = mine.y * f_lane;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const bool broken = __any_sync(0xffffffffu, lane < ns && mine.y == -1.0f);
        float acc = 0.0f;
#pragma unroll
        for (int k = 0; k < kSmallTurns * C; ++k) {
            const float f = __shfl_sync(0xffffffffu, f_lane, k);
            if (k < ns) acc = fmaf(x[k], f, acc);
        }
        if (tid < HD) P.o[pair * HD + tid] = __float2bfloat16_rn(broken || ns == 0 ? 0.0f : acc * (1.0f / l));
    }
    cluster_sync();                                        // nobody leaves while its shared memory is read
}

// ---- staged: one CTA per SM; one producer warp prepares items (Q and the pages), the
// next fills a ring of rounds (the classes' 16-key steps, 64 keys: K, then V) for T
// groups of four consumer warps, one per class.  Group g takes tile g of every item.
// K and V come in TMA boxes of a page's keys, up to a round's: HD / 64 tiles of rows of
// 128 bytes, swizzled, so that the fragments' reads meet no bank twice.
// 32 windows of 5 rows (20 query rows a KV head: 3 tiles; 8 KV heads of 128, 1024 keys at
// the median): 61 us with the join of the splits, 3.5 TB/s of keys.  Larger boxes and a
// warp for the items, since one TMA instruction keeps its warp some 85 cycles (a copy
// per key's row: 240 us).  What bounds it is the serial work of a consumer warp, of
// which registers allow three a scheduler: a step takes some 400 + 360 + 340 cycles
// (scores, weights, values), an item's join 2000 more after four of them; the tensor
// pipe is a fifth busy, shared memory half.  Splits of 512 keys would take a tenth off,
// and add a third to one request's step on a short context.
constexpr int kMaxStages = 6;

struct StagedItem {
    int kvh, split, nsteps, tmax;           // nsteps = 0: no more items
    uint32_t bad;                           // bit i: the page id of step i is out of range
    int page[kSteps];
    alignas(8) int pos[32];                 // of the rows of all tiles, -1: no row (read two at a time)
    long long pair[32];                     // their (row, head)
};

struct StagedBars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t item_set[3], item_full[3], item_empty[3];     // the item alone, the item and its Q, free
    StagedItem item[3];
    int abort_flag;
};
constexpr int kBarBytes = (static_cast<int>(sizeof(StagedBars)) + 15) / 16 * 16;

template <int HD, int T>
struct StagedLayout {
    static constexpr int kRows = 8 * T, kSlots = 3, QP = HD + 8, HDP = HD + 4;
    static constexpr int kHalf = kClasses * kStep * HD * 2;             // bytes of a stage's K (or V)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kBars = (static_cast<int>(sizeof(LiveTable)) + 15) / 16 * 16;
    static constexpr int kQ = kBars + kBarBytes;                              // [slots][rows][QP] bf16
    static constexpr int kMl = kQ + kSlots * kRows * QP * 2;            // [groups][classes][8] float2
    static constexpr int kO = kMl + T * kClasses * 8 * 8;               // [groups][classes][8][HDP] float
    static constexpr int kRing = (kO + T * kClasses * 8 * HDP * 4 + 1023) / 1024 * 1024;   // the swizzle goes by the address
    static constexpr int kFit = (226 * 1024 - kRing) / kStage;
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr int kBytes = kRing + kStages * kStage + 1024;      // the base is aligned to 1024
    static_assert(kStages >= 2, "the ring needs two stages");
};

constexpr int kRoundKeys = kClasses * kStep;

// Four 8 x 8 tiles of bf16, transposed: the A fragment of V^T for 16 dims and 16 keys.
BIV_DEV void ldmatrix_x4_trans(uint32_t addr, uint32_t (&a)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(addr)
                 : "memory");
}

BIV_DEV void group_bar(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
// The barrier and a vote: true if every thread of the group says so.
BIV_DEV bool group_all(int group, bool ok) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(1 + group), "r"(ok ? 1u : 0u)
                 : "memory");
    return r != 0;
}
BIV_DEV void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int HD, int T>
__global__ void __launch_bounds__(T * 128 + 64, 1) paged_attn_staged_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                            const __grid_constant__ CUtensorMap tmV, const PagedAttnParams P) {
    using L = StagedLayout<HD, T>;
    constexpr int KS = HD / 16;
    extern __shared__ uint8_t smem_base[];
    uint8_t* smem_raw = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_base) + 1023) & ~static_cast<uintptr_t>(1023));
    LiveTable& table = *reinterpret_cast<LiveTable*>(smem_raw);
    StagedBars& bars = *reinterpret_cast<StagedBars*>(smem_raw + L::kBars);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], kClasses * T);
        }
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(&bars.item_set[s], 1);
            mbar_init(&bars.item_full[s], 33);             // 32 lanes' copies and one plain arrival
            mbar_init(&bars.item_empty[s], kClasses * T);
        }
        bars.abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    const Items I(P, table, L::kRows);                     // its barriers also publish the mbarriers
    pdl_wait();
    pdl_trigger();
    I.zero_rows<HD>();

    const int box_keys = min(P.pt.page_size, kRoundKeys);
    int slot = 0;
    uint32_t slot_phase = 0;
    auto next_slot = [&]() {
        if (++slot == L::kSlots) {
            slot = 0;
            slot_phase ^= 1u;
        }
    };
    int stage = 0;
    uint32_t phase = 0;
    auto next_stage = [&]() {
        if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
               __all_sync(0xffffffffu, mbar_wait(bar, parity, &bars.abort_flag, &g_paged_err));
    };
    if (warp == T * kClasses) {
        // -------------------------------------------------- items and their Q
        AttnItem it;
        bool ok = true;
        for (bool more = I.first(it); more; more = I.next(it, it)) {
            const int r0 = it.tile * L::kRows;
            const int tmax = I.largest_pos(it, r0, L::kRows), nsteps = Items::steps_to(tmax, it.split);
            if (nsteps == 0) continue;
            int page = 0;                                  // lane i: page of step i
            if (lane < nsteps)
                page = P.pt.table[static_cast<long long>(I.slot_of(it.w0)) * P.pt.max_pages +
                                  ((it.split * kSplit + kStep * lane) >> P.pt.page_shift)];
            const bool real = lane < L::kRows && r0 + lane < it.rows;
            int j, head;                                   // of row `lane`; rows past the group's read its first row and are never used
            row_head(P, real ? r0 + lane : 0, j, head);
            const long long pair = static_cast<long long>(it.w0 + j) * P.Hq + it.kvh * P.G + head;
            ok = wait(&bars.item_empty[slot], slot_phase ^ 1u);
            if (!ok) break;
            constexpr int RPI = 32 / (HD / 8);             // rows of one copy instruction
            const int ck = lane % (HD / 8), rk = lane / (HD / 8);
            __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(smem_raw + L::kQ) + slot * L::kRows * L::QP;
#pragma unroll
            for (int r = 0; r < L::kRows; r += RPI)
                cp_async16(q + (r + rk) * L::QP + ck * 8, P.q + __shfl_sync(0xffffffffu, pair, r + rk) * HD + ck * 8);
            const uint32_t bad = bad_pages(P, page);
            StagedItem& d = bars.item[slot];
            if (lane < kSteps) d.page[lane] = page;
            d.pos[lane] = real ? I.pos_of(it.w0 + j) : -1;
            d.pair[lane] = pair;
            if (lane == 0) {
                d.kvh = it.kvh;
                d.split = it.split;
                d.nsteps = nsteps;
                d.tmax = tmax;
                d.bad = bad;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars.item_set[slot]);
                mbar_arrive(&bars.item_full[slot]);
            }
            cp_async_arrive(&bars.item_full[slot]);
            next_slot();
        }
        if (ok && wait(&bars.item_empty[slot], slot_phase ^ 1u)) {
            if (lane == 0) {
                bars.item[slot].nsteps = 0;
                mbar_arrive(&bars.item_set[slot]);
                mbar_arrive(&bars.item_full[slot]);
            }
            cp_async_arrive(&bars.item_full[slot]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    if (warp > T * kClasses) {
        // ------------------------------------------------------ keys and values
        // keys that one item alone reads leave L2 first; other tiles of the rows read them again
        const uint64_t policy = I.tiles == 1 ? policy_evict_first() : policy_evict_normal();
        const int boxes = kRoundKeys / box_keys, box_bytes = box_keys * HD * 2;
        const bool is_v = lane >= boxes;                   // a lane per box: K, then V
        const int box = is_v ? lane - boxes : lane, box_step = box * (box_keys / kStep);
        int fills = 0;
        bool ok = true;
        while (ok && wait(&bars.item_set[slot], slot_phase)) {
            const StagedItem& it = bars.item[slot];
            const int nsteps = it.nsteps, kvh = it.kvh;    // after the last copy the item may be another
            if (nsteps == 0) break;
            const uint32_t bad = it.bad;
            for (int s0 = 0; s0 < nsteps; s0 += kClasses) {
                const int step = s0 + box_step;
                // boxes that no row reaches, or whose page is none, are not copied
                const bool live = lane < 2 * boxes && step < nsteps && !((bad >> step) & 1u);
                const int page = live ? it.page[step] : 0, key = (kStep * step) & (P.pt.page_size - 1);
                const int n = __popc(__ballot_sync(0xffffffffu, live));
                ok = wait(&bars.empty[stage], phase ^ 1u);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&bars.full[stage], static_cast<uint32_t>(n * box_bytes));
                __syncwarp();
                if (live)
                    tma_load_5d(smem_raw + L::kRing + stage * L::kStage + (is_v ? L::kHalf : 0) + box * box_bytes, is_v ? &tmV : &tmK,
                                &bars.full[stage], 0, key, 0, kvh, page, policy);
                ++fills;
                next_stage();
            }
            next_slot();
        }
        // no copy may land after the CTA has left (the consumers see all of them complete,
        // unless a wait ran out)
        if (lane == 0)
            for (int s = 0; s < L::kStages; ++s)
                if (fills > s) mbar_wait_drain(&bars.full[s], s < stage ? phase : phase ^ 1u);
        return;
    }

    // ---------------------------------------------------------- consumers
    const int g8 = lane >> 2, c4 = lane & 3;
    const int group = warp / kClasses, cls = warp % kClasses;
    float2(*s_ml)[8] = reinterpret_cast<float2(*)[8]>(smem_raw + L::kMl) + group * kClasses;
    float(*s_o)[8][L::HDP] = reinterpret_cast<float(*)[8][L::HDP]>(smem_raw + L::kO) + group * kClasses;
    // this lane's row of the four 8 x 8 tiles of V^T: key (lane & 7) + 8 (lane / 16), dims 8 ((lane / 8) & 1) on
    const int vkey = (lane & 7) + 8 * (lane >> 4), vch = (lane >> 3) & 1;
    const int half = box_keys * 128;                       // bytes of a box's 64 dims
    const int cls_at = cls * kStep / box_keys * (box_keys * HD * 2) + cls * kStep % box_keys * 128;
    const int kbase = cls_at + g8 * 128;
    const uint32_t vbase = static_cast<uint32_t>(L::kHalf + cls_at + vkey * 128);
    while (true) {
        bool ok = wait(&bars.item_full[slot], slot_phase);
        const StagedItem& it = bars.item[slot];            // read again at the end: registers are short
        const int nsteps = ok ? it.nsteps : 0, tmax = it.tmax, key_lo = it.split * kSplit;
        if (ok && nsteps == 0) return;                     // the same in every warp
        const int2 pos2 = *reinterpret_cast<const int2*>(&it.pos[8 * group + 2 * c4]);
        const int pos[2] = {pos2.x, pos2.y};
        const bool any = __any_sync(0xffffffffu, max(pos[0], pos[1]) >= key_lo);     // the tile has rows in this split
        const int see = it.bad ? -1 : all_see(pos, key_lo);
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(smem_raw + L::kQ) + (slot * L::kRows + 8 * group + g8) * L::QP + 16 * c4;
        constexpr bool kHold = T < 4;                      // Q stays in registers where there are enough
        uint4 qh[KS / 2];
#pragma unroll
        for (int k = 0; k < KS / 2; ++k)
            if (kHold) qh[k] = *reinterpret_cast<const uint4*>(q + 64 * (k >> 1) + 8 * (k & 1));
        RowState<HD> rs;
        rs.clear();
        uint32_t bad_rows = 0;                             // bit e: the row met a page id out of range
#pragma unroll 1
        for (int s0 = 0; s0 < nsteps; s0 += kClasses) {
            ok = wait(&bars.full[stage], phase);
            if (!ok) break;
            const int step = s0 + cls, key0 = key_lo + kStep * step;
            if (any && step < nsteps) {
                const uint8_t* base = smem_raw + L::kRing + stage * L::kStage;
                float s2[2][4] = {}, st[4];
#pragma unroll
                for (int k = 0; k < KS / 2; ++k) {
                    const uint4 qv = kHold ? qh[k] : *reinterpret_cast<const uint4*>(q + 64 * (k >> 1) + 8 * (k & 1));
                    // 16 bytes of keys g8 and g8 + 8: the dims that the direct kernel puts into two k-steps
                    const uint8_t* at = base + kbase + (k >> 1) * half + ((2 * c4 + (k & 1)) ^ g8) * 16;
                    const uint4 k0 = *reinterpret_cast<const uint4*>(at), k1 = *reinterpret_cast<const uint4*>(at + 8 * 128);
                    mma_16816(s2[0], k0.x, k1.x, k0.y, k1.y, qv.x, qv.y);
                    mma_16816(s2[1], k0.z, k1.z, k0.w, k1.w, qv.z, qv.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) st[e] = s2[0][e] + s2[1][e];
                if (key0 + kStep - 1 > see) {
                    int live_keys = tmax - key0 + 1;
                    if ((it.bad >> step) & 1u) {               // the rows that reach the step cannot be computed
                        bad_rows |= (pos[0] >= key0 ? 1u : 0u) | (pos[1] >= key0 ? 2u : 0u);
                        live_keys = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) st[e] = 0.0f;
                    }
                    if (live_keys < kStep) {
                        // values behind the last key may be anything; every group that reads them writes these zeros first
                        const uint32_t v0 = smem_u32(base) + static_cast<uint32_t>(L::kHalf + cls_at);
                        for (int h = 0; h < HD / 64; ++h)
                            for (int e = live_keys * 8 + lane; e < kStep * 8; e += 32)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + static_cast<uint32_t>(h * half + e * 16)), "r"(0)
                                             : "memory");
                        fence_proxy_async_smem();              // before the next box in this place
                        __syncwarp();
                    }
                    mask_step(st, pos, key0, g8);
                }
                uint32_t hi[2], low[2];
                rs.step(st, P.scale_log2, hi, low);
                const uint32_t vat = smem_u32(base) + vbase;
                rs.add(hi, low, [&](int k, uint32_t (&a)[4]) {
                    ldmatrix_x4_trans(vat + static_cast<uint32_t>((k >> 2) * half + (((2 * k + vch) & 7) ^ (vkey & 7)) * 16), a);
                });
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.empty[stage]);
            next_stage();
        }
        if (!group_all(group, ok)) return;                 // a wait ran out: all four warps leave (else the last join has been read)
        rs.put_ml(s_ml[cls], bad_rows, g8, c4);
        // acc[k][e], acc[k][e + 2] are dims 16 k + g8 and + 8 of row 2 c4 + e
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            float* o = &s_o[cls][2 * c4][16 * k + g8];
            o[0] = rs.acc[k][0];
            o[L::HDP] = rs.acc[k][1];
            o[8] = rs.acc[k][2];
            o[L::HDP + 8] = rs.acc[k][3];
        }
        group_bar(group);
        const int t = threadIdx.x & (kDirectThreads - 1), split = it.split;
#pragma unroll
        for (int x4 = t; x4 < 8 * (HD / 4); x4 += kDirectThreads) {
            const int row = x4 / (HD / 4), d = (x4 % (HD / 4)) * 4, row_pos = it.pos[8 * group + row];
            if (row_pos >= key_lo) join_row<HD>(P, s_o, s_ml, row, d, row_pos, it.pair[8 * group + row], split);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.item_empty[slot]);            // neither the item nor Q is needed any more
        next_slot();
    }
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

// A pool of pages [n_pages][Hkv][page_size][HD] seen in boxes of a page's keys, up to a round's.
template <int HD>
bool encode_pages(CUtensorMap* map, const __nv_bfloat16* pool, const PagedAttnParams& P) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t row = HD * 2, page = row * static_cast<cuuint64_t>(P.pt.page_size);
    const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(P.pt.page_size), HD / 64, static_cast<cuuint64_t>(P.Hkv),
                                static_cast<cuuint64_t>(P.pt.n_pages)};
    const cuuint64_t strides[4] = {row, 128, page, page * static_cast<cuuint64_t>(P.Hkv)};
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(std::min(P.pt.page_size, kRoundKeys)), HD / 64, 1, 1}, estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<__nv_bfloat16*>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int T>
int launch_staged(const PagedAttnParams& P, long long passes, cudaStream_t s) {
    using L = StagedLayout<HD, T>;
    static DeviceOnce once;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    const int st = once.run(dev, [] {
        return cuda_status(cudaFuncSetAttribute(paged_attn_staged_kernel<HD, T>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes));
    });
    if (st != BIV_OK) return st;
    CUtensorMap tk, tv;
    if (!encode_pages<HD>(&tk, P.kp, P) || !encode_pages<HD>(&tv, P.vp, P)) {
        set_cuda_error(cudaErrorNotSupported);
        return BIV_ERR_CUDA;
    }
    const long long n_groups = (P.W + P.rpg - 1) / P.rpg;
    const long long grid = std::min<long long>(n_groups * P.Hkv * P.s_max * passes, num_sms());
    return launch_pdl(paged_attn_staged_kernel<HD, T>, dim3(static_cast<unsigned>(grid)), dim3(T * 128 + 64), L::kBytes, s, tk, tv, P);
}

// The split kernel and, where a row may have several splits, the combine kernel.
template <int HD>
int launch_paged_attn(const PagedAttnParams& P, cudaStream_t s) {
    const long long rows = static_cast<long long>(P.rpg) * P.G;
    // Few tiles (of 8 query rows of a request and KV head) and short tables: one launch, with
    // as many CTAs a tile as one round of them holds.  A CTA takes its splits one after the
    // other, some 3 to 5 us each, so two at most.  The host knows the tables' width, not the
    // lengths, so a wide table sends short requests through two kernels.  32 and 8 heads, us, with
    // two kernels in brackets: a window of 5 rows, 700 keys, 1 request 6.7 (10.3).  C = 4, under
    // tables of 2048: 5 single tokens of 700 keys 6.7 (9.0), 1024: 8.7 (10.7), 1500: 12.7 (11.6), 2000: 13.0
    // (12.6); 9 of them 8.9 (11.6), 11.1 (12.7), 14.5 (14.4), 15.9 (20.6); 3 windows of 5 rows, 700 keys 7.8
    // (11.1), 1024: 9.3 (11.2), 2000: 13.3 (15.9).  So it may lose a tenth near the middle of its two
    // turns and gains a quarter below and above.  In several rounds (2 windows, C = 8): 12.7 (10.5).
    const long long tiles = (P.W + P.rpg - 1LL) / P.rpg * P.Hkv * ((rows + 7) / 8), slots = 2LL * num_sms();
    if (P.s_max <= kSmallTurns * 8 && tiles * 8 <= slots)
        return launch_cluster_pdl(paged_attn_small_kernel<HD, 8>, dim3(static_cast<unsigned>(tiles * 8)), dim3(kDirectThreads), 0, s, 8, P);
    if (P.s_max <= kSmallTurns * 4 && tiles * 4 <= slots)
        return launch_cluster_pdl(paged_attn_small_kernel<HD, 4>, dim3(static_cast<unsigned>(tiles * 4)), dim3(kDirectThreads), 0, s, 4, P);
    int st;
    if (rows <= 8) {
        static DeviceOnce once;
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_status(e);
        st = once.run(dev, [] {
            return cuda_status(cudaFuncSetAttribute(paged_attn_direct_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    static_cast<int>(sizeof(DirectSmem<HD>))));
        });
        if (st != BIV_OK) return st;
        const long long n_groups = (P.W + P.rpg - 1) / P.rpg;
        const long long grid = std::min<long long>(n_groups * P.Hkv * P.s_max, 3LL * num_sms());
        st = launch_pdl(paged_attn_direct_kernel<HD>, dim3(static_cast<unsigned>(grid)), dim3(kDirectThreads),
                        sizeof(DirectSmem<HD>), s, P);
    } else {
        // as few passes over the keys as four tiles allow, each with as few tiles as they then need
        const long long passes = (rows + 31) / 32;
        const long long T = (rows + 8 * passes - 1) / (8 * passes);
        st = T == 2 ? launch_staged<HD, 2>(P, passes, s) : T == 3 ? launch_staged<HD, 3>(P, passes, s) : launch_staged<HD, 4>(P, passes, s);
    }
    if (st != BIV_OK || P.s_max == 1) return st;
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
    const RopeTurns& turns = rope_turns(theta, hd);
    // few rows: one per CTA, so that all SMs work; many: two (4095 rows of 48 heads:
    // 22.0 us with one, 19.7 with two, 20.7 with four, 22.3 with eight)
    const int rows = W <= 4 * num_sms() ? 1 : 2;
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
    if (!aligned16(q) || !aligned16(o) || !aligned16(workspace)) return BIV_ERR_ALIGN;
    if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 31u) != 0) return BIV_ERR_ALIGN;   // ld_row
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return hd == 128 ? launch_paged_attn<128>(P, s) : launch_paged_attn<64>(P, s);
}
