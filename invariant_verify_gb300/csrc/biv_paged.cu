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

// One warp per (row, head, split): the keys of the split one after the other,
// each lane holding hd / 32 dims, with the running maximum and sum of the
// softmax.
template <int HD>
__global__ void __launch_bounds__(32) paged_attn_kernel(const PagedAttnParams P) {
    constexpr int E = HD / 32;
    const int lane = threadIdx.x;
    const int split = blockIdx.x, h = blockIdx.y, w = blockIdx.z;
    pdl_wait();
    pdl_trigger();
    const int pos = usable_pos(P, w, split == 0 && h == 0 && lane == 0);
    const long long pair = static_cast<long long>(w) * P.Hq + h;
    if (pos < 0) {
        if (split == 0)
            for (int e = 0; e < E; ++e) P.o[pair * HD + lane * E + e] = __float2bfloat16_rn(0.0f);
        return;
    }
    if (split * kSplit > pos) return;
    const int kvh = h / P.G;
    const int32_t* table = P.pt.table + static_cast<long long>(P.row_slot[w]) * P.pt.max_pages;
    float q[E], acc[E], m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(P.q[pair * HD + lane * E + e]);
        acc[e] = 0.0f;
    }
    const int last = min(pos, split * kSplit + kSplit - 1);
    for (int j = split * kSplit; j <= last; ++j) {
        const int page = table[j >> P.pt.page_shift];
        if (page < 0 || page >= P.pt.n_pages) {
            bad = true;
            break;
        }
        const long long at = ((static_cast<long long>(page) * P.Hkv + kvh) * P.pt.page_size + (j & (P.pt.page_size - 1))) * HD + lane * E;
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(P.kp[at + e]), s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= P.scale_log2;
        const float mn = fmaxf(m, s);
        const float f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = fmaf(l, f, p);
        for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, p * __bfloat162float(P.vp[at + e]));
    }
    if (bad && lane == 0) atomicOr(&g_paged_err, BIV_DEVERR_INDEX);
    const long long part = pair * P.s_max + split;
    for (int e = 0; e < E; ++e) P.ws_o[part * HD + lane * E + e] = acc[e];
    if (lane == 0) P.ws_ml[part] = make_float2(m, bad ? -1.0f : l);
}

// One warp per (row, head): the splits in increasing order.
template <int HD>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedAttnParams P) {
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31;
    const long long pair = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (pair >= static_cast<long long>(P.W) * P.Hq) return;
    const int pos = usable_pos(P, static_cast<int>(pair / P.Hq), false);
    if (pos < 0) return;
    const int ns = pos / kSplit + 1;
    float m = -INFINITY, l = 0.0f, acc[E] = {};
    bool bad = false;
    for (int s = 0; s < ns; ++s) m = fmaxf(m, P.ws_ml[pair * P.s_max + s].x);
    for (int s = 0; s < ns; ++s) {
        const float2 ml = P.ws_ml[pair * P.s_max + s];
        bad |= ml.y == -1.0f;
        const float f = exp2f(ml.x - m);
        l = fmaf(ml.y, f, l);
        for (int e = 0; e < E; ++e) acc[e] = fmaf(P.ws_o[(pair * P.s_max + s) * HD + lane * E + e], f, acc[e]);
    }
    for (int e = 0; e < E; ++e)
        P.o[pair * HD + lane * E + e] = __float2bfloat16_rn(bad ? 0.0f : acc[e] / l);
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

template <int HD>
int launch_paged_attn(PagedAttnParams& P, cudaStream_t s) {
    int st = launch_pdl(paged_attn_kernel<HD>, dim3(P.s_max, P.Hq, P.W), dim3(32), 0, s, P);
    if (st != BIV_OK) return st;
    const long long pairs = static_cast<long long>(P.W) * P.Hq;
    return launch_pdl(paged_combine_kernel<HD>, dim3(static_cast<unsigned>((pairs + 7) / 8)), dim3(256), 0, s, P);
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
