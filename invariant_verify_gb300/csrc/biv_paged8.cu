// The paged key-value cache held in 8 bits: rotation and write of new rows, and
// fixed-split decode attention over them.
//
// A block of 16 positions is held in e4m3 with one scale for each KV head, and goes
// into the pages when its last position is written.  Until then, and for as long as a
// rejected draft may take a request back, its rows lie in bf16 in a ring of `tail`
// positions a slot (position p at p % tail).  A row at position p reads positions
// below 16 floor(p / 16) in e4m3 and the rest of its own block in bf16: which form a
// key has goes by the row's position alone, so a row has the same bits in every
// window, and a block is always quantised once, from bf16, whole.
#include "biv_e4m3.cuh"
#define BIV_PAGED_SPLIT 512
#define BIV_PAGED_ROWS 512                             // so that three CTAs of 73 KB share an SM
#include "biv_paged.cuh"

namespace biv {
namespace {

constexpr int kHeldBlock = 16;                         // also the keys of an attention step

// Pools of held blocks, their scales [n_pages][Hkv][page_size / 16] and the rings
// [n_slots][Hkv][tail][hd].
struct HeldPools {
    uint8_t* k;
    uint8_t* v;
    __nv_bfloat16* k_scales;
    __nv_bfloat16* v_scales;
    __nv_bfloat16* k_tail;
    __nv_bfloat16* v_tail;
    int tail;
};

// --------------------------------------------------- RoPE + write
constexpr int kWriteThreads = 256;
constexpr int kWriteBatch = 3;

// One CTA per block of 16 positions that a group's rows touch and KV head: it rotates
// the block's rows of the G query heads and the key head, puts keys and values into the
// ring and, where the block's last position is among the rows, the whole block into its
// page: rows of earlier calls come from the ring, so that no CTA waits for another.
// Bound by its chain of dependent steps (position, rows, rotation, largest, page), which too few
// CTAs an SM hide: 2047 rows of 32 and 8 heads 15.4 us (3.5 TB/s read and written), 8 rows
// 3.9 us with the launch.  128 threads, with the rows asked for after the sines: 20.1; more CTAs an
// SM by fewer registers: 17.3 (five), 20.3 (six).
template <int HD>
__global__ void __launch_bounds__(kWriteThreads)
rope_kv_write_held_kernel(const __nv_bfloat16* __restrict__ qkv, __nv_bfloat16* __restrict__ q_out, const HeldPools hp,
                          const PageTable pt, const int32_t* __restrict__ row_slot, const int32_t* __restrict__ row_pos,
                          const int32_t* __restrict__ rows_keep, int groups, int K, int Hq, int Hkv, int chunks,
                          const __grid_constant__ RopeTurns turns) {
    constexpr int kHalf = HD / 2, kPerHead = kHalf / 8;
    __shared__ __align__(16) float s_cs[kHeldBlock][HD];             // cosines, then sines
    __shared__ __align__(16) __nv_bfloat16 s_kv[2][kHeldBlock][HD];
    __shared__ int s_pos[kHeldBlock];
    __shared__ bool s_ok[kHeldBlock];
    __shared__ int s_page;                                           // of the block if it is full, else -1
    __shared__ float s_max[kWriteThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int h = blockIdx.x % Hkv, rc = blockIdx.x / Hkv, c = rc % chunks, r = rc / chunks;
    const int G = Hq / Hkv, heads = Hq + 2 * Hkv;
    const long long w00 = static_cast<long long>(r) * K;
    pdl_wait();
    pdl_trigger();
    const int p0 = row_pos[w00], slot = row_slot[w00];
    const int before = c == 0 && p0 >= 0 ? p0 & (kHeldBlock - 1) : 0;               // the block's rows of earlier calls
    const int j0 = kHeldBlock * c - (p0 >= 0 ? p0 & (kHeldBlock - 1) : 0);          // row of the block's first position
    if (j0 >= K) return;
    const int i0 = max(0, -j0), i1 = min(kHeldBlock, K - j0);                       // the block's rows of this call
    // A slot that two groups write: neither sees the other's rows when it fills a block.
    const uint32_t cap = static_cast<uint32_t>(pt.max_pages) << pt.page_shift;      // below 2^31
    if (h == 0 && c == 0) {
        auto writes = [&](long long g) { return static_cast<uint32_t>(row_pos[g * K]) < cap && (!rows_keep || rows_keep[g] > 0); };
        bool twice = false;
        for (int g = tid; g < groups; g += kWriteThreads) twice |= g != r && row_slot[static_cast<long long>(g) * K] == slot && writes(g) && writes(r);
        if (twice && slot >= 0 && slot < pt.n_slots) atomicOr(&g_paged_err, BIV_DEVERR_GROUP);
    }
    const int first = (p0 & ~(kHeldBlock - 1)) + kHeldBlock * c;                    // the block's first position
    if (tid < 32) {
        bool ok = false;
        if (lane >= i0 && lane < i1) {
            const int j = j0 + lane;
            const long long w = w00 + j;
            const int pos = row_pos[w];
            if (pos != -1 && (!rows_keep || j < rows_keep[r])) {
                unsigned int bits = 0;
                if (static_cast<uint32_t>(pos) >= cap || slot < 0 || slot >= pt.n_slots) bits = BIV_DEVERR_INDEX;
                else if (p0 < 0 || row_slot[w] != slot || pos - j != p0 || (j > 0 && row_pos[w - 1] != pos - 1)) bits = BIV_DEVERR_GROUP;
                if (bits) atomicOr(&g_paged_err, bits);
                ok = bits == 0;
            }
            s_pos[lane] = pos;
            s_ok[lane] = ok;
        }
        const uint32_t all = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) {
            const uint32_t want = (1u << kHeldBlock) - (1u << i0);
            int page = -1;
            if ((all & want) == want && i1 == kHeldBlock) {
                page = pt.table[static_cast<long long>(slot) * pt.max_pages + (first >> pt.page_shift)];
                if (page < 0 || page >= pt.n_pages) {
                    atomicOr(&g_paged_err, BIV_DEVERR_INDEX);
                    page = -1;
                }
            }
            s_page = page;
        }
    }
    // a thread's next kWriteBatch pieces (eight pairs each): the first ones' loads run under the sines
    const int items = (G + 2) * kPerHead, n_items = (i1 - i0) * items;
    uint4 a[kWriteBatch], b[kWriteBatch];
    int row[kWriteBatch], piece[kWriteBatch];
    auto load = [&](int it0) {
#pragma unroll
        for (int n = 0; n < kWriteBatch; ++n) {
            const int it = it0 + n * kWriteThreads;
            row[n] = -1;
            if (it < n_items) {
                row[n] = i0 + it / items;
                piece[n] = it % items;
                const int x = piece[n] / kPerHead, d = (piece[n] % kPerHead) * 8;
                const int head = x < G ? h * G + x : x == G ? Hq + h : Hq + Hkv + h;
                const __nv_bfloat16* src = qkv + ((w00 + j0 + row[n]) * heads + head) * HD + d;
                a[n] = __ldg(reinterpret_cast<const uint4*>(src));
                b[n] = __ldg(reinterpret_cast<const uint4*>(src + kHalf));
            }
        }
    };
    load(tid);
    for (int e = tid; e < (i1 - i0) * kHalf; e += kWriteThreads) {
        const int i = i0 + e / kHalf, d = e % kHalf;
        const uint64_t phase = static_cast<uint64_t>(static_cast<long long>(row_pos[w00 + j0 + i])) * turns.per_pos[d];
        // the top 32 bits as a signed fraction of half a turn
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &sn, &cs);
        s_cs[i][d] = cs;
        s_cs[i][kHalf + d] = sn;
    }
    __syncthreads();
    const long long ring = (static_cast<long long>(slot) * Hkv + h) * hp.tail;
    for (int it0 = tid; it0 < n_items;) {
#pragma unroll
        for (int n = 0; n < kWriteBatch; ++n) {
            if (row[n] < 0) continue;
            const int i = row[n], x = piece[n] / kPerHead, d = (piece[n] % kPerHead) * 8;
            if (x <= G) {
                uint32_t* a4 = &a[n].x;
                uint32_t* b4 = &b[n].x;
                const float* cs = &s_cs[i][d];
                const float* sn = cs + kHalf;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float al = bf16lo(a4[e]), ah = bf16hi(a4[e]), bl = bf16lo(b4[e]), bh = bf16hi(b4[e]);
                    const float cl = cs[2 * e], ch = cs[2 * e + 1], sl = sn[2 * e], sh = sn[2 * e + 1];
                    a4[e] = pack_bf16x2(al * cl - bl * sl, ah * ch - bh * sh);
                    b4[e] = pack_bf16x2(bl * cl + al * sl, bh * ch + ah * sh);
                }
            }
            __nv_bfloat16* dst = x < G ? q_out + ((w00 + j0 + i) * Hq + h * G + x) * HD
                                       : (x == G ? hp.k_tail : hp.v_tail) + (ring + s_pos[i] % hp.tail) * HD;
            if (x >= G) {
                __nv_bfloat16* held = s_kv[x - G][i];
                *reinterpret_cast<uint4*>(held + d) = a[n];
                *reinterpret_cast<uint4*>(held + kHalf + d) = b[n];
                if (!s_ok[i]) continue;
            }
            *reinterpret_cast<uint4*>(dst + d) = a[n];
            *reinterpret_cast<uint4*>(dst + kHalf + d) = b[n];
        }
        it0 += kWriteBatch * kWriteThreads;
        load(it0);
    }
    const int page = s_page;
    if (page < 0) return;
    for (int e = tid; e < 2 * before * (HD / 8); e += kWriteThreads) {
        const int x = e & 1, i = (e >> 1) / (HD / 8), d = (e >> 1) % (HD / 8) * 8;
        *reinterpret_cast<uint4*>(&s_kv[x][i][d]) =
            *reinterpret_cast<const uint4*>((x ? hp.v_tail : hp.k_tail) + (ring + (first + i) % hp.tail) * HD + d);
    }
    __syncthreads();
    // half of the warps for the keys, half for the values
    constexpr int kSide = kWriteThreads / 2, kLoads = kHeldBlock * HD / 8 / kSide;
    const int x = tid / kSide, t = tid % kSide;
    uint4 y[kLoads];
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
        y[e] = reinterpret_cast<const uint4*>(&s_kv[x][0][0])[t + kSide * e];
        m = fmaxf(m, max_of_halves(max_abs8(y[e])));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) s_max[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kSide / 32; ++n) m = fmaxf(m, s_max[kSide / 32 * x + n]);
    // the next bf16 number: what the scale is rounded by costs range (at most 2^-7 of it), no precision,
    // since the values are divided by the number that is held
    const uint32_t bits = (__float_as_uint(scale_of(m)) + 0xffffu) & 0xffff0000u;
    const float scale = __uint_as_float(bits), inv = __frcp_rn(scale);
    const long long at = static_cast<long long>(page) * Hkv + h;
    const int in_page = first & (pt.page_size - 1);
    uint8_t* dst = (x ? hp.v : hp.k) + (at * pt.page_size + in_page) * HD;
#pragma unroll
    for (int e = 0; e < kLoads; ++e) reinterpret_cast<uint2*>(dst)[t + kSide * e] = e4m3x8(y[e], scale, inv);
    if (t == 0)
        reinterpret_cast<uint16_t*>(x ? hp.v_scales : hp.k_scales)[(at * pt.page_size + in_page) / kHeldBlock] = static_cast<uint16_t>(bits >> 16);
}

// ------------------------------------------------------------ attention
// The split kernels of biv_paged.cu with other keys.  Held keys and values become fp16 in
// registers, which holds every e4m3 number, and meet fp16 queries and weights in
// mma.m16n8k16; a step of 16 keys is one block, so the key scale multiplies the step's
// scores and the value scale its share of the output, both in fp32.  A query row is
// multiplied by a power of two first, so that its largest element lies in [2^14, 2^15):
// nothing above 2^-28 of that is rounded.  A weight is at most 2^15 and rounded to 11
// bits, an eighth of the output's own rounding, and a row's sum adds the rounded weights.
// The rest of a row's own block comes from the ring, in bf16, with weights of 16 bits.
//
// One CTA per item; the split's steps are taken by four warps in turn, whose keys and values
// are copied to shared memory three steps ahead, over the items' ends; an item's pages, scales
// and queries are asked for during the item before.  Up to T tiles of 8 query rows share
// one read.  What bounds it is the instructions of a step (395 with their share of the item's,
// 64 of them conversions) at 12 warps an SM, not bytes: 512 keys a split instead of 256
// halve the items' share, at the cost of a call that is one short row (which the clusters below
// pay back).  Measured with (256, 512) keys a split: one row of 131071 keys 64.5, 54.5 us (4.9 TB/s;
// 67.4, 61.7 before the copies, when the keys went straight to registers), 64 rows of some 1400 keys
// 47.8, 41.8 us, 32 windows of five 68.8, 57.4 us, one row of 700 8.0, 9.9 us.  Two steps at once
// (more independent work a warp, fewer warps) took 20 % longer.

// D[16 x 8] (+)= A[16 x 16] B[16 x 8], fp16 with fp32 sums.
BIV_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
BIV_DEV void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
BIV_DEV uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
BIV_DEV float f16_lo(uint32_t x) {
    float r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(r) : "r"(x));
    return r;
}
BIV_DEV float f16_hi(uint32_t x) {
    float r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(r) : "r"(x));
    return r;
}

// N words of the ring: the kernel before may have written them.
template <int N>
BIV_DEV void ld_tail(const __nv_bfloat16* p, uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]) : "l"(p + 2 * i));
}

// A warp's keys and values of a step on their way to registers: 16 x hd bytes each, copied to shared memory
// kSlots - 1 steps ahead.  A 16-byte piece lies at its place XORed with its line's number,
// so that the eight lanes that are served at once meet all banks: lane (g8, c4) reads
// dims [hd / 4 c4, ..) of keys g8 and g8 + 8 and dims [hd / 8 g8, ..) of values 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9.
constexpr int kSlots = 3;

template <int HD>
struct __align__(128) HeldSlot {
    static constexpr int KS = HD / 16;
    static constexpr int kBytes = kHeldBlock * HD;
    uint8_t k[kBytes], v[kBytes];

    // Where piece c (16 bytes) of a key lies.
    static BIV_DEV int at(int key, int c) {
        if constexpr (HD == 128) return key * 128 + ((c ^ (key & 7)) << 4);
        const int line = key >> 1;
        return line * 128 + ((((key & 1) * 4 + c) ^ (2 * (line & 3))) << 4);
    }
    // Where a lane's first piece of a step goes (pieces lane, lane + 32, ... of the keys and of the values are its own).
    static BIV_DEV int first(int lane) { return at(lane / (HD / 16), lane % (HD / 16)); }
    BIV_DEV void copy(const uint8_t* kp, const uint8_t* vp, int first, uint64_t policy) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < kBytes / 512; ++e) {
                // four lines further: bit 2 of a line's number is bit 6 of the place (hd = 64: the pattern repeats)
                const uint32_t to = smem_u32(x ? v : k) + (HD == 128 && (e & 1) ? first ^ 64 : first) + 512 * e;
                asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(to), "l"((x ? vp : kp) + 512 * e), "l"(policy) : "memory");
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Keys g8 + 8 r of k-steps 4 u .. 4 u + 3.
    BIV_DEV void load_k(uint32_t (&w)[4], int r, int u, int g8, int c4) const {
        const uint4 x = *reinterpret_cast<const uint4*>(k + at(g8 + 8 * r, KS / 4 * c4 + u));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    BIV_DEV void load_v(uint32_t (&w)[HD / 32], int i, int g8, int c4) const {
        const int key = 2 * c4 + (i & 1) + 8 * (i >> 1);
        if constexpr (HD == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(v + at(key, g8));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(v + at(key, g8 >> 1) + (g8 & 1) * 8);
            w[0] = x.x, w[1] = x.y;
        }
    }
};

// Waits for all of this thread's groups of copies but the newest `but`.
BIV_DEV void wait_copies(int but) {
    if (but >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (but == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Q of T tiles in the order of the B fragments: [tile][k / 2][lane] holds the lane's two registers of
// k-steps k and k + 1, as fp16 (times the row's power of two) and as bf16.
template <int HD, int T>
struct __align__(16) HeldQ {
    uint4 f16[T][HD / 32][32];
    uint4 bf[T][HD / 32][32];
    float back[T][8];                  // log2(e) / sqrt(hd) over the row's power of two
};

// A warp's running softmax over T tiles of eight query rows: this lane's columns are rows
// 2 (lane % 4) and the next of a tile.
template <int HD, int T>
struct HeldRows {
    static constexpr int KS = HD / 16;
    static constexpr float kSlack = 8.0f;          // as in RowState: a row's reference follows its maximum with slack
    static constexpr float kLift = 7.0f;           // weights are 2^kLift times as large: up to 2^15, so that fp16 keeps small ones
    float acc[T][KS][4];
    float m[T][2], l[T][2], mu[T][2];

    BIV_DEV void clear() {
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][k][e] = 0.0f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = mu[t][0] = mu[t][1] = 0.0f;
        }
    }

    // Whether this lane's scores of a step ask for another reference.
    BIV_DEV bool above(int t, const float (&st)[4]) const {
        return fmaxf(st[0], st[2]) > m[t][0] + kSlack || fmaxf(st[1], st[3]) > m[t][1] + kSlack;
    }
    // The references of the rows whose scores pass theirs by more than the slack.
    BIV_DEV void refer(int t, const float (&st)[4]) {
        float x[2] = {fmaxf(st[0], st[2]), fmaxf(st[1], st[3])};
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
            if (x[e] > m[t][e] + kSlack) {
                f[e] = ex2_approx(m[t][e] - x[e]);
                m[t][e] = x[e];
                mu[t][e] = x[e] - kLift;
            }
            l[t][e] *= f[e];
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][k][e] *= f[e & 1];
    }
    // Scores of a step in units of log 2 to weights in place (without their sum).
    BIV_DEV void weights(int t, float (&st)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) st[e] = ex2_approx(st[e] - mu[t][e & 1]);
    }

    // One held step: scores, weights and values; key0 its first key, last[t] the lane's rows' last held key.
    BIV_DEV void step(const HeldSlot<HD>& slot, const HeldQ<HD, T>& q, const float (&back)[T][2], float k_scale, float v_scale,
                      const int (&last)[T][2], int see, bool bad, int key0, int lane) {
        const int g8 = lane >> 2, c4 = lane & 3;
        float st[T][4];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) st[t][e] = 0.0f;
#pragma unroll
        for (int u = 0; u < KS / 4; ++u) {
            uint32_t hk[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) slot.load_k(hk[r], r, u, g8, c4);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                uint32_t a[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    a[j][0] = e4m3_lo(hk[0][k + j]);
                    a[j][1] = e4m3_lo(hk[1][k + j]);
                    a[j][2] = e4m3_hi(hk[0][k + j]);
                    a[j][3] = e4m3_hi(hk[1][k + j]);
                }
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const uint4 b = q.f16[t][2 * u + k / 2][lane];
                    mma_f16(st[t], a[0][0], a[0][1], a[0][2], a[0][3], b.x, b.y);
                    mma_f16(st[t], a[1][0], a[1][1], a[1][2], a[1][3], b.z, b.w);
                }
            }
        }
        uint32_t hv[4][HD / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) slot.load_v(hv[i], i, g8, c4);
        uint32_t w[T][2];
        bool up = false;
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) st[t][e] *= back[t][e & 1] * k_scale;
            if (key0 + kStep - 1 > see) mask_step(st[t], last[t], key0, g8);
            up |= above(t, st[t]);
        }
        if (__any_sync(0xffffffffu, up)) {         // one vote for all tiles: a row that need not move keeps its bits
#pragma unroll
            for (int t = 0; t < T; ++t) refer(t, st[t]);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            weights(t, st[t]);
            const uint32_t h0 = pack_f16x2(st[t][0], st[t][1]), h1 = pack_f16x2(st[t][2], st[t][3]);
            l[t][0] += f16_lo(h0) + f16_lo(h1);
            l[t][1] += f16_hi(h0) + f16_hi(h1);
            w[t][0] = transpose8(h0);
            w[t][1] = transpose8(h1);
        }
        if (bad) {                                 // a page out of range: what was read in its place may be NaN
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < HD / 32; ++d) hv[i][d] = 0u;
        }
#pragma unroll
        for (int d = 0; d < HD / 32; ++d) {
            uint32_t p[2][2];                      // [keys, keys + 8][dims 0 and 1, 2 and 3]: pairs of keys
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                p[i][0] = __byte_perm(hv[2 * i][d], hv[2 * i + 1][d], 0x5140);
                p[i][1] = __byte_perm(hv[2 * i][d], hv[2 * i + 1][d], 0x7362);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a0 = e4m3_lo(p[0][j]), a1 = e4m3_hi(p[0][j]), a2 = e4m3_lo(p[1][j]), a3 = e4m3_hi(p[1][j]);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    float y[4];
                    mma_f16_zero(y, a0, a1, a2, a3, w[t][0], w[t][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][2 * d + j][e] = fmaf(v_scale, y[e], acc[t][2 * d + j][e]);
                }
            }
        }
    }

    // The step whose block is a row's own, from the ring: pos[t] are the rows' positions; rows of other
    // blocks are left alone; what lies behind key tmax may be anything.
    BIV_DEV void own_step(const __nv_bfloat16* kt, const __nv_bfloat16* vt, const HeldQ<HD, T>& q, float scale_log2,
                          const int (&pos)[T][2], int tmax, int key0, int lane) {
        const int g8 = lane >> 2, c4 = lane & 3;
        uint32_t k[2][2 * KS];
#pragma unroll
        for (int r = 0; r < 2; ++r) ld_tail(kt + (g8 + 8 * r) * HD + HD / 4 * c4, k[r]);
        uint32_t v[4][KS];
        auto load_v = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) ld_tail(vt + (2 * c4 + (i & 1) + 8 * (i >> 1)) * HD + HD / 8 * g8, v[i]);
        };
        if constexpr (T <= 2) load_v();            // the registers allow it
        float s4[T][4];
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s4[t][e] = 0.0f;
#pragma unroll
            for (int j = 0; j < KS; j += 2) {
                const uint4 b = q.bf[t][j / 2][lane];
                mma_16816(s4[t], k[0][2 * j], k[1][2 * j], k[0][2 * j + 1], k[1][2 * j + 1], b.x, b.y);
                mma_16816(s4[t], k[0][2 * j + 2], k[1][2 * j + 2], k[0][2 * j + 3], k[1][2 * j + 3], b.z, b.w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = pos[t][e & 1];
                s4[t][e] = (p | (kStep - 1)) == (key0 | (kStep - 1)) && key0 + g8 + 8 * (e >> 1) <= p ? s4[t][e] * scale_log2 : -INFINITY;
            }
        }
        if constexpr (T > 2) load_v();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (key0 + 2 * c4 + (i & 1) + 8 * (i >> 1) > tmax) {
#pragma unroll
                for (int d = 0; d < KS; ++d) v[i][d] = 0u;
            }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float(&st)[4] = s4[t];
            if (__any_sync(0xffffffffu, above(t, st))) refer(t, st);
            weights(t, st);
            l[t][0] += st[0] + st[2];
            l[t][1] += st[1] + st[3];
            const uint32_t h0 = pack_bf16x2(st[0], st[1]), h1 = pack_bf16x2(st[2], st[3]);
            const uint32_t hi[2] = {transpose8(h0), transpose8(h1)};
            const uint32_t low[2] = {transpose8(pack_bf16x2(st[0] - bf16lo(h0), st[1] - bf16hi(h0))),
                                     transpose8(pack_bf16x2(st[2] - bf16lo(h1), st[3] - bf16hi(h1)))};
#pragma unroll
            for (int d = 0; d < KS; ++d) {
                const uint32_t a0 = __byte_perm(v[0][d], v[1][d], 0x5410), a1 = __byte_perm(v[0][d], v[1][d], 0x7632);
                const uint32_t a2 = __byte_perm(v[2][d], v[3][d], 0x5410), a3 = __byte_perm(v[2][d], v[3][d], 0x7632);
                mma_16816(acc[t][d], a0, a1, a2, a3, hi[0], hi[1]);
                mma_16816(acc[t][d], a0, a1, a2, a3, low[0], low[1]);
            }
        }
    }

    // As RowState::put_ml and DirectKeys::put: maximum, sum and output of tile t's rows 2 c4 + e; bad: those that
    // met a page id out of range.
    BIV_DEV void put(int t, int e, float2 (*ml)[4], float (*o)[4][HD + 4], int cls, uint32_t bad, int rows, int lane) const {
        const int g8 = lane >> 2, c4 = lane & 3;
        float s = l[t][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (2 * c4 + e >= rows) return;            // nobody's
        if (g8 == 0) ml[cls][c4] = make_float2(m[t][e], (bad >> e) & 1u ? -INFINITY : s);
#pragma unroll
        for (int k = 0; k < KS; k += 2)
            *reinterpret_cast<float4*>(&o[cls][c4][HD / 8 * g8 + 2 * k]) =
                make_float4(acc[t][k][e], acc[t][k][e + 2], acc[t][k + 1][e], acc[t][k + 1][e + 2]);
    }
};

// A 16-byte piece of a query row: as it is, and times the row's power of two.  The HD / 8
// threads of a row stand side by side in a warp.
template <int HD, int T>
BIV_DEV void put_q(HeldQ<HD, T>& q, const uint4& x, int row, int piece, float scale_log2) {
    uint32_t m = max_abs8(x);
    m = __float_as_uint(max_of_halves(m));
#pragma unroll
    for (int d = HD / 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    // exponent field e: 2^(141 - e) takes the largest to [2^14, 2^15)
    const uint32_t e = min(max(m >> 23, 15u), 254u);
    const float up = __uint_as_float((268u - e) << 23), down = __uint_as_float((e - 14u) << 23);
    const int d0 = piece * 8, c4 = d0 / (HD / 4), kk = d0 % (HD / 4) / 8;
    uint4 y;
    y.x = pack_f16x2(bf16lo(x.x) * up, bf16hi(x.x) * up);
    y.y = pack_f16x2(bf16lo(x.y) * up, bf16hi(x.y) * up);
    y.z = pack_f16x2(bf16lo(x.z) * up, bf16hi(x.z) * up);
    y.w = pack_f16x2(bf16lo(x.w) * up, bf16hi(x.w) * up);
    q.f16[row / 8][kk][(row % 8) * 4 + c4] = y;
    q.bf[row / 8][kk][(row % 8) * 4 + c4] = x;
    if (piece == 0) q.back[row / 8][row % 8] = scale_log2 * down;
}

template <int HD, int T>
struct __align__(128) HeldSmem {
    HeldSlot<HD> slots[kClasses][kSlots];
    float o[kClasses][4][HD + 4];          // of half a tile; rows padded against bank conflicts
    HeldQ<HD, T> q;
    float2 ml[kClasses][4];
    int pos[2][8 * T];
    LiveTable table;
};

constexpr int kHeldThreads = 32 * kClasses;

// Where the pool's rows of a 16-key step start, in elements.
template <int HD>
BIV_DEV long long held_at(const PagedAttnParams& P, int page, int kvh, int key0) {
    return ((static_cast<long long>(page) * P.Hkv + kvh) * P.pt.page_size + (key0 & (P.pt.page_size - 1))) * HD;
}

// Pages and scales of a class's steps of a split: lane i has its i-th.
struct HeldSteps {
    int n;                             // steps of this class
    int page;
    long long at;                      // of the step in its pool
    uint32_t bad;                      // bit i: the page id of step i is out of range
    float k_scale, v_scale;
};

// The scales of a lane's step at element `at` of the pools.  Those of a page out of range stay 0: page 0's, read in its
// place, may be NaN, which times the zeros of the rows that do not reach the page would be NaN too.
template <int HD>
BIV_DEV void scales_at(const HeldPools& hp, HeldSteps& st, int lane, long long at) {
    if ((st.bad >> lane) & 1u) return;
    st.k_scale = __bfloat162float(hp.k_scales[at / (kStep * HD)]);
    st.v_scale = __bfloat162float(hp.v_scales[at / (kStep * HD)]);
}

// CTAs an SM: three of up to two tiles, two of more (the accumulators' registers: three of
// three tiles spill, 32 windows of five 81 us for 57; two of one tile: 64 rows 48 us for 42).
constexpr int held_ctas(int T) { return T <= 2 ? 3 : 2; }

template <int HD, int T>
__global__ void __launch_bounds__(kHeldThreads, held_ctas(T)) paged_attn_held_kernel(const PagedAttnParams P, const HeldPools hp) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    HeldSmem<HD, T>& sm = *reinterpret_cast<HeldSmem<HD, T>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, cls = tid >> 5;
    const int c4 = lane & 3;
    const Items I(P, sm.table, 8 * T);
    const uint64_t policy = policy_evict_first();
    pdl_wait();
    pdl_trigger();
    I.zero_rows<HD>();

    // An item's pages (asked for an item ahead), then its scales and the copies of its first steps (asked for
    // during the last steps of the item before).
    auto pages_of = [&](const AttnItem& it, HeldSteps& st) {
        const int last = (I.largest_pos(it, it.tile * 8 * T, 8 * T) & ~(kStep - 1)) - 1;      // -1 & ~15 is -16
        const int nsteps = last < 0 ? 0 : Items::steps_to(last, it.split);
        st.n = (nsteps - cls + kClasses - 1) / kClasses;
        st.page = 0;
        if (lane < st.n)
            st.page = P.pt.table[static_cast<long long>(I.slot_of(it.w0)) * P.pt.max_pages +
                                 ((it.split * kSplit + kStep * (cls + kClasses * lane)) >> P.pt.page_shift)];
    };
    auto scales_of = [&](const AttnItem& it, HeldSteps& st) {
        st.bad = bad_pages(P, st.page);
        st.k_scale = st.v_scale = 0.0f;
        if (lane < st.n) {
            st.at = held_at<HD>(P, st.page, it.kvh, it.split * kSplit + kStep * (cls + kClasses * lane));
            scales_at<HD>(hp, st, lane, st.at);
        }
    };
    constexpr int kPieces = 8 * T * (HD / 8), kMine = (kPieces + kHeldThreads - 1) / kHeldThreads;       // 16-byte pieces of a tile's queries
    auto queries_of = [&](const AttnItem& it, uint4 (&x)[kMine], int (&row_pos)[1]) {
        const int r0 = it.tile * 8 * T;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int e = tid + i * kHeldThreads, row = r0 + e / (HD / 8);
            if (e < kPieces) {
                int j, head;
                row_head(P, row < it.rows ? row : 0, j, head);         // rows past the group's read its first row and are never used
                x[i] = *reinterpret_cast<const uint4*>(P.q + (static_cast<long long>(it.w0 + j) * P.Hq + it.kvh * P.G + head) * HD + e % (HD / 8) * 8);
            }
        }
        if (tid < 8 * T) {
            int j, head;
            row_head(P, r0 + tid, j, head);
            row_pos[0] = r0 + tid < it.rows ? I.pos_of(it.w0 + j) : -1;
        }
    };
    auto put_queries = [&](const uint4 (&x)[kMine], const int (&row_pos)[1], int buf) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int e = tid + i * kHeldThreads;
            if (e < kPieces) put_q(sm.q, x[i], e / (HD / 8), e % (HD / 8), P.scale_log2);
        }
        if (tid < 8 * T) sm.pos[buf][tid] = row_pos[0];
    };

    AttnItem cur, nxt;
    if (!I.first(cur)) return;
    HeldSteps steps, next_steps;
    // copies under way lie in slots [tail_slot, tail_slot + flying) mod kSlots, oldest first
    HeldSlot<HD>* const slots = sm.slots[cls];
    const int first = HeldSlot<HD>::first(lane);
    int tail_slot = 0, flying = 0, asked = 0;          // asked: steps of the item whose copies were begun
    auto ask = [&](const HeldSteps& st, int i) {
        const long long at = __shfl_sync(0xffffffffu, st.at, i) + 16 * lane;
        int slot = tail_slot + flying;
        slot -= slot >= kSlots ? kSlots : 0;
        slots[slot].copy(hp.k + at, hp.v + at, first, policy);
        ++flying;
    };
    {
        uint4 x[kMine];
        int row_pos[1];
        pages_of(cur, steps);
        queries_of(cur, x, row_pos);
        scales_of(cur, steps);
        asked = min(steps.n, kSlots);
        for (int i = 0; i < asked; ++i) ask(steps, i);
        put_queries(x, row_pos, 0);
    }
    for (int buf = 0;; buf ^= 1) {
        __syncthreads();                           // the tile's queries and positions are there, the item before has been joined
        const bool more = I.next(cur, nxt);
        uint4 next_q[kMine];
        int next_pos[1];
        if (more) {
            pages_of(nxt, next_steps);
            queries_of(nxt, next_q, next_pos);
        }
        const int key_lo = cur.split * kSplit;
        int pos[T][2], last[T][2], tmax = -1, tmin = 0x7fffffff, all = 0x7fffffff;
        float back[T][2];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                pos[t][e] = sm.pos[buf][8 * t + 2 * c4 + e];
                back[t][e] = sm.q.back[t][2 * c4 + e];
                last[t][e] = pos[t][e] < 0 ? -1 : (pos[t][e] & ~(kStep - 1)) - 1;
                tmax = max(tmax, pos[t][e]);
                if (pos[t][e] >= 0) tmin = min(tmin, pos[t][e]);
                if (pos[t][e] >= key_lo) all = min(all, last[t][e]);
            }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, d));
            tmin = min(tmin, __shfl_xor_sync(0xffffffffu, tmin, d));
            all = min(all, __shfl_xor_sync(0xffffffffu, all, d));
        }
        HeldRows<HD, T> rs;
        rs.clear();
        uint32_t bad_rows[T] = {};
        // the rows' own blocks that are this class's: first the first of them, in the order of steps
        const int own1 = tmax < key_lo ? -1 : min(kSteps - 1, (tmax - key_lo) / kStep);
        int own = max(0, (tmin - key_lo) / kStep);
        own += (cls - own) & (kClasses - 1);
        int next_asked = 0;
        bool looked_up = false;
        // the next step's copies, of this item or of the next
        auto ask_ahead = [&]() {
            if (asked < steps.n) {
                ask(steps, asked++);
            } else if (more) {
                if (!looked_up) scales_of(nxt, next_steps);
                looked_up = true;
                if (next_asked < next_steps.n) ask(next_steps, next_asked++);
            }
        };
#pragma unroll 1
        for (int i = 0; i < steps.n; ++i) {
            const int key0 = key_lo + kStep * (cls + kClasses * i);
            const bool step_bad = (steps.bad >> i) & 1u;
            if (step_bad) {
#pragma unroll
                for (int t = 0; t < T; ++t) bad_rows[t] |= (last[t][0] >= key0 ? 1u : 0u) | (last[t][1] >= key0 ? 2u : 0u);
            }
            wait_copies(flying - 1);
            __syncwarp();                          // the step before has been read, this one's copies of all lanes are there
            if (flying < kSlots) ask_ahead();
            rs.step(slots[tail_slot], sm.q, back, __shfl_sync(0xffffffffu, steps.k_scale, i), __shfl_sync(0xffffffffu, steps.v_scale, i), last, all, step_bad, key0, lane);
            tail_slot = tail_slot + 1 == kSlots ? 0 : tail_slot + 1;
            --flying;
        }
        __syncwarp();
#pragma unroll 1
        for (int i = flying; i < kSlots; ++i) ask_ahead();
        for (; own <= own1; own += kClasses) {
            const int key0 = key_lo + kStep * own;
            const long long a = ((static_cast<long long>(I.slot_of(cur.w0)) * P.Hkv + cur.kvh) * hp.tail + key0 % hp.tail) * HD;
            rs.own_step(hp.k_tail + a, hp.v_tail + a, sm.q, P.scale_log2, pos, tmax, key0, lane);
        }
        const int r0 = cur.tile * 8 * T;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (t + e > 0) __syncthreads();    // the rows before have been joined
                rs.put(t, e, sm.ml, sm.o, cls, bad_rows[t], cur.rows - r0 - 8 * t, lane);
                __syncthreads();
                for (int x4 = tid; x4 < 4 * (HD / 4); x4 += kHeldThreads) {
                    const int row = x4 / (HD / 4), in_tile = 2 * row + e, d = (x4 % (HD / 4)) * 4, row_pos = sm.pos[buf][8 * t + in_tile];
                    if (row_pos < key_lo) continue;
                    int j, head;
                    row_head(P, r0 + 8 * t + in_tile, j, head);
                    join_row<HD>(P, sm.o, sm.ml, row, d, row_pos, static_cast<long long>(cur.w0 + j) * P.Hq + cur.kvh * P.G + head, cur.split);
                }
            }
        if (!more) break;
        put_queries(next_q, next_pos, buf ^ 1);    // nobody reads this item's any more
        cur = nxt;
        steps = next_steps;
        asked = next_asked;
    }
}

// ---- small calls: a cluster of C CTAs per (request, KV head, 8 query rows), CTA c taking split c;
// the partials stay in shared memory, and CTA c joins query rows c, c + C, ... of all
// splits.  One launch, no table of items and no workspace where the two kernels would mostly wait.
// The same steps, joins and bits.  One row of 700 keys: 6.9 us, 9.9 with the two kernels; the chain of
// a class's eight steps bounds it.
template <int HD>
struct __align__(128) HeldSmallSmem {
    HeldSlot<HD> slots[kClasses][kSlots];
    float o[kClasses][4][HD + 4];          // of half a tile
    float part[8][HD];                     // the split's outputs
    float2 part_ml[8];
    HeldQ<HD, 1> q;
    float2 ml[kClasses][4];
};

template <int HD, int C>
__global__ void __launch_bounds__(kHeldThreads, 3) paged_attn_held_small_kernel(const PagedAttnParams P, const HeldPools hp) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    HeldSmallSmem<HD>& sm = *reinterpret_cast<HeldSmallSmem<HD>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, cls = tid >> 5;
    const int c4 = lane & 3;
    const int split = static_cast<int>(cluster_ctarank()), key_lo = split * kSplit;
    const int tiles = (P.rpg * P.G + 7) / 8, p = blockIdx.x / C / tiles, tile = blockIdx.x / C - p * tiles;
    const int grp = p / P.Hkv, kvh = p - grp * P.Hkv;
    const int w0 = grp * P.rpg, r0 = 8 * tile, rows = min(8, min(P.rpg, P.W - w0) * P.G - r0);   // none: a last group that is not full
    const uint64_t policy = policy_evict_first();
    int pos[1][2], last[1][2], tmax = -1, tmin = 0x7fffffff, all = 0x7fffffff;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * c4 + e;
        pos[0][e] = i < rows ? usable_pos(P, w0 + (r0 + i) / P.G, split == 0 && kvh == 0) : -1;
        last[0][e] = pos[0][e] < 0 ? -1 : (pos[0][e] & ~(kStep - 1)) - 1;
        tmax = max(tmax, pos[0][e]);
        if (pos[0][e] >= 0) tmin = min(tmin, pos[0][e]);
        if (pos[0][e] >= key_lo) all = min(all, last[0][e]);
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, d));
        tmin = min(tmin, __shfl_xor_sync(0xffffffffu, tmin, d));
        all = min(all, __shfl_xor_sync(0xffffffffu, all, d));
    }
    const int held = (tmax & ~(kStep - 1)) - 1, nsteps = held < 0 ? 0 : Items::steps_to(held, split);      // -1 & ~15 is -16
    HeldSteps steps;
    steps.n = (nsteps - cls + kClasses - 1) / kClasses;
    steps.page = 0;
    const int lane_key = key_lo + kStep * (cls + kClasses * lane);
    if (lane < steps.n) steps.page = P.pt.table[static_cast<long long>(P.row_slot[w0]) * P.pt.max_pages + (lane_key >> P.pt.page_shift)];
    steps.bad = bad_pages(P, steps.page);
    pdl_wait();
    pdl_trigger();
    HeldSlot<HD>* const slots = sm.slots[cls];
    const int first = HeldSlot<HD>::first(lane);
    auto ask = [&](int i) {
        const long long at = held_at<HD>(P, __shfl_sync(0xffffffffu, steps.page, i), kvh, key_lo + kStep * (cls + kClasses * i)) + 16 * lane;
        slots[i % kSlots].copy(hp.k + at, hp.v + at, first, policy);
    };
    int asked = min(steps.n, kSlots);
    for (int i = 0; i < asked; ++i) ask(i);
    steps.k_scale = steps.v_scale = 0.0f;
    if (lane < steps.n) scales_at<HD>(hp, steps, lane, held_at<HD>(P, steps.page, kvh, lane_key));
    if (tid < HD) {                                // 8 rows of HD / 8 pieces; rows past the group's read its first row and are never used
        const int row = tid / (HD / 8), d = tid % (HD / 8), i = row < rows ? r0 + row : 0;
        const uint4 x = *reinterpret_cast<const uint4*>(P.q + (static_cast<long long>(w0 + i / P.G) * P.Hq + kvh * P.G + i % P.G) * HD + d * 8);
        put_q(sm.q, x, row, d, P.scale_log2);
    }
    __syncthreads();
    float back[1][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) back[0][e] = sm.q.back[0][2 * c4 + e];
    HeldRows<HD, 1> rs;
    rs.clear();
    uint32_t bad_rows = 0;
#pragma unroll 1
    for (int i = 0; i < steps.n; ++i) {
        const int key0 = key_lo + kStep * (cls + kClasses * i);
        const bool step_bad = (steps.bad >> i) & 1u;
        if (step_bad) bad_rows |= (last[0][0] >= key0 ? 1u : 0u) | (last[0][1] >= key0 ? 2u : 0u);
        wait_copies(asked - i - 1);
        __syncwarp();                              // the step before has been read, this one's copies of all lanes are there
        if (asked - i < kSlots && asked < steps.n) ask(asked++);
        rs.step(slots[i % kSlots], sm.q, back, __shfl_sync(0xffffffffu, steps.k_scale, i), __shfl_sync(0xffffffffu, steps.v_scale, i), last, all, step_bad,
                key0, lane);
    }
    const int own1 = tmax < key_lo ? -1 : min(kSteps - 1, (tmax - key_lo) / kStep);
    int own = max(0, (tmin - key_lo) / kStep);
    own += (cls - own) & (kClasses - 1);
    for (; own <= own1; own += kClasses) {
        const int key0 = key_lo + kStep * own;
        const long long a = ((static_cast<long long>(P.row_slot[w0]) * P.Hkv + kvh) * hp.tail + key0 % hp.tail) * HD;
        rs.own_step(hp.k_tail + a, hp.v_tail + a, sm.q, P.scale_log2, pos, tmax, key0, lane);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (e > 0) __syncthreads();                // the rows before have been joined
        rs.put(0, e, sm.ml, sm.o, cls, bad_rows, rows, lane);
        __syncthreads();
        for (int x4 = tid; x4 < 4 * (HD / 4); x4 += kHeldThreads) {
            const int row = x4 / (HD / 4), d = (x4 % (HD / 4)) * 4;
            if (2 * row + e >= rows) continue;
            float mx, sum;
            *reinterpret_cast<float4*>(&sm.part[2 * row + e][d]) = join_dims<HD>(sm.o, sm.ml, row, d, mx, sum);
            if (d == 0) sm.part_ml[2 * row + e] = make_float2(mx, sum);
        }
    }
    cluster_sync();
    // query rows split, split + C, ..., joined as the combine kernel does (up to 16 splits: one block)
    for (int r = split; r < rows; r += C) {
        const int w = w0 + (r0 + r) / P.G;
        const int row_pos = usable_pos(P, w, false), ns = row_pos < 0 ? 0 : row_pos / kSplit + 1;
        const long long pair = static_cast<long long>(w) * P.Hq + kvh * P.G + (r0 + r) % P.G;
        const float2 mine = lane < ns ? ld_cluster(&sm.part_ml[r], lane) : make_float2(-INFINITY, 0.0f);
        float x[C] = {};
        if (tid < HD) {
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (k < ns) x[k] = ld_cluster(&sm.part[r][tid], k);
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
        for (int k = 0; k < C; ++k) {
            const float f = __shfl_sync(0xffffffffu, f_lane, k);
            if (k < ns) acc = fmaf(x[k], f, acc);
        }
        if (tid < HD) P.o[pair * HD + tid] = __float2bfloat16_rn(broken || ns == 0 ? 0.0f : acc * (1.0f / l));
    }
    cluster_sync();                                // nobody leaves while its shared memory is read
}

template <typename F>
int allow_smem(F* kernel, size_t bytes) {
    return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)));
}

template <int HD, int C>
int launch_held_small(const PagedAttnParams& P, const HeldPools& hp, long long tiles, cudaStream_t s) {
    static DeviceOnce once;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    const int st = once.run(dev, [] { return allow_smem(paged_attn_held_small_kernel<HD, C>, sizeof(HeldSmallSmem<HD>)); });
    if (st != BIV_OK) return st;
    return launch_cluster_pdl(paged_attn_held_small_kernel<HD, C>, dim3(static_cast<unsigned>(tiles * C)), dim3(kHeldThreads), sizeof(HeldSmallSmem<HD>), s, C, P, hp);
}

template <int HD, int T>
int launch_held(const PagedAttnParams& P, const HeldPools& hp, cudaStream_t s) {
    static DeviceOnce once;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    const int st = once.run(dev, [] { return allow_smem(paged_attn_held_kernel<HD, T>, sizeof(HeldSmem<HD, T>)); });
    if (st != BIV_OK) return st;
    const long long n_groups = (P.W + P.rpg - 1) / P.rpg, tiles = (static_cast<long long>(P.rpg) * P.G + 8 * T - 1) / (8 * T);
    const long long grid = std::min<long long>(n_groups * P.Hkv * P.s_max * tiles, static_cast<long long>(held_ctas(T)) * num_sms());
    return launch_pdl(paged_attn_held_kernel<HD, T>, dim3(static_cast<unsigned>(grid)), dim3(kHeldThreads), sizeof(HeldSmem<HD, T>), s, P, hp);
}

template <int HD>
int launch_held_attn(const PagedAttnParams& P, const HeldPools& hp, cudaStream_t s) {
    // Few tiles (of 8 query rows of a request and KV head) and short tables: one launch, with a CTA for every split
    // that the tables may need, if one round of CTAs holds them.  32 and 8 heads, us, with two kernels in
    // brackets: one token of 700 keys 7.0 (10.1), a window of five 7.9 (14.9), three such 10.9 (17.3); C = 2, 28
    // tokens of 700 (448 CTAs) 13.5 (15.4); C = 4, nine (288) 10.4 (13.2), 2048 keys 11.9 (14.3), but fourteen
    // (448) 15.7 (13.8): of larger clusters three CTAs an SM are no single round.
    const long long small = (P.W + P.rpg - 1LL) / P.rpg * P.Hkv * ((static_cast<long long>(P.rpg) * P.G + 7) / 8);
    if (P.s_max <= 2 && small * 2 <= 3LL * num_sms()) return launch_held_small<HD, 2>(P, hp, small, s);
    if (P.s_max <= 4 && small * 4 <= 2LL * num_sms()) return launch_held_small<HD, 4>(P, hp, small, s);
    if (P.s_max <= 8 && small * 8 <= 2LL * num_sms()) return launch_held_small<HD, 8>(P, hp, small, s);
    // as few passes over the keys as four tiles allow, each with as few tiles as they then need: 20 query rows
    // (windows of five, G = 4) in one pass of three tiles 57.7 us, in two of two 71.2
    const long long rows = static_cast<long long>(P.rpg) * P.G, passes = (rows + 31) / 32, T = (rows + 8 * passes - 1) / (8 * passes);
    const int st = T == 1 ? launch_held<HD, 1>(P, hp, s) : T == 2 ? launch_held<HD, 2>(P, hp, s)
                 : T == 3 ? launch_held<HD, 3>(P, hp, s) : launch_held<HD, 4>(P, hp, s);
    if (st != BIV_OK || P.s_max == 1) return st;
    return launch_combine<HD>(P, s);
}

// What both calls ask of the pools.
int check_held(const HeldPools& hp, const void* const (&p)[6]) {
    for (const void* x : p)
        if (!x) return BIV_ERR_NULL;
    for (int i = 0; i < 6; ++i)
        if (i == 2 || i == 3 ? (reinterpret_cast<uintptr_t>(p[i]) & 1u) != 0 : i < 2 ? (reinterpret_cast<uintptr_t>(p[i]) & 31u) != 0 : !aligned16(p[i]))
            return BIV_ERR_ALIGN;
    return BIV_OK;
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" int biv_rope_kv_write_paged_e4m3(const void* qkv, void* q_out, void* k_pages, void* v_pages, void* k_scales,
                                            void* v_scales, void* k_tail, void* v_tail, const int32_t* page_table,
                                            const int32_t* row_slot, const int32_t* row_pos, const int32_t* rows_keep, int W,
                                            int K, int Hq, int Hkv, int hd, int n_slots, int max_pages, int n_pages,
                                            int page_size, int tail, float theta, biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (W < 0 || K < 1 || Hq <= 0 || Hkv <= 0 || hd <= 0 || W % K != 0 || Hq % Hkv != 0 || Hq > (1 << 20)) return BIV_ERR_SHAPE;
    PageTable pt;
    int st = check_pages(n_slots, max_pages, n_pages, page_size, &pt);
    if (st != BIV_OK) return st;
    if (hd != 64 && hd != 128) return BIV_ERR_UNSUPPORTED;
    if (tail % kHeldBlock != 0 || tail < K + kHeldBlock - 1LL) return BIV_ERR_SHAPE;
    const int chunks = (K + kHeldBlock - 2) / kHeldBlock + 1;
    const long long grid = static_cast<long long>(W / K) * chunks * Hkv;
    if (grid > 0x7fffffffLL) return BIV_ERR_SHAPE;
    if (!(theta > 1.0f) || !std::isfinite(theta)) return BIV_ERR_VALUE;
    if (W == 0) return BIV_OK;
    if (!qkv || !q_out || !page_table || !row_slot || !row_pos) return BIV_ERR_NULL;
    const HeldPools hp{static_cast<uint8_t*>(k_pages), static_cast<uint8_t*>(v_pages), static_cast<__nv_bfloat16*>(k_scales),
                       static_cast<__nv_bfloat16*>(v_scales), static_cast<__nv_bfloat16*>(k_tail), static_cast<__nv_bfloat16*>(v_tail), tail};
    st = check_held(hp, {k_pages, v_pages, k_scales, v_scales, k_tail, v_tail});
    if (st != BIV_OK) return st;
    if (!aligned16(qkv) || !aligned16(q_out)) return BIV_ERR_ALIGN;
    pt.table = page_table;
    const RopeTurns& turns = rope_turns(theta, hd);
    return launch_pdl(hd == 128 ? rope_kv_write_held_kernel<128> : rope_kv_write_held_kernel<64>, dim3(static_cast<unsigned>(grid)),
                      dim3(kWriteThreads), 0, reinterpret_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(qkv),
                      static_cast<__nv_bfloat16*>(q_out), hp, pt, row_slot, row_pos, rows_keep, W / K, K, Hq, Hkv, chunks, turns);
}

extern "C" int biv_decode_attn_paged_e4m3(const void* q, const void* k_pages, const void* v_pages, const void* k_scales,
                                          const void* v_scales, const void* k_tail, const void* v_tail,
                                          const int32_t* page_table, const int32_t* row_slot, const int32_t* row_pos, void* o,
                                          int W, int rows_per_group, int Hq, int Hkv, int hd, int n_slots, int max_pages,
                                          int n_pages, int page_size, int tail, void* workspace, size_t ws_bytes,
                                          biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (W < 0 || rows_per_group <= 0 || Hq <= 0 || Hkv <= 0 || hd <= 0 || Hq % Hkv != 0) return BIV_ERR_SHAPE;
    PagedAttnParams P;
    int st = check_pages(n_slots, max_pages, n_pages, page_size, &P.pt);
    if (st != BIV_OK) return st;
    if (hd != 64 && hd != 128) return BIV_ERR_UNSUPPORTED;
    if (static_cast<long long>(W) * Hq > 0x7fffffffLL || tail < kHeldBlock || tail % kHeldBlock != 0) return BIV_ERR_SHAPE;
    if (W == 0) return BIV_OK;
    if (!q || !page_table || !row_slot || !row_pos || !o || !workspace) return BIV_ERR_NULL;
    auto out = [](const void* x) { return const_cast<void*>(x); };
    const HeldPools hp{static_cast<uint8_t*>(out(k_pages)), static_cast<uint8_t*>(out(v_pages)), static_cast<__nv_bfloat16*>(out(k_scales)),
                       static_cast<__nv_bfloat16*>(out(v_scales)), static_cast<__nv_bfloat16*>(out(k_tail)), static_cast<__nv_bfloat16*>(out(v_tail)), tail};
    st = check_held(hp, {k_pages, v_pages, k_scales, v_scales, k_tail, v_tail});
    if (st != BIV_OK) return st;
    if (!aligned16(q) || !aligned16(o) || !aligned16(workspace)) return BIV_ERR_ALIGN;
    if (ws_bytes < biv_decode_attn_paged_workspace_size(W, Hq, hd, max_pages, page_size)) return BIV_ERR_SHAPE;
    if (o == q) return BIV_ERR_VALUE;
    fill_attn(P, q, o, page_table, row_slot, row_pos, W, rows_per_group, Hq, Hkv, hd, max_pages, page_size, workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return hd == 128 ? launch_held_attn<128>(P, hp, s) : launch_held_attn<64>(P, hp, s);
}
