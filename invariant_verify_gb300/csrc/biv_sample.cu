// Sampled verification: softmax with temperature, and the rejection sampling of
// drafted tokens from given uniform numbers.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "biv_common.cuh"

namespace biv {
namespace {

BIV_DEFINE_ERR_WORD(g_sample_err)

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPerLoad = 4 * kThreads;        // entries that one 16-byte load a thread covers

// A NaN logit counts as -infinity (fmaxf returns the operand that is a number).
BIV_DEV float no_nan(float x) { return fmaxf(x, -INFINITY); }
BIV_DEV float4 no_nan(float4 r) { return make_float4(no_nan(r.x), no_nan(r.y), no_nan(r.z), no_nan(r.w)); }

// Four entries of a row from v on, `fill` past its end.  VEC: rows are 16-byte
// aligned and whole groups are read at once; else one by one.  The same entries
// either way, so the same bits.
template <bool VEC>
BIV_DEV float4 load4(const float* x, int v, int V, float fill) {
    if (VEC && v + 4 <= V) {
        float4 r;
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(x + v));
        return r;
    }
    float4 r = make_float4(fill, fill, fill, fill);
    if (v < V) r.x = x[v];
    if (v + 1 < V) r.y = x[v + 1];
    if (v + 2 < V) r.z = x[v + 2];
    if (v + 3 < V) r.w = x[v + 3];
    return r;
}
template <bool VEC>
BIV_DEV void store4(float* p, int v, int V, float4 r) {
    if (VEC && v + 4 <= V) {
        *reinterpret_cast<float4*>(p + v) = r;
        return;
    }
    if (v < V) p[v] = r.x;
    if (v + 1 < V) p[v + 1] = r.y;
    if (v + 2 < V) p[v + 2] = r.z;
    if (v + 3 < V) p[v + 3] = r.w;
}

// A CTA's shared memory may be written by the others of its cluster once all have
// started: each says so as it begins and waits for the others before its first write.
BIV_DEV void cluster_started() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
BIV_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// A shared variable of the cluster's CTA `rank`.
BIV_DEV void put_cluster(const void* p, uint32_t rank, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(p, rank)), "f"(x) : "memory");
}
BIV_DEV void put_cluster(const void* p, uint32_t rank, int x) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(mapa_shared(p, rank)), "r"(x) : "memory");
}
BIV_DEV void put_cluster(const void* p, uint32_t rank, unsigned long long x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(p, rank)), "l"(x) : "memory");
}

// ---------------------------------------------------------------- softmax
// A row belongs to a cluster of C CTAs, each of which keeps its slice in registers
// (NV groups of four per thread): one read and one write of the row, and one
// exchange of (maximum, sum) between the CTAs.  p = e^((x - m_c) / T) / S_c's share:
// each CTA's exponentials stand on its own maximum m_c and are scaled once by
// e^((m_c - m) / T) / S.  C and NV go by V alone, so a row's bits do not depend on the
// batch.  Rows past 8 x 16 x 2048 entries are read twice.  A few rows are bound by
// latency: 5 x 32000 take 3.6 us.
constexpr int kMaxCluster = 8;
constexpr unsigned long long kLandingNs = 1000000ull;      // for a message between two SMs, about 1 us: plenty

// Exponentials of a slice on its own maximum: an infinite maximum's entries share the
// mass (differences would be NaN), a slice of nothing but -infinity gives zeros.
struct SlicePower {
    float zero_at, scale;
    bool infinite;
    BIV_DEV SlicePower(float m, float s) : zero_at(m == INFINITY || m == -INFINITY ? 0.0f : m), scale(s), infinite(m == INFINITY) {}
    BIV_DEV float4 operator()(float4 y) const {
        if (infinite)
            y = make_float4(y.x == INFINITY ? 0.0f : -INFINITY, y.y == INFINITY ? 0.0f : -INFINITY,
                            y.z == INFINITY ? 0.0f : -INFINITY, y.w == INFINITY ? 0.0f : -INFINITY);
        return make_float4(ex2_approx((y.x - zero_at) * scale), ex2_approx((y.y - zero_at) * scale),
                           ex2_approx((y.z - zero_at) * scale), ex2_approx((y.w - zero_at) * scale));
    }
};

BIV_DEV float max4(float m, float4 r) { return fmaxf(m, fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w))); }

// Largest value (sum) over the CTA, in an order that goes by the thread alone.
BIV_DEV float cta_max(float m, float* s_m) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) m = fmaxf(m, s_m[k]);
    return m;
}
BIV_DEV float cta_sum(float l, float* s_l) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if ((threadIdx.x & 31) == 0) s_l[threadIdx.x >> 5] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) l += s_l[k];
    return l;
}

// The factor of this CTA's exponentials, from (maximum, sum) of all C CTAs.
BIV_DEV float slice_factor(float m_cta, float scale, const float2* ml, int C) {
    float m = -INFINITY, sum = 0.0f;
    for (int k = 0; k < C; ++k) m = fmaxf(m, ml[k].x);
    auto share = [&](float mk) { return mk == -INFINITY ? 0.0f : mk == m ? 1.0f : m == INFINITY ? 0.0f : ex2_approx((mk - m) * scale); };
    for (int k = 0; k < C; ++k) sum = fmaf(ml[k].y, share(ml[k].x), sum);
    return m == -INFINITY ? 0.0f : share(m_cta) / sum;
}

BIV_DEV unsigned long long pack2(float a, float b) {
    return static_cast<unsigned long long>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}

BIV_DEV float4 times(float4 r, float f) { return make_float4(r.x * f, r.y * f, r.z * f, r.w * f); }

template <bool VEC, int NV, bool LONG>
__global__ void __launch_bounds__(kThreads, LONG || NV > 10 ? 1 : NV > 4 ? 2 : 3)
softmax_kernel(const float* logits, int V, long long ld, float scale, float* probs, long long ld_p, int C) {
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ __align__(8) float2 c_ml[kMaxCluster];
    const int tid = threadIdx.x;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const long long row = blockIdx.x / C;
    if (C > 1) cluster_started();
    pdl_wait();
    pdl_trigger();
    const float* x = logits + row * ld;
    float* p = probs + row * ld_p;
    // slices of whole rounds of NV loads; a CTA's are consecutive
    const int per = LONG ? (V + C * kPerLoad - 1) / (C * kPerLoad) * kPerLoad : NV * kPerLoad;
    const int v0 = rank * per + 4 * tid;
    const int end = min(V, (rank + 1) * per);

    float4 r[NV];
    float m = -INFINITY;
    for (int base = 0; base < per; base += NV * kPerLoad) {
#pragma unroll
        for (int k = 0; k < NV; ++k) r[k] = load4<VEC>(x, v0 + base + k * kPerLoad, end, -INFINITY);
#pragma unroll
        for (int k = 0; k < NV; ++k) m = max4(m, r[k] = no_nan(r[k]));
    }
    m = cta_max(m, s_m);
    const SlicePower power(m, scale);
    float l = 0.0f;
    for (int base = 0; base < per; base += NV * kPerLoad) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (LONG) r[k] = no_nan(load4<VEC>(x, v0 + base + k * kPerLoad, end, -INFINITY));
            r[k] = power(r[k]);
            l += (r[k].x + r[k].y) + (r[k].z + r[k].w);
        }
    }
    l = cta_sum(l, s_l);
    float factor = m == -INFINITY ? 0.0f : 1.0f / l;
    if (C > 1) {
        cluster_wait();
        if (tid < C) put_cluster(&c_ml[rank], tid, pack2(m, l));
        cluster_sync();
        factor = slice_factor(m, scale, c_ml, C);
    }
    for (int base = 0; base < per; base += NV * kPerLoad) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = v0 + base + k * kPerLoad;
            if constexpr (LONG) r[k] = power(no_nan(load4<VEC>(x, v, end, -INFINITY)));
            if (v < end) store4<VEC>(p, v, end, times(r[k], factor));
        }
    }
}

// Many rows of a large vocabulary: the clusters stay and take row after row, and the
// next row's slice is on its way into shared memory (one bulk copy, as soon as the
// threads hold the row before) while a row is summed and written.  The same slices,
// orders and bits as softmax_kernel, whose CTAs read, wait for one another and write
// in turn.  (Maximum, sum) travel by asynchronous stores that count on a barrier of
// the receiving CTA: a cluster barrier's release would wait until the row before has
// been written out.  Bound by memory: 320 x 128256 take 57 to 58 us, 5.7 TB/s (a cluster
// a row: 72; cluster barriers: 73).
// A wait that runs out raises its bit and the CTA's flag, and the CTA leaves at the row's
// next barrier, where all its threads see the flag; its cluster's other CTAs then miss its
// numbers and leave in the same way, and the cluster's rows from there on are not written.
// LOSE (the self-test): rank 0 never asks for row `lose`.
template <int NV, bool LOSE = false>
__global__ void __launch_bounds__(kThreads, 2)
softmax_rows_kernel(const float* logits, int R, int V, long long ld, float scale, float* probs, long long ld_p, int lose) {
    constexpr int kSlice = NV * kPerLoad, C = kMaxCluster;
    extern __shared__ __align__(16) float s_x[];           // [kSlice]
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ __align__(8) float2 c_ml[2][C];
    __shared__ uint64_t full, heard[2];
    __shared__ int abort_flag;
    const int tid = threadIdx.x;
    const int rank = static_cast<int>(cluster_ctarank());
    const int step = gridDim.x / C;
    const int start = rank * kSlice, n = min(max(V - start, 0), kSlice);      // this CTA's slice of every row
    if (tid == 0) {
        mbar_init(&full, 1);
        mbar_init(&heard[0], 1);
        mbar_init(&heard[1], 1);
        abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    cluster_started();
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    auto fetch = [&](int row) {                            // by one thread
        mbar_arrive_expect_tx(&full, static_cast<uint32_t>(n) * 4u);
        if (LOSE && rank == 0 && row == lose) return;
        if (n > 0)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(s_x)),
                         "l"(logits + static_cast<long long>(row) * ld + start), "r"(n * 4), "r"(smem_u32(&full))
                         : "memory");
    };
    int row = blockIdx.x / C;
    if (tid == 0) fetch(row);                              // the grid holds no more clusters than rows
    cluster_wait();
    uint32_t heard_phase = 0, phase = 0;
    volatile int* const gave_up = &abort_flag;
    for (; row < R; row += step, phase ^= 1u) {
        mbar_wait(&full, phase, gave_up, &g_sample_err);
        const float* x = s_x + 4 * tid;
        float4 r[NV];
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            r[k] = 4 * tid + k * kPerLoad < n ? no_nan(*reinterpret_cast<const float4*>(x + k * kPerLoad))
                                              : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            m = max4(m, r[k]);
        }
        m = cta_max(m, s_m);                               // its barrier: every thread has read the buffer, or raised the flag
        if (*gave_up) break;                               // (nothing raises it between that barrier and the next one)
        if (tid == 0 && row + step < R) fetch(row + step);
        const SlicePower power(m, scale);
        float l = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            r[k] = power(r[k]);
            l += (r[k].x + r[k].y) + (r[k].z + r[k].w);
        }
        l = cta_sum(l, s_l);
        // to every CTA's buffer of this row (two in turn: a CTA sends a row's only after
        // all its threads are done with the one before, so none is overwritten early)
        if (tid == 0) mbar_arrive_expect_tx(&heard[phase], C * 8);
        if (tid < C)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                             mapa_shared(&c_ml[phase][rank], tid)),
                         "l"(pack2(m, l)), "r"(mapa_shared(&heard[phase], tid))
                         : "memory");
        if (!mbar_wait(&heard[phase], heard_phase, gave_up, &g_sample_err, false, true)) continue;
        if (phase) heard_phase ^= 1u;
        const float factor = slice_factor(m, scale, c_ml[phase], C);
        float* p = probs + static_cast<long long>(row) * ld_p + start + 4 * tid;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (4 * tid + k * kPerLoad < n) *reinterpret_cast<float4*>(p + k * kPerLoad) = times(r[k], factor);
    }
    __syncthreads();
    if (!*gave_up) return;
    // Nothing may land here once the CTA has left: its own copy, and the numbers of peers, which
    // have stopped sending when they come to this barrier (or have left), a moment later.
    if (row < R && tid == 0) mbar_wait_drain(&full, phase);
    cluster_started();
    cluster_wait();
    for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < kLandingNs;) {}
}

// T == 0: one CTA per row finds the lowest index of its largest entry and writes the row.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
softmax_greedy_kernel(const float* logits, int V, long long ld, float* probs, long long ld_p) {
    __shared__ float s_m[kWarps];
    __shared__ int s_i[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const float* x = logits + static_cast<long long>(blockIdx.x) * ld;
    float* p = probs + static_cast<long long>(blockIdx.x) * ld_p;
    float m = -INFINITY;
    int at = 0x7fffffff;
    auto take = [&](float om, int oi) {
        if (om > m || (om == m && oi < at)) m = om, at = oi;
    };
    for (int v = 4 * tid; v < V; v += kPerLoad) {
        const float4 r = no_nan(load4<VEC>(x, v, V, -INFINITY));
        const float m4 = fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w));
        if (m4 > m) m = m4, at = v + (r.x == m4 ? 0 : r.y == m4 ? 1 : r.z == m4 ? 2 : 3);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, d);
        const int oi = __shfl_xor_sync(0xffffffffu, at, d);
        take(om, oi);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_i[warp] = at;
    }
    __syncthreads();
    for (int k = 0; k < kWarps; ++k) take(s_m[k], s_i[k]);
    for (int v = 4 * tid; v < V; v += kPerLoad)
        store4<VEC>(p, v, V, make_float4(v == at ? 1.0f : 0.0f, v + 1 == at ? 1.0f : 0.0f, v + 2 == at ? 1.0f : 0.0f, v + 3 == at ? 1.0f : 0.0f));
}

// ----------------------------------------------------------------- verify
// A weight in units of 2^-60 (truncated), clamped to [0, 1]; a NaN counts as 0.
BIV_DEV float clamp01(float w) { return fminf(fmaxf(w, 0.0f), 1.0f); }
// By shifts of the significand: conversions to 64-bit integers run at the rate of
// this part's few FP64 units (64 x 128256 entries: 44 us with them, 32 without).
BIV_DEV unsigned long long units(float w) {
    const uint32_t b = __float_as_uint(w), down = 130u - (b >> 23);
    const unsigned long long top = static_cast<unsigned long long>((b << 8) | 0x80000000u) << 32;      // 2^63 (1 + fraction)
    return down < 64u ? top >> down : 0ull;
}

// floor(u x) for 0 <= u < 1, exactly: the product of u's 24-bit significand and x, in 128
// bits, shifted down.  (A double keeps 53 of the product's up to 88 bits.)
BIV_DEV unsigned long long floor_share(float u, unsigned long long x) {
    const uint32_t b = __float_as_uint(u) & 0x7fffffffu, e = b >> 23;      // a zero may be a negative one
    const unsigned long long m = e ? (b & 0x7fffffu) | 0x800000u : b;
    const uint32_t down = 150u - (e ? e : 1u);             // u = m 2^-down, 24 <= down
    const unsigned long long lo = m * x, hi = __umul64hi(m, x);
    return down < 64u ? hi << (64u - down) | lo >> down : down < 128u ? hi >> (down - 64u) : 0ull;
}

BIV_DEV unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// One request per cluster of C CTAs, a contiguous chunk of the row per warp.  Every
// CTA finds the first rejected draft (a few gathered numbers), each warp sums the
// weights of its chunk in 64-bit integers, and the warp that holds the border reads
// the part of its chunk again (from L2) where its kept sums pass the border, down to the
// entry.  Sums of integers do not depend on their order, so C may follow the batch.
// 64 requests of 128256 entries: 16.0 us, of which some 10 stream the rows at the rate of
// memory; the rest are the dependent reads before a request's rows are known and the
// steps from the sums to the token.
constexpr int kKeptGoes = 4;           // goes of 512 entries whose sums are kept (64 x 128256 entries, four to a warp: 18.4 -> 16.3 us)
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
verify_sample_kernel(const float* __restrict__ target, const float* __restrict__ draft_probs,
                     const int32_t* __restrict__ draft, const float* __restrict__ u_accept,
                     const float* __restrict__ u_sample, const int32_t* __restrict__ p0, int K, int V,
                     int32_t* __restrict__ tokens, int32_t* __restrict__ accept_len, int32_t* __restrict__ new_len, int C) {
    __shared__ int s_n;
    __shared__ unsigned long long s_sum[kWarps];
    __shared__ float s_f[kWarps];
    __shared__ unsigned long long c_sum[2][kMaxCluster];
    __shared__ float c_f[2][kMaxCluster];
    __shared__ unsigned long long s_go[kWarps][kKeptGoes][32];     // the lanes' sums of a warp's first goes
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const long long r = blockIdx.x / C;
    if (tid == 0) s_n = K;
    if (C > 1) cluster_started();
    pdl_wait();
    pdl_trigger();
    const float u = fminf(fmaxf(u_sample[r], 0.0f), 0.99999994f);
    __syncthreads();
    for (int j = tid; j < K; j += kThreads) {
        const long long row = r * K + j;
        const int d = draft[row];
        bool ok = false;
        if (d < 0 || d >= V) {
            if (rank == 0) atomicOr(&g_sample_err, BIV_DEVERR_INDEX);
        } else {
            const float p = clamp01(target[(r * (K + 1) + j) * V + d]);
            const float q = draft_probs ? clamp01(draft_probs[row * V + d]) : 1.0f;
            // the product of two 24-bit numbers is exact in 64 bits
            ok = static_cast<double>(u_accept[row]) * static_cast<double>(q) < static_cast<double>(p);
        }
        if (!ok) atomicMin(&s_n, j);
    }
    __syncthreads();
    const int n = s_n;
    const float* p = target + (r * (K + 1) + n) * V;
    const float* q = draft_probs && n < K ? draft_probs + (r * K + n) * V : nullptr;
    const int skip = !draft_probs && n < K ? draft[r * K + n] : -1;
    constexpr int kRound = 128;                            // entries of one load of a warp
    const int parts = C * kWarps;
    const int chunk = (V + parts * kRound - 1) / (parts * kRound) * kRound;
    const int v0 = min(V, (rank * kWarps + warp) * chunk), end = min(V, v0 + chunk);

    // kDeep rounds of weights, all their loads first
    constexpr int kDeep = 4, kGo = kDeep * kRound;
    auto weights = [&](int v, bool plain, float4 (&w)[kDeep]) {
        float4 y[kDeep];
        const bool diff = q && !plain;
#pragma unroll
        for (int k = 0; k < kDeep; ++k) w[k] = load4<VEC>(p, v + k * kRound, end, 0.0f);
        if (diff) {
#pragma unroll
            for (int k = 0; k < kDeep; ++k) y[k] = load4<VEC>(q, v + k * kRound, end, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            if (diff) w[k] = make_float4(w[k].x - y[k].x, w[k].y - y[k].y, w[k].z - y[k].z, w[k].w - y[k].w);
            w[k] = make_float4(clamp01(w[k].x), clamp01(w[k].y), clamp01(w[k].z), clamp01(w[k].w));
        }
        if (skip >= 0 && !plain) {
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                const int at = skip - v - k * kRound;
                if (at == 0) w[k].x = 0.0f;
                if (at == 1) w[k].y = 0.0f;
                if (at == 2) w[k].z = 0.0f;
                if (at == 3) w[k].w = 0.0f;
            }
        }
    };
    unsigned long long total = 0, before = 0;
    float all = 0.0f;
    bool plain = false;
    for (int round = 0; round < 2; ++round) {
        unsigned long long sum = 0;
        float f = 0.0f;
        for (int go = 0; v0 + go * kGo < end; ++go) {
            float4 w[kDeep];
            unsigned long long part = 0;
            weights(v0 + go * kGo + 4 * lane, plain, w);
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                part += (units(w[k].x) + units(w[k].y)) + (units(w[k].z) + units(w[k].w));
                f += (w[k].x + w[k].y) + (w[k].z + w[k].w);
            }
            if (go < kKeptGoes && end - v0 > kGo) s_go[warp][go][lane] = part;
            sum += part;
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) f += __shfl_xor_sync(0xffffffffu, f, d);
        __syncthreads();                                   // the round before has read s_sum
        if (lane == 0) {
            s_sum[warp] = sum;
            s_f[warp] = f;
        }
        __syncthreads();
        sum = 0;
        f = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            sum += s_sum[k];
            f += s_f[k];
        }
        before = 0;
        if (C > 1) {
            if (round == 0) cluster_wait();
            if (tid < C) {
                put_cluster(&c_sum[round][rank], tid, sum);
                put_cluster(&c_f[round][rank], tid, f);
            }
            cluster_sync();
            total = 0;
            all = 0.0f;
            for (int k = 0; k < C; ++k) {
                if (k == rank) before = total;
                total += c_sum[round][k];
                all += c_f[round][k];
            }
            sum = c_sum[round][rank];
        } else {
            total = sum;
            all = f;
        }
        if (total > 0 || plain) break;                     // the same in every CTA
        plain = true;
    }
    // Below 8 by the exact sum, whatever order `all` was added in: that sum, some 2^-10 off at
    // most (8192 additions a thread of the largest row), only tells whether total has passed
    // its 64 bits, at 16.
    const bool valid = total > 0 && all < 12.0f && total < 8ull << 60;
    const unsigned long long border = floor_share(u, total);       // S_v > u S where S_v is above it: both are integers
    if (rank == 0) {
        for (int j = tid; j <= K; j += kThreads)
            if (j != n || !valid) tokens[r * (K + 1) + j] = j < n ? draft[r * K + j] : j == n ? 0 : -1;
        if (tid == 0) {
            if (!valid) atomicOr(&g_sample_err, BIV_DEVERR_VALUE);
            accept_len[r] = n + 1;
            new_len[r] = p0[r] + n + 1;
        }
    }
    if (!valid) return;
    // s_sum still holds the warps' sums: the warp whose share holds the border walks its chunk
    unsigned long long at = before;
    for (int k = 0; k < warp; ++k) at += s_sum[k];
    if (border < at || border >= at + s_sum[warp]) return;
    int go0 = 0;                                           // the go that holds the border, or the first one not kept
    if (end - v0 > kGo) {
        unsigned long long kept[kKeptGoes];
#pragma unroll
        for (int k = 0; k < kKeptGoes; ++k) kept[k] = v0 + k * kGo < end ? warp_sum(s_go[warp][k][lane]) : 0;
        while (go0 < kKeptGoes) {
            unsigned long long here = 0;
#pragma unroll
            for (int k = 0; k < kKeptGoes; ++k) here = k == go0 ? kept[k] : here;
            if (border < at + here) break;
            at += here;
            ++go0;
        }
    }
    for (int v = v0 + go0 * kGo; v < end; v += kGo) {
        float4 w[kDeep];
        weights(v + 4 * lane, plain, w);
        unsigned long long four[kDeep], incl[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) incl[k] = four[k] = (units(w[k].x) + units(w[k].y)) + (units(w[k].z) + units(w[k].w));
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                const unsigned long long o = __shfl_up_sync(0xffffffffu, incl[k], s);
                if (lane >= s) incl[k] += o;
            }
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const unsigned long long pre = at + incl[k] - four[k];
            if (border >= pre && border < pre + four[k]) {
                const unsigned long long a = pre + units(w[k].x), b = a + units(w[k].y), c = b + units(w[k].z);
                tokens[r * (K + 1) + n] = v + 4 * lane + k * kRound + (border < a ? 0 : border < b ? 1 : border < c ? 2 : 3);
            }
            at += __shfl_sync(0xffffffffu, incl[k], 31);
        }
        if (border < at) return;
    }
}

bool aligned_rows(const float* p, long long ld) { return aligned16(p) && ld % 4 == 0; }

template <bool VEC, int NV, bool LONG>
int launch_softmax(const float* x, int R, int V, long long ld, float scale, float* p, long long ld_p, int C,
                   cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(R) * C);
    if (C == 1)
        return launch_pdl(softmax_kernel<VEC, NV, LONG>, grid, dim3(kThreads), 0, s, x, V, ld, scale, p, ld_p, C);
    return launch_cluster_pdl(softmax_kernel<VEC, NV, LONG>, grid, dim3(kThreads), 0, s, C, x, V, ld, scale, p, ld_p, C);
}

// Many rows: as many clusters of softmax_rows_kernel as the device holds at once.
// *done = false: the rows fit softmax_kernel's one wave (or the device holds none).
template <int NV, bool LOSE = false>
int launch_softmax_rows(const float* x, int R, int V, long long ld, float scale, float* p, long long ld_p, bool* done,
                        cudaStream_t s, int lose = -1) {
    constexpr int smem = NV * kPerLoad * 4;
    static std::mutex mu;
    static int resident[kMaxDevices] = {};                 // clusters, 0: not yet asked, -1: none
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    if (dev < 0 || dev >= kMaxDevices) return BIV_ERR_DEVICE;
    int n = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (resident[dev] == 0) {
            e = cudaFuncSetAttribute(softmax_rows_kernel<NV, LOSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return cuda_status(e);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(2 * num_sms() / kMaxCluster * kMaxCluster));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = kMaxCluster;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int most = 0;
            e = cudaOccupancyMaxActiveClusters(&most, softmax_rows_kernel<NV, LOSE>, &cfg);
            if (e != cudaSuccess) return cuda_status(e);
            resident[dev] = most > 0 ? most : -1;
        }
        n = resident[dev];
    }
    *done = n > 0 && R > n;
    if (!*done) return BIV_OK;
    return launch_cluster_pdl(softmax_rows_kernel<NV, LOSE>, dim3(static_cast<unsigned>(n) * kMaxCluster), dim3(kThreads), smem, s,
                              kMaxCluster, x, R, V, ld, scale, p, ld_p, lose);
}

// Loads a thread and CTAs a row, by V alone: up to four loads a thread, then up to
// eight CTAs, then more loads.
template <bool VEC>
int launch_softmax(const float* x, int R, int V, long long ld, float scale, bool greedy, float* p, long long ld_p,
                   cudaStream_t s) {
    if (greedy)
        return launch_pdl(softmax_greedy_kernel<VEC>, dim3(static_cast<unsigned>(R)), dim3(kThreads), 0, s, x, V, ld, p, ld_p);
    const int loads = (V + kPerLoad - 1) / kPerLoad;
    if (loads <= 1) return launch_softmax<VEC, 1, false>(x, R, V, ld, scale, p, ld_p, 1, s);
    if (loads <= 4) return launch_softmax<VEC, 4, false>(x, R, V, ld, scale, p, ld_p, 1, s);
    if (VEC && V % 4 == 0 && loads > 16 && loads <= 80) {           // a bulk copy takes whole 16-byte groups
        bool done = false;
        const int st = loads <= 32   ? launch_softmax_rows<4>(x, R, V, ld, scale, p, ld_p, &done, s)
                       : loads <= 64 ? launch_softmax_rows<8>(x, R, V, ld, scale, p, ld_p, &done, s)
                                     : launch_softmax_rows<10>(x, R, V, ld, scale, p, ld_p, &done, s);
        if (st != BIV_OK || done) return st;
    }
    if (loads <= 32) return launch_softmax<VEC, 4, false>(x, R, V, ld, scale, p, ld_p, loads <= 8 ? 2 : loads <= 16 ? 4 : 8, s);
    if (loads <= 64) return launch_softmax<VEC, 8, false>(x, R, V, ld, scale, p, ld_p, 8, s);
    if (loads <= 80) return launch_softmax<VEC, 10, false>(x, R, V, ld, scale, p, ld_p, 8, s);
    if (loads <= 128) return launch_softmax<VEC, 16, false>(x, R, V, ld, scale, p, ld_p, 8, s);
    return launch_softmax<VEC, 8, true>(x, R, V, ld, scale, p, ld_p, 8, s);
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" int biv_softmax(const float* logits, int R, int V, long long ld, float temperature, float* probs,
                           long long ld_p, biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (R < 0 || V < 1 || ld < V || ld_p < V) return BIV_ERR_SHAPE;
    if (V > (1 << 22)) return BIV_ERR_UNSUPPORTED;
    if (!(temperature >= 0.0f) || !(temperature < INFINITY)) return BIV_ERR_VALUE;
    if (R == 0) return BIV_OK;
    if (!logits || !probs) return BIV_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(logits) & 3u) || (reinterpret_cast<uintptr_t>(probs) & 3u)) return BIV_ERR_ALIGN;
    if (logits == probs && ld != ld_p) return BIV_ERR_VALUE;
    // log2(e) / T; a T so small that it would overflow leaves the largest entries alone, as it should
    const float scale = temperature == 0.0f ? 0.0f
                                            : static_cast<float>(std::min(1.4426950408889634 / temperature, 3.4028234663852886e38));
    if (static_cast<long long>(R) * kMaxCluster > 0x7fffffffLL) return BIV_ERR_SHAPE;
    const bool greedy = temperature == 0.0f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return aligned_rows(logits, ld) && aligned_rows(probs, ld_p)
               ? launch_softmax<true>(logits, R, V, ld, scale, greedy, probs, ld_p, s)
               : launch_softmax<false>(logits, R, V, ld, scale, greedy, probs, ld_p, s);
}

extern "C" int biv_selftest_softmax_lost_row(const float* logits, int R, int V, float* probs, int row, biv_stream_t stream) {
    BIV_TRACE_CALL();
    constexpr int NV = 4;
    if (R < 1 || row < 0 || row >= R || V % 4 != 0) return BIV_ERR_SHAPE;
    if (V <= 16 * kPerLoad || V > NV * kPerLoad * kMaxCluster) return BIV_ERR_UNSUPPORTED;
    if (!logits || !probs) return BIV_ERR_NULL;
    if (!aligned16(logits) || !aligned16(probs)) return BIV_ERR_ALIGN;
    bool done = false;
    const int st = launch_softmax_rows<NV, true>(logits, R, V, V, 1.4426950408889634f, probs, V, &done,
                                                 reinterpret_cast<cudaStream_t>(stream), row);
    return st != BIV_OK ? st : done ? BIV_OK : BIV_ERR_SHAPE;
}

extern "C" int biv_verify_sample(const float* target, const float* draft_probs, const int32_t* draft,
                                 const float* u_accept, const float* u_sample, const int32_t* p0, int N, int K, int V,
                                 int32_t* tokens, int32_t* accept_len, int32_t* new_len, biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (N < 0 || K < 0 || K > 1024 || V < 1) return BIV_ERR_SHAPE;
    if (V > (1 << 22)) return BIV_ERR_UNSUPPORTED;
    if (N == 0) return BIV_OK;
    if (!target || !u_sample || !p0 || !tokens || !accept_len || !new_len) return BIV_ERR_NULL;
    if (K > 0 && (!draft || !u_accept)) return BIV_ERR_NULL;
    if (static_cast<long long>(N) * kMaxCluster > 0x7fffffffLL) return BIV_ERR_SHAPE;
    // CTAs of a request: as many as its row gives work, fewer where the requests alone fill the machine
    int C = 1;
    while (C < kMaxCluster && C * kPerLoad < V && 2LL * N * C <= 2LL * num_sms()) C *= 2;
    const bool vec = aligned_rows(target, V) && (!draft_probs || aligned_rows(draft_probs, V));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto kernel = vec ? verify_sample_kernel<true> : verify_sample_kernel<false>;
    const dim3 grid(static_cast<unsigned>(N) * C);
    if (C == 1)
        return launch_pdl(kernel, grid, dim3(kThreads), 0, s, target, draft_probs, draft, u_accept, u_sample, p0, K, V, tokens,
                          accept_len, new_len, C);
    return launch_cluster_pdl(kernel, grid, dim3(kThreads), 0, s, C, target, draft_probs, draft, u_accept, u_sample, p0, K, V,
                              tokens, accept_len, new_len, C);
}
