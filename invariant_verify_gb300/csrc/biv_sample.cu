// Sampled verification: softmax with temperature, and the rejection sampling of
// drafted tokens from given uniform numbers.
#include <algorithm>
#include <cmath>

#include "biv_common.cuh"

namespace biv {
namespace {

BIV_DEFINE_ERR_WORD(g_sample_err)

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// A NaN logit counts as -infinity.
BIV_DEV float no_nan(float x) { return x == x ? x : -INFINITY; }

// One CTA per row, three passes.
__global__ void __launch_bounds__(kThreads)
softmax_kernel(const float* logits, int V, long long ld, float scale, int greedy, float* probs, long long ld_p) {
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ int s_i[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const float* x = logits + blockIdx.x * ld;
    float* p = probs + blockIdx.x * ld_p;
    float m = -INFINITY;
    int at = 0x7fffffff;
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float y = no_nan(x[v]);
        if (y > m) m = y, at = v;
    }
    for (int d = 16; d > 0; d >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, d);
        const int oi = __shfl_xor_sync(0xffffffffu, at, d);
        if (om > m || (om == m && oi < at)) m = om, at = oi;
    }
    if (lane == 0) s_m[warp] = m, s_i[warp] = at;
    __syncthreads();
    for (int k = 0; k < kWarps; ++k)
        if (s_m[k] > m || (s_m[k] == m && s_i[k] < at)) m = s_m[k], at = s_i[k];
    if (greedy || m == -INFINITY) {
        for (int v = threadIdx.x; v < V; v += kThreads) p[v] = v == at ? 1.0f : 0.0f;
        return;
    }
    float l = 0.0f;
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float y = no_nan(x[v]);
        l += m == INFINITY ? (y == INFINITY ? 1.0f : 0.0f) : exp2f((y - m) * scale);
    }
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    l = 0.0f;
    for (int k = 0; k < kWarps; ++k) l += s_l[k];
    for (int v = threadIdx.x; v < V; v += kThreads) {
        const float y = no_nan(x[v]);
        p[v] = (m == INFINITY ? (y == INFINITY ? 1.0f : 0.0f) : exp2f((y - m) * scale)) / l;
    }
}

// A weight in units of 2^-60 (truncated), clamped to [0, 1]; a NaN counts as 0.
BIV_DEV float clamp01(float w) { return fminf(fmaxf(w, 0.0f), 1.0f); }
BIV_DEV unsigned long long units(float w) { return __float2ull_rz(w * 1152921504606846976.0f); }

// One CTA per request.
__global__ void __launch_bounds__(kThreads)
verify_sample_kernel(const float* __restrict__ target, const float* __restrict__ draft_probs,
                     const int32_t* __restrict__ draft, const float* __restrict__ u_accept,
                     const float* __restrict__ u_sample, const int32_t* __restrict__ p0, int K, int V,
                     int32_t* __restrict__ tokens, int32_t* __restrict__ accept_len, int32_t* __restrict__ new_len) {
    __shared__ int s_n, s_found;
    __shared__ unsigned long long s_sum[kThreads];
    __shared__ float s_f[kThreads];
    const int r = blockIdx.x, t = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (t == 0) s_n = K;
    __syncthreads();
    for (int j = t; j < K; j += kThreads) {
        const long long row = static_cast<long long>(r) * K + j;
        const int d = draft[row];
        bool ok = false;
        if (d < 0 || d >= V) {
            atomicOr(&g_sample_err, BIV_DEVERR_INDEX);
        } else {
            const float p = clamp01(target[(static_cast<long long>(r) * (K + 1) + j) * V + d]);
            const float q = draft_probs ? clamp01(draft_probs[row * V + d]) : 1.0f;
            // the product of two 24-bit numbers is exact in 64 bits
            ok = static_cast<double>(u_accept[row]) * static_cast<double>(q) < static_cast<double>(p);
        }
        if (!ok) atomicMin(&s_n, j);
    }
    __syncthreads();
    const int n = s_n;
    const float* p = target + (static_cast<long long>(r) * (K + 1) + n) * V;
    const float* q = draft_probs && n < K ? draft_probs + (static_cast<long long>(r) * K + n) * V : nullptr;
    const int skip = !draft_probs && n < K ? draft[static_cast<long long>(r) * K + n] : -1;
    const int per = (V + kThreads - 1) / kThreads, v0 = min(V, t * per), v1 = min(V, v0 + per);
    unsigned long long total = 0, before = 0;
    bool plain = false, valid = true;
    for (int round = 0; round < 2; ++round) {
        unsigned long long sum = 0;
        float f = 0.0f;
        for (int v = v0; v < v1; ++v) {
            const float w = plain ? clamp01(p[v]) : v == skip ? 0.0f : q ? clamp01(p[v] - q[v]) : clamp01(p[v]);
            sum += units(w);
            f += w;
        }
        __syncthreads();
        s_sum[t] = sum;
        s_f[t] = f;
        __syncthreads();
        total = before = 0;
        float all = 0.0f;
        for (int k = 0; k < kThreads; ++k) {
            if (k == t) before = total;
            total += s_sum[k];
            all += s_f[k];
        }
        valid = total > 0 && all < 8.0f;
        if (total > 0 || plain) break;
        plain = true;
    }
    if (t == 0) s_found = 0;
    __syncthreads();
    const float u = fminf(fmaxf(u_sample[r], 0.0f), 0.99999994f);
    const unsigned long long border = static_cast<unsigned long long>(static_cast<double>(u) * static_cast<double>(total));
    if (valid && before <= border) {
        unsigned long long sum = before;
        for (int v = v0; v < v1; ++v) {
            const float w = plain ? clamp01(p[v]) : v == skip ? 0.0f : q ? clamp01(p[v] - q[v]) : clamp01(p[v]);
            sum += units(w);
            if (sum > border) {
                s_found = v;
                break;
            }
        }
    }
    __syncthreads();
    if (!valid && t == 0) atomicOr(&g_sample_err, BIV_DEVERR_VALUE);
    for (int j = t; j <= K; j += kThreads)
        tokens[static_cast<long long>(r) * (K + 1) + j] =
            j < n ? draft[static_cast<long long>(r) * K + j] : j == n ? s_found : -1;
    if (t == 0) {
        accept_len[r] = n + 1;
        new_len[r] = p0[r] + n + 1;
    }
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
    return launch_pdl(softmax_kernel, dim3(static_cast<unsigned>(R)), dim3(kThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), logits, V, ld, scale, temperature == 0.0f ? 1 : 0,
                      probs, ld_p);
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
    return launch_pdl(verify_sample_kernel, dim3(static_cast<unsigned>(N)), dim3(kThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), target, draft_probs, draft, u_accept, u_sample, p0, K, V,
                      tokens, accept_len, new_len);
}
