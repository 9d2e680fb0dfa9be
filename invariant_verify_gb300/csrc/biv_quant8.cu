// Quantisation of bf16 matrices to e4m3 with a scale for 128 values of a row
// (activations) or for 128 x 128 values (weights).
#include "biv_e4m3.cuh"

namespace biv {
namespace {

constexpr int kGroup = 128;

struct QuantArgs {
    const __nv_bfloat16* x;
    uint8_t* q;
    float* scales;
    long long ld_x;
    int rows, K, groups;
};

constexpr int kRowThreads = 256;

// One scale for 128 values of a row: sixteen lanes take 8 values each (16 bytes), find the
// largest in four exchanges and write 8 bytes each, so a value is read once and written once.
// TURNS groups' loads are under way at once.  Bound by memory, and by latency below some
// 10^6 values.
template <int TURNS>
__global__ void __launch_bounds__(kRowThreads) quant_rows_kernel(const QuantArgs a) {
    const int lane = threadIdx.x & 15;
    const long long tasks = static_cast<long long>(a.rows) * a.groups;
    const long long t0 = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) / 16 * TURNS;
    pdl_wait();
    pdl_trigger();
    uint4 x[TURNS];
    int row[TURNS], g[TURNS];
    bool in[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const long long t = t0 + i;
        row[i] = static_cast<int>(t / a.groups);
        g[i] = static_cast<int>(t - static_cast<long long>(row[i]) * a.groups);
        in[i] = t < tasks && g[i] * kGroup + lane * 8 < a.K;
        x[i] = make_uint4(0, 0, 0, 0);
        if (in[i]) x[i] = __ldg(reinterpret_cast<const uint4*>(a.x + row[i] * a.ld_x + g[i] * kGroup + lane * 8));
    }
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        float m = max_of_halves(max_abs8(x[i]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float s = scale_of(m), inv = __frcp_rn(s);
        if (in[i]) *reinterpret_cast<uint2*>(a.q + static_cast<long long>(row[i]) * a.K + g[i] * kGroup + lane * 8) = e4m3x8(x[i], s, inv);
        if (lane == 0 && t0 + i < tasks) a.scales[static_cast<long long>(g[i]) * a.rows + row[i]] = s;
    }
}

constexpr int kTileThreads = 256;
constexpr int kTileLoads = kGroup * kGroup / 8 / kTileThreads;

// One scale for 128 x 128 values: a CTA holds the square in registers (8 x 16 bytes a thread)
// between the search for the largest and the writes.
__global__ void __launch_bounds__(kTileThreads) quant_squares_kernel(const QuantArgs a) {
    __shared__ float s_max[kTileThreads / 32];
    const int g = blockIdx.x % a.groups, r0 = blockIdx.x / a.groups * kGroup;
    const int col = g * kGroup + (threadIdx.x & 15) * 8;
    pdl_wait();
    pdl_trigger();
    uint4 x[kTileLoads];
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
        const int row = r0 + i * (kTileThreads / 16) + static_cast<int>(threadIdx.x / 16);
        x[i] = make_uint4(0, 0, 0, 0);
        if (row < a.rows && col < a.K) x[i] = __ldg(reinterpret_cast<const uint4*>(a.x + row * a.ld_x + col));
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) m = fmaxf(m, max_of_halves(max_abs8(x[i])));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileThreads / 32; ++i) m = fmaxf(m, s_max[i]);
    const float s = scale_of(m), inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
        const int row = r0 + i * (kTileThreads / 16) + static_cast<int>(threadIdx.x / 16);
        if (row < a.rows && col < a.K) *reinterpret_cast<uint2*>(a.q + static_cast<long long>(row) * a.K + col) = e4m3x8(x[i], s, inv);
    }
    if (threadIdx.x == 0) a.scales[blockIdx.x] = s;
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" int biv_quant_e4m3(const void* x, long long ld_x, int rows, int K, int block_rows, void* q, float* scales,
                              biv_stream_t stream) {
    BIV_TRACE_CALL();
    if (rows < 0 || K <= 0 || K % 16 != 0 || ld_x < K || ld_x % 8 != 0) return BIV_ERR_SHAPE;
    if (block_rows != 1 && block_rows != kGroup) return BIV_ERR_UNSUPPORTED;
    QuantArgs a;
    a.groups = (K + kGroup - 1) / kGroup;
    const long long blocks = (static_cast<long long>(rows) + block_rows - 1) / block_rows * a.groups;
    if (block_rows == 1 ? blocks / (kRowThreads / 16) >= 0x7fffffffLL : blocks > 0x7fffffffLL) return BIV_ERR_SHAPE;
    if (rows == 0) return BIV_OK;
    if (!x || !q || !scales) return BIV_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(scales)) return BIV_ERR_ALIGN;
    if (x == q) return BIV_ERR_VALUE;
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.q = static_cast<uint8_t*>(q);
    a.scales = scales;
    a.ld_x = ld_x;
    a.rows = rows;
    a.K = K;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (block_rows == kGroup) return launch_pdl(quant_squares_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kTileThreads), 0, s, a);
    // few groups: one each, so that all SMs work; many: four loads under way a thread
    constexpr int kPer = kRowThreads / 16;
    if (blocks <= 16LL * kPer * num_sms())
        return launch_pdl(quant_rows_kernel<1>, dim3(static_cast<unsigned>((blocks + kPer - 1) / kPer)), dim3(kRowThreads), 0, s, a);
    return launch_pdl(quant_rows_kernel<4>, dim3(static_cast<unsigned>((blocks + 4 * kPer - 1) / (4 * kPer))), dim3(kRowThreads), 0, s, a);
}
