// Quantisation of bf16 matrices to e4m3 with a scale for 128 values of a row
// (activations) or for 128 x 128 values (weights).
#include <algorithm>

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
    int chunks, shift;                 // rows' form: a CTA takes 2^shift groups of a row, and there are `chunks` such
};

constexpr int kRowThreads = 256;

// One scale for 128 values of a row: sixteen lanes take 8 values each (16 bytes), find the
// largest in four exchanges and write 8 bytes each, so a value is read once and written once.
// Sixteen lanes take TURNS rows of a group, whose loads are under way at once and whose scales
// lie side by side.  Bound by memory (8192 x 4096: 19.9 us, 5.1 TB/s; with a row's neighbouring groups
// instead of a group's rows 25.0, for scales written four bytes here and there), and by latency
// below some 10^6 values (64 x 4096: 2.5 us with its launch).
template <int TURNS>
__global__ void __launch_bounds__(kRowThreads) quant_rows_kernel(const QuantArgs a) {
    const int lane = threadIdx.x & 15, part = threadIdx.x / 16;
    const int chunk = static_cast<int>(blockIdx.x % a.chunks);
    const int g = (chunk << a.shift) + (part & ((1 << a.shift) - 1)), col = g * kGroup + lane * 8;
    const long long r0 = (static_cast<long long>(blockIdx.x / a.chunks) * (kRowThreads / 16 >> a.shift) + (part >> a.shift)) * TURNS;
    const int n = g < a.groups ? static_cast<int>(min(static_cast<long long>(TURNS), a.rows - r0)) : 0;
    const bool in = col < a.K;
    pdl_wait();
    pdl_trigger();
    uint4 x[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (i < n && in) x[i] = __ldg(reinterpret_cast<const uint4*>(a.x + (r0 + i) * a.ld_x + col));
    }
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        float m = max_of_halves(max_abs8(x[i]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float s = scale_of(m), inv = __frcp_rn(s);
        if (i < n && in) *reinterpret_cast<uint2*>(a.q + (r0 + i) * a.K + col) = e4m3x8(x[i], s, inv);
        if (lane == i) mine = s;
    }
    if (lane < n) a.scales[static_cast<long long>(g) * a.rows + r0 + lane] = mine;
}

constexpr int kTileThreads = 256;
constexpr int kTileLoads = kGroup * kGroup / 8 / kTileThreads;

// One scale for 128 x 128 values: a CTA holds the square in registers (8 x 16 bytes a thread)
// between the search for the largest and the writes.  Bound by memory: 28672 x 4096 in 54 us, 6.5 TB/s.
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
    QuantArgs a = {};
    a.groups = (K - 1) / kGroup + 1;               // no sum that passes 31 bits
    const long long blocks = (static_cast<long long>(rows) + block_rows - 1) / block_rows * a.groups;
    if (blocks > (block_rows == 1 ? 0x7fffffffLL * (kRowThreads / 16) / 2 : 0x7fffffffLL)) return BIV_ERR_SHAPE;
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
    // rows: as many groups side by side as a row has, up to a CTA's sixteen
    constexpr int kPer = kRowThreads / 16;
    while ((1 << a.shift) < std::min(a.groups, kPer)) ++a.shift;
    a.chunks = (a.groups + (1 << a.shift) - 1) >> a.shift;
    auto ctas = [&](int turns) {
        const long long per = static_cast<long long>(kPer >> a.shift) * turns;
        return (rows + per - 1) / per * a.chunks;
    };
    // few groups: one each, so that all SMs work (8 x 4096: 1.2 us, four rows each 1.9; 1024 x 4096: 4.4, 5.0); many:
    // four loads under way a thread (2048 x 4096: 6.9 us, one each 7.8; 8192 x 4096: 19.9, 26.0; two 21.6, eight 21.5)
    if (blocks <= 16LL * kPer * num_sms())
        return launch_pdl(quant_rows_kernel<1>, dim3(static_cast<unsigned>(ctas(1))), dim3(kRowThreads), 0, s, a);
    return launch_pdl(quant_rows_kernel<4>, dim3(static_cast<unsigned>(ctas(4))), dim3(kRowThreads), 0, s, a);
}
