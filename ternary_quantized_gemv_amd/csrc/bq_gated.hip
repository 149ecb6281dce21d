// bq_gated.hip -- activation, gate and activation quantizer in one pass
// (bq_gated_q8).
//
// v = act(gate) * up in binary64, rounded once: a quant next to a border then
// does not hang on the last bits of an f32 exp.  Eight values a lane, a block of
// qa in qa / 8 neighbouring lanes, quantized as the norm does (bq_quant8.h).
#include "bq_half.h"
#include "bq_model.h"
#include "bq_quant8.h"

namespace bq {

constexpr int kGatedThreads = 256;

template <int ACT>
__device__ __forceinline__ double activate(double x)
{
    if constexpr (ACT == BQ_SILU)
        return x / (1.0 + exp(-x));
    else if constexpr (ACT == BQ_GELU)  // 1.5957691216 = 2 sqrt(2 / pi)
        return x / (1.0 + exp(-1.5957691216057307117 * __builtin_fma(0.044715 * x * x, x, x)));
    else if constexpr (ACT == BQ_RELU2)
        return x > 0.0 ? x * x : 0.0;
    else
        return x;
}

template <class T, int ACT>
__global__ __launch_bounds__(kGatedThreads) void gated_kernel(const bq_gated a)
{
    const int per_row = (int)(a.n / 8);
    const int64_t total = a.tokens * per_row;
    const int log2 = __builtin_ctz((unsigned)a.qa);
    for (int64_t first = (int64_t)blockIdx.x * kGatedThreads; first < total; first += (int64_t)gridDim.x * kGatedThreads) {
        // the division by the row length once a workgroup in 64 bits, then in 32
        const int64_t t0 = first / per_row;
        const uint32_t off = (uint32_t)(first - t0 * per_row) + threadIdx.x;
        const int64_t t = t0 + off / (uint32_t)per_row;
        const int i = 8 * (int)(off % (uint32_t)per_row);
        // rows hold whole blocks, and a workgroup starts with one: a block's lanes are all in or all out
        const bool live = t < a.tokens;
        float v[8] = {}, m = 0.0f;
        if (live) {
            float g[8], u[8];
            load8(static_cast<const T *>(a.gate) + t * a.ld_gate + i, g);
            load8(static_cast<const T *>(a.up) + t * a.ld_up + i, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = (float)(activate<ACT>((double)g[e]) * (double)u[e]);
                m = fmaxf(m, fabsf(v[e]));
            }
        }
        m = block_max(m, a.qa);
        if (!live)
            return;
        quantize8(v, m, a.f16_scale, a.q + t * a.ld_q + i, (i & (a.qa - 1)) == 0 ? a.d + t * a.ld_d + (i >> log2) : nullptr);
        if (a.y)
            store8(static_cast<T *>(a.y) + t * a.ld_y + i, v);
    }
}

template <class T>
static void gated_type(const bq_gated &a, dim3 grid, hipStream_t st)
{
    const dim3 block(kGatedThreads);
    switch (a.act) {
    case BQ_SILU: hipLaunchKernelGGL((gated_kernel<T, BQ_SILU>), grid, block, 0, st, a); break;
    case BQ_GELU: hipLaunchKernelGGL((gated_kernel<T, BQ_GELU>), grid, block, 0, st, a); break;
    case BQ_RELU2: hipLaunchKernelGGL((gated_kernel<T, BQ_RELU2>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((gated_kernel<T, BQ_NONE>), grid, block, 0, st, a); break;
    }
}

hipError_t launch_gated(const bq_gated &a, hipStream_t st)
{
    // a grid holds fewer than 2^32 threads; workgroups walk on from there
    const int64_t blocks = (a.tokens * (a.n / 8) + kGatedThreads - 1) / kGatedThreads, most = int64_t(1) << 22;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    switch (a.type) {
    case BQ_F16: gated_type<_Float16>(a, grid, st); break;
    case BQ_BF16: gated_type<__bf16>(a, grid, st); break;
    default: gated_type<float>(a, grid, st); break;
    }
    return hipGetLastError();
}

}  // namespace bq
