// bq_gated.hip -- activation, gate and activation quantizer in one pass
// (bq_gated_q8).
//
// v = act(gate) * up in binary64, rounded once: a quant next to a border then
// does not hang on the last bits of an f32 exp.  Before that rounding v is off by less
// than 2^-50 of itself: 2^-52 from the table, 2^-53 from each of the series, its product
// with the table, the sum, the quotient and the product with up.  GELU's argument 2 z has
// six roundings more, 2^-53 each, which move exp by 2 |z| times as much.  Eight values a lane, a block of
// qa in qa / 8 neighbouring lanes, quantized as the norm does (bq_quant8.h).
//
// Measured: 4099 x 12288 bf16 with the values kept (359 MB) 121 us, 3.0 TB/s: about 30
// operations of binary64 a value beside the memory's 76 us at the rate of a copy (the
// next piece's loads under way meanwhile: 126).  16 x 12288 f32 4.4 us, latency.
#include "bq_half.h"
#include "bq_model.h"
#include "bq_quant8.h"

namespace bq {

constexpr int kGatedThreads = 256;

// exp(x) for |x| of any size: 2^(n / 32) with n the nearest integer to 32 x log2(e), the rest (at most ln 2 / 64) by its
// series (the first term left out is below 2^-56), 2^(n % 32 / 32) from a table in LDS; n is held to where the result is
// past every f32 that could matter (x of +-1500: 1 + exp is 1 or infinite against any product of two f32).
__device__ __forceinline__ double exp_of(const double *table, double x)
{
    const double y = fmin(fmax(x, -1500.0), 1500.0) * (32.0 * 1.44269504088896340736), n = __builtin_rint(y);
    // ln 2 / 32 in two parts, the first with zeros at its end: n times it is exact
    const double f = __builtin_fma(n, -1.0 * 0x1.62e42fefa0000p-6, fmin(fmax(x, -1500.0), 1500.0)) - n * 0x1.cf79abc9e3b3ap-45;
    double p = 1.0 / 720.0;
    p = __builtin_fma(p, f, 1.0 / 120.0);
    p = __builtin_fma(p, f, 1.0 / 24.0);
    p = __builtin_fma(p, f, 1.0 / 6.0);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    const int i = (int)n;
    return __builtin_ldexp(p * table[i & 31], i >> 5);
}
// x / d for d >= 1 (or infinite) to the last bit but one: the reciprocal's 2^-23 or better, squared twice.
__device__ __forceinline__ double over(double x, double d)
{
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    const double q = x * r;
    return __builtin_copysign(d > 1e300 ? 0.0 : __builtin_fma(__builtin_fma(-d, q, x), r, q), x);  // -0 stays so
}

template <int ACT>
__device__ __forceinline__ double activate(const double *table, double x)
{
    if constexpr (ACT == BQ_SILU)
        return over(x, 1.0 + exp_of(table, -x));
    else if constexpr (ACT == BQ_GELU)  // 1.5957691216 = 2 sqrt(2 / pi)
        return over(x, 1.0 + exp_of(table, -1.5957691216057307117 * __builtin_fma(0.044715 * x * x, x, x)));
    else if constexpr (ACT == BQ_RELU2)
        return x > 0.0 ? x * x : 0.0;
    else
        return x;
}

template <class T, int ACT>
__global__ __launch_bounds__(kGatedThreads) void gated_kernel(const bq_gated a)
{
    __shared__ double table[32];  // 2^(i / 32)
    if (ACT == BQ_SILU || ACT == BQ_GELU) {
        if (threadIdx.x < 32)
            table[threadIdx.x] = exp2((double)threadIdx.x / 32.0);
        __syncthreads();
    }
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
                v[e] = (float)(activate<ACT>(table, (double)g[e]) * (double)u[e]);
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
    const int64_t blocks = (a.tokens * (a.n / 8) + kGatedThreads - 1) / kGatedThreads, most = 2048;
    // eight workgroups a compute unit, which walk on: the table once for many pieces
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    switch (a.type) {
    case BQ_F16: gated_type<_Float16>(a, grid, st); break;
    case BQ_BF16: gated_type<__bf16>(a, grid, st); break;
    default: gated_type<float>(a, grid, st); break;
    }
    return hipGetLastError();
}

}  // namespace bq
