// bq_norm.hip -- residual addition, root-mean-square norm and activation
// quantizer in one pass over a row (bq_rmsnorm_q8).
//
// h = round(x + res); r = fl32(1 / sqrt(sum(h^2) / n + eps)); v = fl(fl(h r) w);
// d = max|v| * fl32(1 / 127) and q = half-away(v / d) per block of qa.  The sum runs in
// binary64 (the squares of f32 values are exact there), so r does not depend
// on the order of the sum and q, d are reproducible bit for bit; at 2 f64
// operations per value they are nowhere near a bound.  What bounds it is
// memory: x, res in; h, q, d (y) out, every value touched once -- a row stays
// in registers between the sum and the quantizer.
//
// Measured: 4099 rows of 4096 bf16 (153 MB with res and h) 31.6 us, 4.8 TB/s,
// the rate of a large copy; one row of f32 3.6 us, two waits for memory and
// the launch.
#include "bq_device.h"
#include "bq_half.h"
#include "bq_layer.h"

namespace bq {

// One workgroup per row; a thread holds R pieces of 8 consecutive values
// (16-byte loads), piece c at 8 (c blockDim + thread).  A block of qa values
// is qa / 8 neighbouring lanes.
template <class T, int R>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a)
{
    __shared__ double sums[16];
    const int64_t row = a.row0 + blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    const T *w = static_cast<const T *>(a.w);
    float v[R][8];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < R; ++c) {
        const int i = 8 * (c * (int)blockDim.x + (int)threadIdx.x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[c][e] = 0.0f;
        if (i < a.n) {
            load8(x + i, v[c]);
            if (a.res) {
                float g[8];
                load8(static_cast<const T *>(a.res) + row * a.ld_res + i, g);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[c][e] = (float)(T)(v[c][e] + g[e]);
            }
            if (a.h)
                store8(static_cast<T *>(a.h) + row * a.ld_h + i, v[c]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum = __builtin_fma((double)v[c][e], (double)v[c][e], sum);
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0)
        sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int k = 0; k < (int)(blockDim.x >> 6); ++k)
        sum += sums[k];
    const float r = (float)(1.0 / __builtin_sqrt(sum / (double)a.n + a.eps));
#pragma unroll
    for (int c = 0; c < R; ++c) {
        const int i = 8 * (c * (int)blockDim.x + (int)threadIdx.x);
        float m = 0.0f;
        if (i < a.n) {
            float g[8];
            load8(w + i, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[c][e] = (v[c][e] * r) * g[e];
                m = fmaxf(m, fabsf(v[c][e]));
            }
        }
        // n and the piece of a wavefront's lanes are multiples of a block: its lanes are all in or all out
        m = fmaxf(m, __shfl_xor(m, 1, 64));
        m = fmaxf(m, __shfl_xor(m, 2, 64));
        if (a.qa > 32)
            m = fmaxf(m, __shfl_xor(m, 4, 64));
        if (a.qa > 64)
            m = fmaxf(m, __shfl_xor(m, 8, 64));
        if (i >= a.n)
            continue;
        float db = m * (1.0f / 127.0f), q[8];
        // the product is rounded to f32 before it is narrowed: seen together, the two become one
        // instruction that rounds once (another f16 scale for one block in about 2^14)
        asm("" : "+v"(db));
        if (a.f16_scale)
            db = (float)(_Float16)db;
        if (a.f16_scale && db < 0x1p-14f) {
            // a subnormal f16 scale is coarser than 1/127 of the maximum: the clamp can bind
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[e] = (float)quant_of(v[c][e], db);
        } else {
            quant_block<8>(v[c], db, q);
        }
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo |= (uint32_t)((int)q[e] & 0xFF) << (8 * e);
            hi |= (uint32_t)((int)q[4 + e] & 0xFF) << (8 * e);
        }
        uint2 *qp = reinterpret_cast<uint2 *>(a.q + row * a.ld_q + i);
        *qp = make_uint2(lo, hi);
        if (i % a.qa == 0)
            a.d[row * a.ld_d + i / a.qa] = db;
        if (a.y)
            store8(static_cast<T *>(a.y) + row * a.ld_y + i, v[c]);
    }
}

template <class T>
static void norm_type(const NormArgs &a, int64_t rows, hipStream_t st)
{
    // few rows: one piece a thread, for latency; many: two, for loads in flight
    const int pieces = (a.n + 7) / 8;
    int R = rows >= 512 ? 2 : 1;
    while (R * 1024 < pieces)
        R *= 2;
    const int threads = ((pieces + R - 1) / R + 63) / 64 * 64;
    const dim3 grid((unsigned)rows), block((unsigned)threads);
    switch (R) {
    case 1: hipLaunchKernelGGL((norm_kernel<T, 1>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((norm_kernel<T, 2>), grid, block, 0, st, a); break;
    case 4: hipLaunchKernelGGL((norm_kernel<T, 4>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((norm_kernel<T, 8>), grid, block, 0, st, a); break;
    }
}

hipError_t launch_norm(int type, NormArgs a, int64_t rows, hipStream_t st)
{
    // a grid holds fewer than 2^32 threads: at most 2^21 rows of up to 1024 a launch
    const int64_t most = int64_t(1) << 21;
    for (a.row0 = 0; a.row0 < rows; a.row0 += most) {
        const int64_t n = rows - a.row0 < most ? rows - a.row0 : most;
        switch (type) {
        case BQ_F16: norm_type<_Float16>(a, n, st); break;
        case BQ_BF16: norm_type<__bf16>(a, n, st); break;
        default: norm_type<float>(a, n, st); break;
        }
    }
    return hipGetLastError();
}

}  // namespace bq
