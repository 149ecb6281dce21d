// bq_adapters.hip -- low-rank updates of many requests beside a shared
// projection (bq_adapters_add): out = y + gain B (A x), row by row, each
// request with its own A (rank x n) and B (rows x rank).
#include "bq_half.h"
#include "bq_layer.h"

namespace bq {

// u[t][r] = gain A[r] . x[t]: one workgroup per row, a wavefront per rank.
template <class T, class X>
__global__ __launch_bounds__(256) void adapters_down(const bq_adapters a)
{
    const int64_t t = blockIdx.x;
    const int b = request_of(a.cu, a.requests, (int)t);
    const int id = b < 0 ? -1 : a.ids[b];
    if ((unsigned)id >= (unsigned)a.count)
        return;
    const int lane = threadIdx.x & 63;
    const X *x = static_cast<const X *>(a.x) + t * a.ld_x;
    for (int r = threadIdx.x >> 6; r < a.rank; r += 4) {
        const T *w = static_cast<const T *>(a.a) + ((int64_t)id * a.rank + r) * a.n;
        float sum = 0.0f;
        for (int64_t i = 8 * lane; i < a.n; i += 512) {
            float u[8], v[8];
            load8(w + i, u);
            load8(x + i, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(u[e], v[e], sum);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            sum += __shfl_xor(sum, off, 64);
        if (lane == 0)
            static_cast<float *>(a.work)[t * a.rank + r] = sum * a.gain[id];
    }
}

// out[t][row] = y[t][row] + B[row] . u[t]: one thread per row of B.
template <class T>
__global__ __launch_bounds__(256) void adapters_up(const bq_adapters a)
{
    const int64_t t = blockIdx.x;
    const int b = request_of(a.cu, a.requests, (int)t);
    if (b < 0)
        return;
    const int id = a.ids[b];
    const int64_t row = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (row >= a.rows)
        return;
    float sum = a.y[t * a.ld_y + row];
    if ((unsigned)id < (unsigned)a.count) {
        const T *w = static_cast<const T *>(a.b) + ((int64_t)id * a.rows + row) * a.rank;
        const float *u = static_cast<const float *>(a.work) + t * a.rank;
        float add = 0.0f;
        for (int r = 0; r < a.rank; r += 8) {
            float v[8];
            load8(w + r, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                add = __builtin_fmaf(v[e], u[r + e], add);
        }
        sum += add;
    }
    a.out[t * a.ld_out + row] = sum;
}

int64_t adapters_work(const bq_adapters &a) { return a.tokens * a.rank * 4; }

hipError_t launch_adapters(const bq_adapters &a, hipStream_t st)
{
    const dim3 down((unsigned)a.tokens), up((unsigned)a.tokens, (unsigned)((a.rows + 255) / 256));
    if (a.type == BQ_F16) {
        if (a.x_type == BQ_F32)
            hipLaunchKernelGGL((adapters_down<_Float16, float>), down, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((adapters_down<_Float16, _Float16>), down, dim3(256), 0, st, a);
        hipLaunchKernelGGL((adapters_up<_Float16>), up, dim3(256), 0, st, a);
    } else {
        if (a.x_type == BQ_F32)
            hipLaunchKernelGGL((adapters_down<__bf16, float>), down, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((adapters_down<__bf16, __bf16>), down, dim3(256), 0, st, a);
        hipLaunchKernelGGL((adapters_up<__bf16>), up, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace bq
