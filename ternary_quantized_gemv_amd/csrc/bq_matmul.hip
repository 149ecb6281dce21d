// bq_matmul.hip -- a packed matrix times the activations of few tokens (bq_matmul).
//
// A workgroup makes 32 tokens x 32 rows; its wavefronts take every kFewWaves-th
// step of k and add their f32 sums through LDS, in their order.  Each wavefront
// lays its tokens' quants out by itself (bq_matmul.h).
#include "bq_matmul.h"

namespace bq {

constexpr int kFewWaves = 8;

template <int FMT, int QA, class T>
__global__ __launch_bounds__(64 * kFewWaves) void matmul_few(const bq_product a)
{
    typedef Shape<FMT, QA> P;
    __shared__ float part[kFewWaves][16][64];
    __shared__ __attribute__((aligned(16))) float d1s[kFewWaves][P::NG][32];
    __shared__ __attribute__((aligned(16))) int starts[kFewWaves][P::NG][32];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, in32 = lane & 31;
    const int64_t K = a.w.cols, nb = K / P::BL, ng = (nb + 7) / 8, tokens = a.a.ncols, rows = a.w.rows;
    const int64_t row_tiles = (rows + 31) / 32, items = row_tiles * ((tokens + 31) / 32);
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t t0 = item / row_tiles * 32, r0 = item % row_tiles * 32;
        const int64_t t = t0 + in32 < tokens ? t0 + in32 : tokens - 1;
        const int8_t *q = a.a.q + t * a.a.ld_q;
        const float *d1 = a.a.d + t * a.a.ld_d;
        const int64_t tile = r0 / kTileRows, row = r0 % kTileRows + in32;
        const u32x4 *bits = static_cast<const u32x4 *>(a.w.bits) + tile_block0(FMT, tile, nb) * kTileRows + row;
        const uint16_t *scales = a.w.scales + (tile * ng * kTileRows + row) * 8;
        f32x16 acc;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[i] = 0.0f;
        for (int64_t k = (int64_t)wave * kStepK; k < K; k += kFewWaves * kStepK) {
            u32x4 w[P::BLOCKS];
            float d0[P::BLOCKS];
#pragma unroll
            for (int j = 0; j < P::BLOCKS; ++j) {
                const int64_t b = clamp_block<FMT>(k / P::BL + j, nb);
                w[j] = bits[b * kTileRows];
                d0[j] = f16_bits_to_f32(scales[b / 8 * kTileRows * 8 + b % 8]);
            }
            const int valid = K - k < kStepK ? (int)(K - k) : kStepK;
            u32x4 f[4];
            act_operands<FMT, QA>(q + k, half, valid, f);
#pragma unroll
            for (int g = 0; g < P::NG; ++g) {
                int s = 0;
#pragma unroll
                for (int m = g * P::GM; m < (g + 1) * P::GM; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s = __builtin_amdgcn_sdot4((int)f[m][e], 0x01010101, s, false);
                s += __shfl_xor(s, 32, 64);
                // both halves write the same
                d1s[wave][g][in32] = g * P::G < valid ? d1[(k + g * P::G) / QA] : 0.0f;
                starts[wave][g][in32] = kMagic - s;
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int g = 0; g < P::NG; ++g) {
                i32x16 s;
                f32x16 d;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const i32x4 c = *reinterpret_cast<const i32x4 *>(&starts[wave][g][8 * j + 4 * half]);
                    const f32x4 e = *reinterpret_cast<const f32x4 *>(&d1s[wave][g][8 * j + 4 * half]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[4 * j + x] = c[x];
                        d[4 * j + x] = e[x];
                    }
                }
#pragma unroll
                for (int m = g * P::GM; m < (g + 1) * P::GM; ++m) {
                    i32x4 b;
                    weight_operand<FMT, QA>(w, half, m, b);
                    s = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, f[m]), b, s, 0, 0, 0);
                }
                const float dw = d0[g * P::G / P::BL], off = -kMagicF * dw;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[i] = __builtin_fmaf(__builtin_fmaf(as_float(s[i]), dw, off), d[i], acc[i]);
            }
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            part[wave][i][lane] = acc[i];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16 / kFewWaves; ++j) {
            const int i = wave + j * kFewWaves;
            float y = part[0][i][lane];
#pragma unroll
            for (int x = 1; x < kFewWaves; ++x)
                y += part[x][i][lane];
            const int64_t ty = t0 + 8 * (i / 4) + 4 * half + i % 4, r = r0 + in32;
            if (ty < tokens && r < rows)
                finish<T>(a, y, ty, r);
        }
        __syncthreads();
    }
}

template <int FMT, int QA>
static void few_type(const bq_product &a, hipStream_t st)
{
    const int64_t items = (a.w.rows + 31) / 32 * ((a.a.ncols + 31) / 32), most = int64_t(1) << 22;
    const dim3 grid((unsigned)(items < most ? items : most)), block(64 * kFewWaves);
    switch (a.type) {
    case BQ_F16: hipLaunchKernelGGL((matmul_few<FMT, QA, _Float16>), grid, block, 0, st, a); break;
    case BQ_BF16: hipLaunchKernelGGL((matmul_few<FMT, QA, __bf16>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((matmul_few<FMT, QA, float>), grid, block, 0, st, a); break;
    }
}

template <int FMT>
static void few_qa(const bq_product &a, hipStream_t st)
{
    switch (a.a.qa) {
    case 32: few_type<FMT, 32>(a, st); break;
    case 64: few_type<FMT, 64>(a, st); break;
    default: few_type<FMT, 128>(a, st); break;
    }
}

int64_t matmul_work(const bq_product &) { return 0; }

hipError_t launch_matmul(const bq_product &a, hipStream_t st)
{
    if (a.w.fmt == BQ_Q1_0)
        few_qa<BQ_Q1_0>(a, st);
    else
        few_qa<BQ_Q2_0>(a, st);
    return hipGetLastError();
}

}  // namespace bq
