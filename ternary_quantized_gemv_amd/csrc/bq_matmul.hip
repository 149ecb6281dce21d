// bq_matmul.hip -- a packed matrix times the activations of many tokens (bq_matmul): the
// choice of the kernel, the layout of the activations, and the kernel for few tokens or
// rows.
//
// matmul_split makes 32 tokens x 32 rows a workgroup; its wavefronts take every
// kSplitWaves-th step of k and add their f32 sums through LDS, in their order.  Each lays
// its tokens' quants out by itself: one launch.  (Operands laid out by matmul_lay and read
// from memory: 13.4 us instead of 8.9 at 64 tokens, 14.5 and 14.4 at 128.)
#include "bq_matmul.h"

namespace bq {

constexpr int kSplitWaves = 8, kLayThreads = 256;

template <int FMT, int QA>
__global__ __launch_bounds__(kLayThreads) void matmul_lay(const MatmulArgs g)
{
    typedef Shape<FMT, QA> P;
    const bq_product &a = g.p;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, in32 = lane & 31;
    const int64_t items = ((int64_t)a.a.ncols + kTileTokens - 1) / kTileTokens * g.steps;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t k = item % g.steps * kStepK, t = item / g.steps * kTileTokens + 32 * wave + in32;
        const bool live = t < a.a.ncols;
        const int64_t row = live ? t : a.a.ncols - 1;
        const int valid = !live ? 0 : a.w.cols - k < kStepK ? (int)(a.w.cols - k) : kStepK;
        u32x4 f[4];
        act_operands<FMT, QA>(a.a.q + row * a.a.ld_q + k, half, valid, f);
        char *stage = static_cast<char *>(a.work) + item * Stage<FMT, QA>::BYTES;
        u32x4 *to = reinterpret_cast<u32x4 *>(stage) + wave * 256 + lane;
#pragma unroll
        for (int m = 0; m < 4; ++m)
            to[64 * m] = f[m];
        float *scales = reinterpret_cast<float *>(stage + Stage<FMT, QA>::QUANTS) + 32 * wave + in32;
#pragma unroll
        for (int j = 0; j < P::NG; ++j) {
            const int start = kMagic - quant_sum<P::GM>(f + j * P::GM);
            if (half == 0)
                scales[256 * j] = j * P::G < valid ? a.a.d[row * a.a.ld_d + (k + j * P::G) / QA] : 0.0f;
            else
                scales[256 * j + 128] = as_float(start);
        }
    }
}

template <int FMT, int QA>
__global__ __launch_bounds__(64 * kSplitWaves) void matmul_split(const MatmulArgs g)
{
    typedef Shape<FMT, QA> P;
    __shared__ float part[kSplitWaves][16][64];
    __shared__ __attribute__((aligned(16))) float own[kSplitWaves][2][P::NG][32];  // scales, starts
    const bq_product &a = g.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, in32 = lane & 31;
    const int64_t tokens = a.a.ncols, rows = a.w.rows, items = g.row_tiles * g.token_tiles;
    const int nb = (int)(a.w.cols / P::BL);
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t t0 = item / g.row_tiles * 32, r0 = item % g.row_tiles * 32, tile = r0 / kTileRows;
        const TileOf planes = tile_of<FMT>(a.w, tile, nb);
        const int row0 = (int)(r0 % kTileRows);
        const int64_t t = t0 + in32 < tokens ? t0 + in32 : tokens - 1;
        const int8_t *q = a.a.q + t * a.a.ld_q;
        const float *d1 = a.a.d + t * a.a.ld_d;
        f32x16 acc;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[i] = 0.0f;
        for (int step = wave; step < g.steps; step += kSplitWaves) {
            uint32_t w[Words<FMT, QA>::N];
            uint16_t d0[P::BLOCKS];
            load_weights<FMT, QA>(planes, row0, 16 * in32 + 8 * half, step * P::BLOCKS, nb, w, d0);
            const int64_t k = (int64_t)step * kStepK;
            const int valid = a.w.cols - k < kStepK ? (int)(a.w.cols - k) : kStepK;
            u32x4 f[4];
            act_operands<FMT, QA>(q + k, half, valid, f);
#pragma unroll
            for (int j = 0; j < P::NG; ++j) {
                // both halves write the same
                own[wave][0][j][in32] = j * P::G < valid ? d1[(k + j * P::G) / QA] : 0.0f;
                own[wave][1][j][in32] = as_float(kMagic - quant_sum<P::GM>(f + j * P::GM));
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            i32x4 b[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                b[x] = weight_operand<FMT, QA>(w, half, x);
#pragma unroll
            for (int j = 0; j < P::NG; ++j) {
                const float *scales = &own[wave][0][j][4 * half], *starts = &own[wave][1][j][4 * half];
                i32x16 s;
                f32x16 d;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const i32x4 c = *reinterpret_cast<const i32x4 *>(starts + 8 * x);
                    const f32x4 e = *reinterpret_cast<const f32x4 *>(scales + 8 * x);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        s[4 * x + y] = c[y];
                        d[4 * x + y] = e[y];
                    }
                }
#pragma unroll
                for (int x = j * P::GM; x < (j + 1) * P::GM; ++x)
                    s = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, f[x]), b[x], s, 0, 0, 0);
                float dw = f16_bits_to_f32(d0[j * P::G / P::BL]);
                asm("" : "+v"(dw));  // widened once, not in every fma
                const float off = -kMagicF * dw;
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
        constexpr int MINE = 16 / kSplitWaves;
        float y[MINE];
        int64_t ty[MINE];
        bool live[MINE];
#pragma unroll
        for (int j = 0; j < MINE; ++j) {
            const int i = wave + j * kSplitWaves;
            y[j] = part[0][i][lane];
#pragma unroll
            for (int x = 1; x < kSplitWaves; ++x)
                y[j] += part[x][i][lane];
            const int64_t at = t0 + 8 * (i / 4) + 4 * half + i % 4;
            live[j] = at < tokens;
            ty[j] = live[j] ? at : tokens - 1;
        }
        if (r0 + in32 < rows)
            finish<MINE>(a, y, ty, live, r0 + in32);
        __syncthreads();
    }
}

static int64_t up(int64_t x, int64_t n) { return (x + n - 1) / n; }
static dim3 grid_of(int64_t items)
{
    const int64_t most = int64_t(1) << 22;  // a grid holds fewer than 2^32 threads; workgroups walk on from there
    return dim3((unsigned)(items < most ? items : most));
}

template <int FMT, int QA>
static void lay_kind(const MatmulArgs &g, hipStream_t st)
{
    hipLaunchKernelGGL((matmul_lay<FMT, QA>), grid_of(up(g.p.a.ncols, kTileTokens) * g.steps), dim3(kLayThreads), 0, st, g);
}

template <int FMT, int QA>
static void split_kind(const MatmulArgs &g, hipStream_t st)
{
    hipLaunchKernelGGL((matmul_split<FMT, QA>), grid_of(g.token_tiles * g.row_tiles), dim3(64 * kSplitWaves), 0, st, g);
}

static hipError_t launch_matmul_split(MatmulArgs g, hipStream_t st)
{
    g.token_tiles = up(g.p.a.ncols, 32);
    g.row_tiles = up(g.p.w.rows, 32);
    const int qa = g.p.a.qa;
    if (g.p.w.fmt == BQ_Q1_0)
        qa == 32 ? split_kind<BQ_Q1_0, 32>(g, st) : qa == 64 ? split_kind<BQ_Q1_0, 64>(g, st) : split_kind<BQ_Q1_0, 128>(g, st);
    else
        qa == 32 ? split_kind<BQ_Q2_0, 32>(g, st) : qa == 64 ? split_kind<BQ_Q2_0, 64>(g, st) : split_kind<BQ_Q2_0, 128>(g, st);
    return hipGetLastError();
}

// Which kernel: 0, matmul_split; 32 or 64, matmul_tiles with so many tokens a workgroup
// (32: two groups of four wavefronts, each every other step), behind matmul_lay.
// Measured (us; 4096 x 4096 in Q1_0 / 128 unless noted; split, 32, 64):
//   24 tokens    7.7   23    39        512 tokens    45   27   45
//   64           8.9   23    41       1024           85   40   49
//   128         14.4   25    41       2048          166   66   64
//   256         25     25    42       4096          328  132  118
//   Q2_0: 256 tokens 32, 33, 65; 96 tokens of 12288 rows 39, 32, 61; 4096 tokens of 12288 columns 1261, 590, 378
//   Q1_0 in groups of 32: 256 tokens 51, 37, 76; 1000 tokens of 5000 rows 236, 99, 87
//   151936 rows: 17 tokens 78, 52, 85 (Q2_0 118, 89, 121); 32 tokens 104, 51, 82 (141, 91, 122); 48 tokens 164, 74, 84
//   (241, 144, 123)
//   20000 tokens: 40 rows 36, 74, 76 (Q2_0 42, 110, 98); 128 rows 58, 74, 77 (74, 112, 99); 200 rows 100, 74, 78
//   (127, 112, 100).  100000 tokens of 256 columns in groups of 32, Q2_0: 40 rows 44, 98, 64; 128 rows 83, 99, 65
// A tile kernel needs its workgroups to fill the 256 compute units: below 128 of 32 tokens (1024 of the split kernel's)
// the split kernel, whose wavefronts share out the steps, is faster; it lays the tokens out anew for every 32 rows,
// which costs more with short groups.  So it is with up to 64 rows, where three of a tile's four wavefronts would work
// for nothing.
// 64 tokens decode the weights half as often, and pay from a second workgroup a compute unit on; not with 32 tokens or
// fewer, which are one tile either way, half of it empty.
static int kernel_for(const bq_product &a)
{
    const int64_t t = a.a.ncols, r = a.w.rows;
    if (r <= kTileRows || up(t, 32) * up(r, 32) <= (a.a.qa < block_len(a.w.fmt) ? 640 : 1024))
        return 0;
    return t <= 32 || up(t, 64) * up(r, kTileOut) <= 256 ? 32 : 64;
}

int64_t matmul_work(const bq_product &a)
{
    if (kernel_for(a) == 0)
        return 0;
    const int group = a.a.qa < block_len(a.w.fmt) ? a.a.qa : block_len(a.w.fmt);
    return up(a.a.ncols, kTileTokens) * up(a.w.cols, kStepK) * (kTileTokens * kStepK + kStepK / group * 1024);
}

hipError_t launch_matmul(const bq_product &a, hipStream_t st)
{
    const int kernel = kernel_for(a);
    MatmulArgs g;
    g.p = a;
    g.steps = (int)up(a.w.cols, kStepK);
    if (kernel == 0)
        return launch_matmul_split(g, st);
    if (a.w.fmt == BQ_Q1_0)
        a.a.qa == 32 ? lay_kind<BQ_Q1_0, 32>(g, st) : a.a.qa == 64 ? lay_kind<BQ_Q1_0, 64>(g, st) : lay_kind<BQ_Q1_0, 128>(g, st);
    else
        a.a.qa == 32 ? lay_kind<BQ_Q2_0, 32>(g, st) : a.a.qa == 64 ? lay_kind<BQ_Q2_0, 64>(g, st) : lay_kind<BQ_Q2_0, 128>(g, st);
    return launch_matmul_tiles(g, kernel, st);
}

}  // namespace bq
