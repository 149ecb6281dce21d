// bq_matmul_tiles.hip -- a packed matrix times the activations of many tokens
// (bq_matmul).
//
// matmul_tiles makes 32 M tokens x 256 rows a workgroup: four wavefronts of 64 rows,
// whose weights each decodes for itself (two operations per four weights), all on the
// same stage of laid-out activations (bq_matmul.h), copied to LDS as it lies, two steps
// ahead.  KG groups of four wavefronts take every KG-th step, for few tiles.
//
// What bounds it: 32 tokens x 32 rows x 128 k are four matrix instructions of 32 cycles
// and 32 scaling fma (Q2_0: 64).  The counters at 4096 x 4096 x 4096 in Q1_0 say 63 vector
// and matrix instructions for each such unit (16 decode the weights, the others are
// addresses and the outputs) and 467 cycles of a SIMD (239 K for 512 units): its vector
// unit is busy for 54% of them, its matrix cores for 27%, mostly in turn (two wavefronts a
// SIMD, a matrix instruction keeps the vector unit for about 15 of its 32 cycles: measured
// with both in a loop); the rest is waiting.  118 us (1170 TFLOP/s of the matrix cores'
// 5000), of which 9 are the layout and about 24 the outputs (67 MB at 2.8 TB/s); 12288
// columns in Q2_0 380 us (1085).  128 tokens a workgroup spill registers (114 and 380 us),
// as do three wavefronts a SIMD (122 and 840); outputs from the products' own places, 128
// bytes a token, took 47 us instead of 30; orders of the instructions by hand, priorities
// around the matrix instructions and starting values kept in registers changed nothing.
#include "bq_matmul.h"

namespace bq {

typedef __attribute__((address_space(3))) char *lptr;

template <int FMT, int QA, int M, int KG>
__global__ __launch_bounds__(256 * KG, 2) void matmul_tiles(const MatmulArgs g)
{
    typedef Shape<FMT, QA> P;
    typedef Stage<FMT, QA> S;
    // of a stage: M 4 KiB of operands, then for every group 32 M scales and 32 M starts
    constexpr int QUANTS = M * 4096, BYTES = QUANTS + P::NG * 256 * M, TOKENS = 32 * M;
    constexpr int PIECES = P::NG * M, LOADS = PIECES >= 4 ? PIECES / 4 : 1;  // of 256 bytes, scales and starts; a wavefront
    __shared__ __attribute__((aligned(16))) char lds[3 * KG * BYTES > 32768 ? 3 * KG * BYTES : 32768];
    const bq_product &a = g.p;
    const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);  // of KG groups of wavefronts: every KG-th step
    char *const mine = lds + kg * 3 * BYTES;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3, half = lane >> 5, in32 = lane & 31;
    const int nb = (int)(a.w.cols / P::BL), steps = (int)g.steps;
    // workgroups go to the eight XCDs in turn, each with an L2 of its own: an XCD takes a run of tiles, eight token
    // tiles by as many row tiles as come, so that the 64 it has at a time share 8 stages and 8 tiles of weights
    const int64_t items = g.token_tiles * g.row_tiles, run = (items + 7) / 8;
    for (int64_t slot = blockIdx.x; slot < 8 * run; slot += gridDim.x) {
        const int64_t item = slot % 8 * run + slot / 8;
        if (item >= items)
            continue;
        const int64_t band = item / (8 * g.row_tiles), in_band = item % (8 * g.row_tiles);
        const int wide = g.token_tiles - 8 * band < 8 ? (int)(g.token_tiles - 8 * band) : 8;
        const int64_t tt = 8 * band + in_band % wide, rt = in_band / wide;
        const int64_t t0 = tt * TOKENS;
        const int part = (int)(t0 % kTileTokens) / 32;  // of the stage, in 32 tokens
        const char *stages = static_cast<const char *>(a.work) + t0 / kTileTokens * g.steps * S::BYTES;
        // this wavefront's 64 rows, a tile of the packed planes; past the last one the last again
        const int64_t want = rt * (kTileOut / 64) + wave, last = (a.w.rows + 63) / 64 - 1;
        const int64_t tile = want < last ? want : last;
        const TileOf planes = tile_of<FMT>(a.w, tile, nb);
        uint32_t w[2][Words<FMT, QA>::N];
        uint16_t d0[2][P::BLOCKS];
        const int lane16 = 16 * lane;
        // lane16 anew: what follows from it is computed where it is used, and not kept (there are no registers left for it)
        auto anew = [&] {
            int x = lane16;
            asm volatile("" : "+v"(x));
            return x;
        };
        // a stage: as many loads in every wavefront, so that they can be counted (fewer pieces than wavefronts:
        // two load the same)
        auto fetch_stage = [&](int step) {
            const rsrc_t from = rsrc_of(reinterpret_cast<const u32x4 *>(stages + (int64_t)step * S::BYTES));
            char *to = mine + step / KG % 3 * BYTES;
#pragma unroll
            for (int c = 0; c < M; ++c)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lptr)(to + (M * wave + c) * 1024), 16, lane16,
                                                         4096 * part + (M * wave + c) * 1024, 0, 0);
#pragma unroll
            for (int c = 0; c < LOADS; ++c) {
                // piece: 64 values, first all of a group's scales, then its starts
                const int piece = (LOADS * wave + c) % PIECES, at = piece * 256, in = at % (TOKENS * 8);
                const int j = at / (TOKENS * 8), kind = in / (TOKENS * 4), off = in % (TOKENS * 4);
                int lane4 = anew() >> 2;
                if (M == 1)  // 32 scales and 32 starts, 512 bytes apart
                    lane4 += lane4 >= 128 ? 384 : 0;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lptr)(to + QUANTS + at), 4, lane4,
                                                         S::QUANTS + 1024 * j + 512 * kind + 128 * part + off, 0, 0);
            }
        };
        auto fetch_weights = [&](int step) {
            const int x = anew(), at = (x & 0x1F0) | (x >> 9 << 3);
#pragma unroll
            for (int n = 0; n < 2; ++n)
                load_weights<FMT, QA>(planes, 32 * n, at, step * P::BLOCKS, nb, w[n], d0[n]);
        };
        f32x16 acc[M][2];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[m][n][i] = 0.0f;
        if (kg < steps) {
            fetch_stage(kg);
            fetch_weights(kg);
        }
        if (kg + KG < steps)
            fetch_stage(kg + KG);
        // all groups go around alike; a group without a step waits
        for (int step = kg; step - kg < steps; step += KG) {
            i32x4 b[2][4];
            float dw[2][P::BLOCKS], off[2][P::BLOCKS];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    b[n][m] = weight_operand<FMT, QA>(w[n], half, m);
#pragma unroll
                for (int j = 0; j < P::BLOCKS; ++j) {
                    dw[n][j] = f16_bits_to_f32(d0[n][j]);
                    asm("" : "+v"(dw[n][j]));
                    off[n][j] = -kMagicF * dw[n][j];
                }
            }
            // what was asked for before the last stage is here: this step's part of the stage
            if (step + KG < steps)
                __builtin_amdgcn_s_waitcnt(0x0F70 | (M + LOADS));
            else
                __builtin_amdgcn_s_waitcnt(0x0F70);
            __syncthreads();
            if (KG > 1 && step >= steps)
                continue;
            if (step + KG < steps)
                fetch_weights(step + KG);
            if (step + 2 * KG < steps)
                fetch_stage(step + 2 * KG);
            const char *stage = mine + step / KG % 3 * BYTES;
            const int half16 = anew() >> 9 << 4;
            // units: 32 tokens, a group of k, 32 rows.  A unit's products are issued among the scaling of the unit before.
            i32x4 f[4];
            f32x16 d;
            i32x16 s[2];
            constexpr int UNITS = M * P::NG * 2;
#pragma unroll
            for (int u = 0; u <= UNITS; ++u) {
                const int n = u & 1, j = u / 2 % P::NG, m = u / 2 / P::NG;
                if (u < UNITS) {
                    if (n == 0 && j == 0)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            f[x] = *reinterpret_cast<const i32x4 *>(stage + (4 * m + x) * 1024 + lane16);
                    const int *starts = reinterpret_cast<const int *>(stage + QUANTS + half16) + 2 * TOKENS * j + 32 * m + TOKENS;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const i32x4 c = *reinterpret_cast<const i32x4 *>(starts + 8 * x);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            s[n][4 * x + y] = c[y];
                    }
#pragma unroll
                    for (int x = j * P::GM; x < (j + 1) * P::GM; ++x)
                        s[n] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[x], b[n][x], s[n], 0, 0, 0);
                }
                if (u > 0) {
                    const int mm = (u - 1) / 2 / P::NG, nn = n ^ 1, jj = (u - 1) / 2 % P::NG;
                    if (nn == 0) {
                        const float *sc = reinterpret_cast<const float *>(stage + QUANTS + half16) + 2 * TOKENS * jj + 32 * mm;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const f32x4 e = *reinterpret_cast<const f32x4 *>(sc + 8 * x);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                d[4 * x + y] = e[y];
                        }
                    }
                    const float p = dw[nn][jj * P::G / P::BL], o = off[nn][jj * P::G / P::BL];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[mm][nn][i] = __builtin_fmaf(__builtin_fmaf(as_float(s[nn][i]), p, o), d[i], acc[mm][nn][i]);
                }
            }
        }
        // through LDS, 32 tokens at a time, to 64 rows side by side: column c of token t at c ^ 32 (t / 4 % 2), so that
        // the lane halves, 4 tokens apart, write to different banks.  The groups of wavefronts add up there.
        float *out = reinterpret_cast<float *>(lds) + wave * 2048;
        const int64_t r = want * 64 + lane;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            auto place = [&](int i, int n) { return (8 * (i / 4) + 4 * half + i % 4) * 64 + ((32 * n + in32) ^ 32 * half); };
#pragma unroll
            for (int from = KG - 1; from >= 0; --from) {
                __syncthreads();
                if (kg == from)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            out[place(i, n)] = from == KG - 1 ? acc[m][n][i] : acc[m][n][i] + out[place(i, n)];
            }
            __syncthreads();
            if (r < a.w.rows)
#pragma unroll 1
                for (int c = 32 / KG * kg; c < 32 / KG * (kg + 1); c += 8) {
                    const int64_t first = t0 + 32 * m + c;
                    float x[8];
                    int64_t t[8];
                    bool live[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = out[(c + e) * 64 + (lane ^ 32 * (e / 4))];
                        live[e] = first + e < a.a.ncols;
                        t[e] = live[e] ? first + e : a.a.ncols - 1;
                    }
                    finish<8>(a, x, t, live, r);
                }
        }
        __syncthreads();
    }
}

template <int FMT, int QA>
static void tiles_kind(const MatmulArgs &g, int tokens, hipStream_t st)
{
    const int64_t most = int64_t(1) << 22, items = (g.token_tiles * g.row_tiles + 7) / 8 * 8;
    const dim3 grid((unsigned)(items < most ? items : most));
    if (tokens == 64)
        hipLaunchKernelGGL((matmul_tiles<FMT, QA, 2, 1>), grid, dim3(256), 0, st, g);
    else
        hipLaunchKernelGGL((matmul_tiles<FMT, QA, 1, 2>), grid, dim3(512), 0, st, g);
}

hipError_t launch_matmul_tiles(MatmulArgs g, int tokens, hipStream_t st)
{
    g.token_tiles = (g.p.a.ncols + (int64_t)tokens - 1) / tokens;
    g.row_tiles = (g.p.w.rows + kTileOut - 1) / kTileOut;
    const int qa = g.p.a.qa;
    if (g.p.w.fmt == BQ_Q1_0)
        qa == 32 ? tiles_kind<BQ_Q1_0, 32>(g, tokens, st) : qa == 64 ? tiles_kind<BQ_Q1_0, 64>(g, tokens, st) : tiles_kind<BQ_Q1_0, 128>(g, tokens, st);
    else
        qa == 32 ? tiles_kind<BQ_Q2_0, 32>(g, tokens, st) : qa == 64 ? tiles_kind<BQ_Q2_0, 64>(g, tokens, st) : tiles_kind<BQ_Q2_0, 128>(g, tokens, st);
    return hipGetLastError();
}

}  // namespace bq
