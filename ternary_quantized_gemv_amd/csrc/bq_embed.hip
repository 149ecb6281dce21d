// bq_embed.hip -- rows of a token table, packed or dense, scaled (bq_embed).
//
// A lane makes eight neighbouring values: of a packed row one byte (Q1_0) or
// half a word (Q2_0) and the block's scale, of a dense row 16 or 32 bytes.  The
// pieces of a packed row lie 1 KiB apart (64 rows a tile), 16 bytes each.
//
// Measured: 8191 ternary rows of 4096 to bf16 28 us.  That is memory: of every 16-byte
// piece a line of 128 comes along (75 MB, 9.4 of them needed), beside 67 MB of outputs
// (5 TB/s).  Four pieces a lane with their loads under way together: 29.6.  One row 2.2 us.
// Dense rows: 8191 of 4096 bf16 to bf16 25 us, f16 to f32 36, f32 to f32 45 (5.3 to 5.9 TB/s).
#include "bq_device.h"
#include "bq_half.h"
#include "bq_model.h"

namespace bq {

constexpr int kEmbedThreads = 256;

// TABLE: value type of a dense table, or void with FMT.
template <int FMT, class TABLE, class OUT>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(const bq_table a)
{
    const int per_row = (int)(a.w.cols / 8);
    const int64_t total = a.tokens * per_row;
    for (int64_t first = (int64_t)blockIdx.x * kEmbedThreads; first < total; first += (int64_t)gridDim.x * kEmbedThreads) {
        // the division by the row length once a workgroup in 64 bits, then in 32
        const int64_t t0 = first / per_row;
        const uint32_t off = (uint32_t)(first - t0 * per_row) + threadIdx.x;
        const int64_t t = t0 + off / (uint32_t)per_row;
        const int c = (int)(off % (uint32_t)per_row);
        if (t >= a.tokens)
            return;
        const int64_t id = a.ids[t];
        float v[8] = {};
        if (id >= 0 && id < a.w.rows) {
            if constexpr (FMT == 0) {
                load8(static_cast<const TABLE *>(a.dense) + id * a.ld_dense + 8 * (int64_t)c, v);
            } else {
                constexpr int EACH = FMT == BQ_Q1_0 ? 16 : 8;  // lanes a block
                const int64_t nb = a.w.cols / (8 * EACH), tile = id / kTileRows, lane = id % kTileRows;
                const int64_t b = c / EACH, block = tile_block0(FMT, tile, nb) + b;
                const int part = c % EACH;
                const uint32_t *w = static_cast<const uint32_t *>(a.w.bits) + (block * kTileRows + lane) * 4;
                const float d = f16_bits_to_f32(
                    a.w.scales[((tile * ((nb + 7) / 8) + b / 8) * kTileRows + lane) * 8 + b % 8]);
                const uint32_t word = w[part / (EACH / 4)];
                const uint32_t plain = word >> 2 | word << 30;
                if constexpr (FMT == BQ_Q1_0) {
                    const uint32_t bits = plain >> (8 * (part & 3));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = (bits >> e & 1) ? d : -d;
                } else {
                    const uint32_t bits = plain >> (16 * (part & 1));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = (float)((int)(bits >> (2 * e) & 3) - 1) * d;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= a.scale;
                // rounded to f32 before it is narrowed: seen together, the two become one instruction that rounds once
                asm("" : "+v"(v[e]));
            }
        }
        store8(static_cast<OUT *>(a.out) + t * a.ld_out + 8 * (int64_t)c, v);
    }
}

template <int FMT, class TABLE>
static void embed_out(const bq_table &a, dim3 grid, hipStream_t st)
{
    switch (a.type) {
    case BQ_F16: hipLaunchKernelGGL((embed_kernel<FMT, TABLE, _Float16>), grid, dim3(kEmbedThreads), 0, st, a); break;
    case BQ_BF16: hipLaunchKernelGGL((embed_kernel<FMT, TABLE, __bf16>), grid, dim3(kEmbedThreads), 0, st, a); break;
    default: hipLaunchKernelGGL((embed_kernel<FMT, TABLE, float>), grid, dim3(kEmbedThreads), 0, st, a); break;
    }
}

hipError_t launch_embed(const bq_table &a, hipStream_t st)
{
    // a grid holds fewer than 2^32 threads; workgroups walk on from there
    const int64_t blocks = (a.tokens * (a.w.cols / 8) + kEmbedThreads - 1) / kEmbedThreads, most = int64_t(1) << 22;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    if (a.w.fmt == BQ_Q1_0)
        embed_out<BQ_Q1_0, void>(a, grid, st);
    else if (a.w.fmt == BQ_Q2_0)
        embed_out<BQ_Q2_0, void>(a, grid, st);
    else if (a.dense_type == BQ_F16)
        embed_out<0, _Float16>(a, grid, st);
    else if (a.dense_type == BQ_BF16)
        embed_out<0, __bf16>(a, grid, st);
    else
        embed_out<0, float>(a, grid, st);
    return hipGetLastError();
}

}  // namespace bq
