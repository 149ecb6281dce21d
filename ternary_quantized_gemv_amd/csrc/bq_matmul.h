// bq_matmul.h -- internal to libbq: what the kernels of bq_matmul share.
//
// A step is 128 values of k (one Q1_0 block, two of Q2_0), in NG groups: a group
// is what one weight scale and one activation scale cover.  The exact sums of a
// group come from v_mfma_i32_32x32x32_i8 over 32 tokens and 32 rows: A holds the
// quants of token lane % 32, B the weights of row lane % 32, both at 16 values of
// k a lane half; D holds row lane % 32 of tokens 8 (i / 4) + 4 (lane / 32) + i % 4.
//
// Weights become bytes by a shift and a mask: (word >> i) & 0x0202.. are 2 b for
// sign bits b, & 0x0303.. codes c, four weights eight bits apart.  Since w = 2 b - 1
// = c - 1, sum w q = sum (2 b or c) q - S with S the group's sum of quants, and the
// accumulator starts at kMagic - S: as an f32 the result then reads 1.5 2^23 + sum
// w q without a conversion, and fma(result, d0, -1.5 2^23 d0) is d0 times the sum,
// rounded once (1.5 2^23 times an f16 is exact).  Which k a byte holds is the same
// for A and B, and the sums are exact, so it need not be the order in memory.
#pragma once

#include "bq_device.h"
#include "bq_half.h"
#include "bq_model.h"

namespace bq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kMagic = 0x4B400000;        // 1.5 2^23 as f32
constexpr float kMagicF = 12582912.0f;
constexpr int kStepK = 128;

template <int FMT, int QA> struct Shape {
    static constexpr int BL = FMT == BQ_Q1_0 ? 128 : 64;
    static constexpr int G = QA < BL ? QA : BL;  // values of k a group
    static constexpr int NG = kStepK / G;        // groups a step
    static constexpr int GM = G / 32;            // matrix instructions a group
    static constexpr int BLOCKS = kStepK / BL;   // weight blocks a step
};

// (by value: a bit cast of a vector's element in place reads its first one)
__device__ __forceinline__ float as_float(int32_t x) { return __builtin_bit_cast(float, x); }

__device__ __forceinline__ uint32_t bytes_of(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }

// The quants of a lane in the order of the weights' bytes.  Rotated words hold
// canonical weight k at bit k + 2 (Q2_0: 2 k + 2).
//
// Q1_0, n[8] the 32 quants of a word: half 0 gives bit positions 0 .. 3 (and 8, 16,
// 24 further on), half 1 positions 4 .. 7.
__device__ __forceinline__ void word_half_q1(const uint32_t (&n)[8], int half, uint32_t (&p)[4])
{
    uint32_t a[4], b[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        a[c] = half ? n[2 * c + 1] : n[2 * c];
        b[c] = half ? n[2 * c] : n[(2 * c + 7) & 7];
    }
    const uint32_t a01 = bytes_of(a[1], a[0], 0x05010400u), a23 = bytes_of(a[3], a[2], 0x05010400u);  // bytes 0, 0, 1, 1
    const uint32_t b01 = bytes_of(b[1], b[0], 0x07030602u), b23 = bytes_of(b[3], b[2], 0x07030602u);  // bytes 2, 2, 3, 3
    p[0] = bytes_of(b23, b01, 0x05040100u);
    p[1] = bytes_of(b23, b01, 0x07060302u);
    p[2] = bytes_of(a23, a01, 0x05040100u);
    p[3] = bytes_of(a23, a01, 0x07060302u);
}
// Q2_0, n[4] the 16 quants of a word: bit positions 0, 2, 4, 6.
__device__ __forceinline__ void word_q2(const uint32_t (&n)[4], uint32_t (&p)[4])
{
    const uint32_t l01 = bytes_of(n[1], n[0], 0x05010400u), l23 = bytes_of(n[3], n[2], 0x05010400u);
    const uint32_t h01 = bytes_of(n[1], n[0], 0x07030602u), h23 = bytes_of(n[3], n[2], 0x07030602u);
    const uint32_t last = bytes_of(h23, h01, 0x07060302u);
    p[0] = last << 8 | last >> 24;
    p[1] = bytes_of(l23, l01, 0x05040100u);
    p[2] = bytes_of(l23, l01, 0x07060302u);
    p[3] = bytes_of(h23, h01, 0x05040100u);
}

// Which words of a row a lane half has.  Where a group is a whole block, half h has
// words 2 h and 2 h + 1 (8 bytes together); otherwise both halves share the words of
// a group: words h and 2 + h, or (Q1_0 in groups of 32) half of every word.
template <int FMT, int QA> struct Words {
    typedef Shape<FMT, QA> P;
    static constexpr bool PAIR = P::G == P::BL;
    static constexpr int N = FMT == BQ_Q1_0 && P::G > 32 ? 2 : 4;  // words a lane and step
    // first value of k (of the step) that word i of a lane half holds
    static __device__ __forceinline__ int first(int i, int half)
    {
        if constexpr (FMT == BQ_Q1_0)
            return 32 * (P::G == 32 ? i : PAIR ? 2 * half + i : 2 * i + half);
        else
            return 64 * (i / 2) + 16 * (PAIR ? 2 * half + i % 2 : i % 2 * 2 + half);
    }
};

// The four A operands of a step for the token row whose quants of the step are at q
// (the row has `valid` of them, a multiple of 32; the others count as zeros).
template <int FMT, int QA>
__device__ __forceinline__ void act_operands(const int8_t *q, int half, int valid, u32x4 (&f)[4])
{
    typedef Words<FMT, QA> W;
#pragma unroll
    for (int i = 0; i < W::N; ++i) {
        const int k = W::first(i, half);
        const u32x4 *p = reinterpret_cast<const u32x4 *>(q + k);
        if constexpr (FMT == BQ_Q1_0) {
            uint32_t n[8], o[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const u32x4 v = k < valid ? p[x] : u32x4{0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    n[4 * x + e] = v[e];
            }
            if constexpr (W::N == 4) {
                word_half_q1(n, half, o);
                f[i] = u32x4{o[0], o[1], o[2], o[3]};
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    word_half_q1(n, x, o);
                    f[2 * i + x] = u32x4{o[0], o[1], o[2], o[3]};
                }
            }
        } else {
            const u32x4 v = k < valid ? *p : u32x4{0, 0, 0, 0};
            const uint32_t n[4] = {v[0], v[1], v[2], v[3]};
            uint32_t o[4];
            word_q2(n, o);
            f[i] = u32x4{o[0], o[1], o[2], o[3]};
        }
    }
}

// The packed planes of a tile of 64 rows: uniform bases, 32-bit offsets of the lane's
// row (no vector addresses are kept).
struct TileOf {
    rsrc_t bits, scales;
};
template <int FMT>
__device__ __forceinline__ TileOf tile_of(const bq_weights &w, int64_t tile, int64_t nb)
{
    return TileOf{rsrc_of(static_cast<const u32x4 *>(w.bits) + tile_block0(FMT, tile, nb) * kTileRows),
                  rsrc_of(reinterpret_cast<const u32x4 *>(w.scales) + tile * ((nb + 7) / 8) * kTileRows)};
}

// A lane's words of the step that starts with block b, and its scales.  Its row of the
// tile is row0 (the same in all lanes) + lane % 32; at = 16 (lane % 32) + 8 half.  Past
// the last block (Q2_0, an odd number of them) the last one again: its quants are zeros.
template <int FMT, int QA>
__device__ __forceinline__ void load_weights(const TileOf &t, int row0, int at, int b, int nb, uint32_t (&w)[Words<FMT, QA>::N],
                                             uint16_t (&d0)[Shape<FMT, QA>::BLOCKS])
{
    typedef Words<FMT, QA> W;
    constexpr int BLOCKS = Shape<FMT, QA>::BLOCKS, EACH = W::N / BLOCKS;
    const int row = at & ~15, half4 = (at & 8) >> 1;
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {
        const uint32_t block = b + j < nb ? b + j : nb - 1, from = block * kStep + row0 * 16;
        if constexpr (W::PAIR) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(t.bits, at, from, 0);
            w[2 * j] = v[0];
            w[2 * j + 1] = v[1];
        } else if constexpr (W::N == 4 && FMT == BQ_Q1_0) {
            const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(t.bits, row, from, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = v[i];
        } else {  // words h and 2 + h
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                w[EACH * j + i] = __builtin_amdgcn_raw_buffer_load_b32(t.bits, row + half4, from + 8 * i, 0);
        }
        d0[j] = __builtin_amdgcn_raw_buffer_load_b16(t.scales, row, (block >> 3) * kStep + row0 * 16 + (block & 7) * 2, 0);
    }
}

// B operand m of a step from a lane's words.
template <int FMT, int QA>
__device__ __forceinline__ i32x4 weight_operand(const uint32_t (&w)[Words<FMT, QA>::N], int half, int m)
{
    typedef Words<FMT, QA> W;
    i32x4 f;
    if constexpr (FMT == BQ_Q1_0) {
        uint32_t x = W::N == 4 ? w[m] : w[m / 2];
        if constexpr (W::N == 4)
            x = half ? x >> 4 | x << 28 : x;
        const int at = W::N == 4 ? 0 : 4 * (m & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (int32_t)((at + i ? x >> (at + i - 1) : x << 1) & 0x02020202u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (int32_t)(w[m] >> (2 * i) & 0x03030303u);
    }
    return f;
}

// The sum of a group's quants, from the operands of both lane halves.
template <int GM>
__device__ __forceinline__ int quant_sum(const u32x4 *f)
{
    int s = 0;
#pragma unroll
    for (int m = 0; m < GM; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s = __builtin_amdgcn_sdot4((int)f[m][e], 0x01010101, s, false);
    return s + __shfl_xor(s, 32, 64);
}

// act(x + bias) * mul + res of row r, and the stores, for tokens t[0 .. N) as far as they
// are live.  The others' t is the last token: loads of all are under way together.
template <class T, int N>
__device__ __forceinline__ void store_rows(const bq_product &a, float (&x)[N], const int64_t (&t)[N], const bool (&live)[N], int64_t r)
{
    if (a.mul) {
        T v[N];
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] = static_cast<const T *>(a.mul)[t[e] * a.ld_mul + r];
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] *= (float)v[e];
    }
    if (a.res) {
        T v[N];
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] = static_cast<const T *>(a.res)[t[e] * a.ld_res + r];
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] += (float)v[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (live[e])
            static_cast<T *>(a.y)[t[e] * a.ld_y + r] = (T)x[e];
}
// x / (1 + exp(-z)) with z = z_of(x), which has x's sign and rises with x.  v_rcp_f32 is good to one unit in the last
// place, but gives 0 where the inverse is subnormal, from 1 + exp(-z) = 2^126 (z below -87.3) on; the result is down to
// -1e-36 there.  With exp(-|z|) the sum is 1 to 2: for all N of a lane if one is that far below zero (2049 x 12288 x 4096
// 202 us with this form alone, 200 with both).
template <int N, class Z>
__device__ __forceinline__ void times_sigmoid(float (&x)[N], Z z_of)
{
    float low = x[0];
#pragma unroll
    for (int e = 1; e < N; ++e)
        low = fminf(low, x[e]);
    if (z_of(low) > -80.0f) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] *= __builtin_amdgcn_rcpf(1.0f + expf(-z_of(x[e])));
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float y = expf(-fabsf(z_of(x[e])));
        x[e] = (x[e] < 0.0f ? x[e] * y : x[e]) * __builtin_amdgcn_rcpf(1.0f + y);
    }
}
template <int N>
__device__ __forceinline__ void finish(const bq_product &a, float (&x)[N], const int64_t (&t)[N], const bool (&live)[N], int64_t r)
{
    if (a.bias) {
        const float b = a.bias[r];
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] += b;
    }
    switch (a.act) {
    case BQ_SILU: times_sigmoid<N>(x, [](float v) { return v; }); break;
    case BQ_GELU:
        times_sigmoid<N>(x, [](float v) { return 1.59576912160573f * __builtin_fmaf(0.044715f * v * v, v, v); });
        break;
    case BQ_RELU2:
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] = fmaxf(x[e], 0.0f) * fmaxf(x[e], 0.0f);
        break;
    default: break;
    }
    switch (a.type) {
    case BQ_F16: store_rows<_Float16, N>(a, x, t, live, r); break;
    case BQ_BF16: store_rows<__bf16, N>(a, x, t, live, r); break;
    default: store_rows<float, N>(a, x, t, live, r); break;
    }
}

// Laid-out activations (matmul_lay): for every 128 tokens and step of k a stage of 4 x 4
// operands (32 tokens and 32 values of k: 64 lanes of 16 bytes), then for every group
// 128 scales and 128 starting values.
constexpr int kTileTokens = 128, kTileOut = 256;
template <int FMT, int QA> struct Stage {
    static constexpr int QUANTS = kTileTokens * kStepK;
    static constexpr int BYTES = QUANTS + Shape<FMT, QA>::NG * 1024;
};

struct MatmulArgs {
    bq_product p;
    int64_t token_tiles, row_tiles;  // of the kernel that follows
    int steps;                       // of k
};
// bq_matmul_tiles.hip, behind matmul_lay: 32 or 64 tokens a workgroup
hipError_t launch_matmul_tiles(MatmulArgs g, int tokens, hipStream_t st);

}  // namespace bq
