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

// The four A operands of a step for token row q (its first quant; valid: values
// of k that the row has from the step on, a multiple of 32 below 128 at its end).
template <int FMT, int QA>
__device__ __forceinline__ void act_operands(const int8_t *q, int half, int valid, u32x4 (&f)[4])
{
    typedef Shape<FMT, QA> P;
    uint32_t n[4][8];  // the four words of 32 values of the step
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            u32x4 v = {0, 0, 0, 0};
            if (FMT == BQ_Q1_0 || 32 * w < valid)
                v = *reinterpret_cast<const u32x4 *>(q + 32 * w + 16 * x);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                n[w][4 * x + e] = v[e];
        }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        uint32_t p[4];
        if constexpr (FMT == BQ_Q1_0) {
            if constexpr (P::G == 32) {  // word m, its halves in the lane halves
                word_half_q1(n[m], half, p);
            } else {  // words 2 (m / 2) + half
                uint32_t mine[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    mine[e] = half ? n[m / 2 * 2 + 1][e] : n[m / 2 * 2][e];
                word_half_q1(mine, m & 1, p);
            }
        } else {  // word 2 (m % 2) + half of block m / 2, 16 quants each
            uint32_t mine[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mine[e] = half ? n[m][4 + e] : n[m][e];
            word_q2(mine, p);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f[m][e] = p[e];
    }
}

// The four B operands of a step from the row's payload words.  Q1_0: w[0], the
// block's four words; Q2_0: two blocks.
template <int FMT, int QA>
__device__ __forceinline__ void weight_operand(const u32x4 (&w)[Shape<FMT, QA>::BLOCKS], int half, int m, i32x4 &f)
{
    typedef Shape<FMT, QA> P;
    if constexpr (FMT == BQ_Q1_0) {
        uint32_t x = P::G == 32 ? w[0][m] : half ? w[0][m / 2 * 2 + 1] : w[0][m / 2 * 2];
        if constexpr (P::G == 32)
            x = half ? x >> 4 | x << 28 : x;
        const int at = P::G == 32 ? 0 : 4 * (m & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (int32_t)((at + i ? x >> (at + i - 1) : x << 1) & 0x02020202u);
    } else {
        const uint32_t x = half ? w[m / 2][m % 2 * 2 + 1] : w[m / 2][m % 2 * 2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (int32_t)(x >> (2 * i) & 0x03030303u);
    }
}

// The block of the payload plane (in units of 64 rows) where rows r0 .. of a step
// start, and the row's scale; past the last block (Q2_0, an odd number of them)
// the last one again: its quants are zeros.
template <int FMT>
__device__ __forceinline__ int64_t clamp_block(int64_t b, int64_t nb) { return b < nb ? b : nb - 1; }

// act(x + bias) * mul + res, and the store.
template <class T>
__device__ __forceinline__ void finish(const bq_product &a, float x, int64_t t, int64_t r)
{
    if (a.bias)
        x += a.bias[r];
    switch (a.act) {
    case BQ_SILU: x = x / (1.0f + expf(-x)); break;
    case BQ_GELU: x = x / (1.0f + expf(-1.59576912160573f * __builtin_fmaf(0.044715f * x * x, x, x))); break;
    case BQ_RELU2: x = fmaxf(x, 0.0f) * fmaxf(x, 0.0f); break;
    default: break;
    }
    if (a.mul)
        x *= (float)static_cast<const T *>(a.mul)[t * a.ld_mul + r];
    if (a.res)
        x += (float)static_cast<const T *>(a.res)[t * a.ld_res + r];
    static_cast<T *>(a.y)[t * a.ld_y + r] = (T)x;
}

}  // namespace bq
