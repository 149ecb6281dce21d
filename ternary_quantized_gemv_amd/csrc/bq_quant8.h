// bq_quant8.h -- internal to libbq: how the norm and the gated activation turn
// values into quants and scales, eight values a lane.
#pragma once

#include "bq_device.h"

namespace bq {

// The largest m of the qa / 8 neighbouring lanes that hold a block.
__device__ __forceinline__ float block_max(float m, int qa)
{
    m = fmaxf(m, __shfl_xor(m, 1, 64));
    m = fmaxf(m, __shfl_xor(m, 2, 64));
    if (qa > 32)
        m = fmaxf(m, __shfl_xor(m, 4, 64));
    if (qa > 64)
        m = fmaxf(m, __shfl_xor(m, 8, 64));
    return m;
}

// Eight values of a block whose largest magnitude is m: their quants to q, the
// block's scale to d (null in all lanes but the block's first).
__device__ __forceinline__ void quantize8(const float (&v)[8], float m, bool f16_scale, int8_t *q_out, float *d_out)
{
    float db = m * (1.0f / 127.0f), q[8];
    // the product is rounded to f32 before it is narrowed: seen together, the two become one
    // instruction that rounds once (another f16 scale for one block in about 2^14)
    asm("" : "+v"(db));
    if (f16_scale)
        db = (float)(_Float16)db;
    if (f16_scale && db < 0x1p-14f) {
        // a subnormal f16 scale is coarser than 1/127 of the maximum: the clamp can bind
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = (float)quant_of(v[e], db);
    } else {
        quant_block<8>(v, db, q);
    }
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        lo |= (uint32_t)((int)q[e] & 0xFF) << (8 * e);
        hi |= (uint32_t)((int)q[4 + e] & 0xFF) << (8 * e);
    }
    *reinterpret_cast<uint2 *>(q_out) = make_uint2(lo, hi);
    if (d_out)
        *d_out = db;
}

}  // namespace bq
