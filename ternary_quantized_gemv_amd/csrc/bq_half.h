// bq_half.h -- internal to libbq: the three value types of the operators
// between the products, their 16-byte loads and stores, and the matrix
// instructions of the two 16-bit ones.
//
// Lane layout of v_mfma_f32_16x16x32 (wavefront lane l): A holds row l % 16,
// B column l % 16, both at k = 8 (l / 16) + e for element e of the lane's
// eight; C and D hold rows 4 (l / 16) + i, i < 4, of column l % 16.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/bq.h"
#include "bq_types.h"

namespace bq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int TYPE> struct Num;
template <> struct Num<BQ_F32> { typedef float t; };
template <> struct Num<BQ_F16> {
    typedef _Float16 t;
    typedef f16x8 v8;
    static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(v8 a, v8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Num<BQ_BF16> {
    typedef __bf16 t;
    typedef bf16x8 v8;
    static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(v8 a, v8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// Eight consecutive values (16-byte aligned) widened to f32; the store rounds
// to nearest even.
template <class T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    } else {
        typedef T tx8 __attribute__((ext_vector_type(8)));
        const tx8 a = *reinterpret_cast<const tx8 *>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = (float)a[e];
    }
}

template <class T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        f32x4 a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = v[e];
            b[e] = v[4 + e];
        }
        reinterpret_cast<f32x4 *>(p)[0] = a;
        reinterpret_cast<f32x4 *>(p)[1] = b;
    } else {
        typedef T tx8 __attribute__((ext_vector_type(8)));
        tx8 a;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            a[e] = (T)v[e];
        *reinterpret_cast<tx8 *>(p) = a;
    }
}

// Sixteen bytes as a vector of 16-bit values; ONCE: nothing reads them again,
// so they need no place in the caches (non-temporal).
template <class V, bool ONCE, class T>
__device__ __forceinline__ V stream8(const T *p)
{
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
    return __builtin_bit_cast(V, ONCE ? __builtin_nontemporal_load(q) : *q);
}

// The maximum (or sum) over the two halves of a wavefront, and over the pairs
// of 16-lane rows: lanes l, l ^ 32 and l, l ^ 16.
template <class OP>
__device__ __forceinline__ float across32(float x, OP op)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x), false, false);
    return op(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
template <class OP>
__device__ __forceinline__ float across16(float x, OP op)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x), false, false);
    return op(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// A value of another lane of the same 16 (DPP control CTRL); lanes without one,
// and rows of 16 that ROWS leaves out, get `none`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp(int x, int none)
{
    return __builtin_amdgcn_update_dpp(none, x, CTRL, ROWS, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp_all(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

// The sum (maximum) over a wavefront in every lane, without LDS: rotations by 8,
// 4, 2 and 1 within 16 lanes, then the rows of 16.
template <class OP>
__device__ __forceinline__ float wave_all(float x, OP op)
{
    x = op(x, dpp_all<0x128>(x));
    x = op(x, dpp_all<0x124>(x));
    x = op(x, dpp_all<0x122>(x));
    x = op(x, dpp_all<0x121>(x));
    return across32(across16(x, op), op);
}

// Inclusive sum over the lanes up to this one: shifts within 16 lanes, then the
// last lane of each row of 16 to the next rows.
__device__ __forceinline__ int wave_scan(int x)
{
    x += dpp<0x111>(x, 0);
    x += dpp<0x112>(x, 0);
    x += dpp<0x114>(x, 0);
    x += dpp<0x118>(x, 0);
    x += dpp<0x142, 0xA>(x, 0);
    x += dpp<0x143, 0xC>(x, 0);
    return x;
}

// A 32-bit word that the whole wavefront reads from device memory that the
// kernel does not write: one scalar load.
__device__ __forceinline__ int uniform_word(const int32_t *p)
{
    typedef const int32_t __attribute__((address_space(4))) *cptr;
    return *(cptr)(uintptr_t)p;
}

// Sizes in bytes of the three types.
inline int type_size(int type) { return type == BQ_F32 ? 4 : 2; }

// The items of all requests in a row: request i has count(i, other) of them,
// and a workgroup asks for items in increasing order (item, item + grid, ...).
// Each lane counts one request of 64 at a time.  `other` is a second number
// that is added up beside the items.  Between two items only these are kept
// (scalars: the registers of a workgroup at work are its products').
struct Walk {
    int base = 0;                 // the first of the 64 requests in hand
    int before = 0, before2 = 0;  // items (second numbers) of the requests in front of them
};
// Request b that has the item, its number there, and the second numbers of the
// requests in front of b (TWO); false behind the last item.  The same in all lanes.
template <bool TWO, class COUNT>
__device__ __forceinline__ bool find_item(Walk &w, int requests, int item, int &b, int &within, int &front, COUNT count)
{
    const int lane = threadIdx.x & 63;
    for (; w.base < requests; w.base += 64) {
        int mine = 0, mine2 = 0;
        if (w.base + lane < requests)
            mine = count(w.base + lane, mine2);
        const int upto = wave_scan(mine), upto2 = TWO ? wave_scan(mine2) : 0;
        const unsigned long long has = __ballot(item - w.before < upto);
        if (has) {
            const int at = __builtin_ctzll(has);
            b = w.base + at;
            within = item - w.before - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(mine, at));
            front = TWO ? w.before2 + __builtin_amdgcn_readlane(upto2, at) - __builtin_amdgcn_readlane(mine2, at) : 0;
            return true;
        }
        w.before += __builtin_amdgcn_readlane(upto, 63);
        if (TWO)
            w.before2 += __builtin_amdgcn_readlane(upto2, 63);
    }
    return false;
}

// The request that row t belongs to, of n requests with rows cu[b] ..
// cu[b+1] - 1: the last b with cu[b] <= t (requests without rows are skipped
// by it); n or more, or -1, where no request has the row.
__device__ __forceinline__ int request_of(const int32_t *cu, int n, int t)
{
    if (t < cu[0] || t >= cu[n])
        return -1;
    int lo = 0, hi = n;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace bq
