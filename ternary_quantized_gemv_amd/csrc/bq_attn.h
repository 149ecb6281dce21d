// bq_attn.h -- internal to libbq: what the two attention kernels share
// (bq_attn.hip: few rows, keys split over wavefronts; bq_attn_tiles.hip: many
// rows, keys shared through LDS).
#pragma once

#include "bq_half.h"
#include "bq_layer.h"
#include "bq_rows.h"

namespace bq {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNone = -__builtin_inff();

// Parts of an f32 value in 16-bit type T, and the power of two that the
// weights are scaled by (both in the numerator and in l).
template <class T> struct Parts { static constexpr int n = 3; static constexpr float up = 0.0f; };
template <> struct Parts<_Float16> { static constexpr int n = 2; static constexpr float up = 14.0f; };

struct AttnArgs {
    bq_attn a;
    AttnPlan p;
    int group;  // query heads per key head
    int page_log2;
};

// Which of the two kernels has a request of this many rows, where both run:
// the one for many rows has those of more than kFewRows.
constexpr int kFewRows = 64;
__device__ __forceinline__ bool has_few(const AttnPlan &p, int rows)
{
    return p.many.tiles == 0 || (p.few.cols && rows <= kFewRows);
}

// The keys and rows of one request (the same in all lanes), bounded by what the
// launch was given.
struct Request {
    int row0, n, keys;
};
__device__ __forceinline__ Request request_at(const bq_attn &a, int b)
{
    Request r;
    const Rows rows = rows_between(uniform_word(a.cu + b), uniform_word(a.cu + b + 1), a.tokens);
    r.row0 = rows.first;
    r.n = rows.n;
    const int64_t most = (int64_t)a.table_cols * a.cache.page;
    const int len = uniform_word(a.lens + b);
    r.keys = len < 0 ? 0 : len > most ? (int)most : len;
    return r;
}

// The same for a request of each lane: rows of query heads (0: not this
// kernel's, which `few` says) and keys.
__device__ __forceinline__ void lane_request(const AttnArgs &g, int b, bool few, int &rows, int &keys)
{
    const int len = g.a.lens[b], n = rows_between(g.a.cu[b], g.a.cu[b + 1], g.a.tokens).n;
    const int64_t most = (int64_t)g.a.table_cols * g.a.cache.page;
    rows = n > 0 && has_few(g.p, n * g.group) == few ? n * g.group : 0;
    keys = len < 0 ? 0 : len > most ? (int)most : len;
}

// Page of the 16 keys from `key` (a multiple of 16, the same in all lanes) of a
// request, -1 where there is none.
__device__ __forceinline__ int page_at(const AttnArgs &g, const int32_t *table, int key, int end)
{
    if (key >= end)
        return -1;
    const int p = uniform_word(table + (key >> g.page_log2));
    return (unsigned)p < (unsigned)g.a.cache.pages ? p : -1;
}

// Eight values in NP parts of type T: rounded, then the rest rounded.  Three
// parts of bf16 cut an f32's 24 bits into eights, exactly and without
// conversions (512 f32 rows over 30011 keys: 755 -> 717 us).
template <class T, int NP> struct Split {
    typedef T t8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ void parts(const float (&x)[8], t8 (&f)[NP])
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float rest = x[e];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                f[p][e] = (T)rest;
                rest -= (float)f[p][e];
            }
        }
    }
};
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
template <> struct Split<__bf16, 3> {
    static __device__ __forceinline__ void parts(const float (&x)[8], bf16x8 (&f)[3])
    {
        float rest[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            rest[e] = x[e];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = upper_halves(__builtin_bit_cast(uint32_t, rest[2 * i]), __builtin_bit_cast(uint32_t, rest[2 * i + 1]));
            f[p] = __builtin_bit_cast(bf16x8, w);
            if (p < 2)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    rest[e] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, rest[e]) & 0xFFFF0000u);
        }
    }
};

// One column's query fragments: element e of fragment j is q[at + step j + e].
// Returns the factor from products with the fragments to log2 units, never
// negative: a negative scale turns the sign of q instead, so that the largest
// score is the largest product.  f32 rows come in NP parts; over an f16 cache
// they are first scaled so that the row's largest value is 2^13 to 2^14
// (`across` is the maximum over the lanes that share a column).
template <class T, class v8, int NP, int N, bool F32, class ACROSS>
__device__ __forceinline__ float load_query(const bq_attn &a, int64_t at, int step, v8 (&f)[NP][N], ACROSS across)
{
    const bool neg = a.scale < 0.0f;
    float factor = fabsf(a.scale) * kLog2e;
    if constexpr (!F32) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            f[0][j] = *reinterpret_cast<const v8 *>(static_cast<const T *>(a.q) + at + step * j);
            if (neg)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[0][j][e] = -f[0][j][e];
        }
    } else {
        float x[N][8], top = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            load8(static_cast<const float *>(a.q) + at + step * j, x[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[j][e] = neg ? -x[j][e] : x[j][e];
                top = fmaxf(top, fabsf(x[j][e]));
            }
        }
        if constexpr (NP == 2) {
            top = across(top);
            int ex = 0;
            (void)__builtin_frexpf(top, &ex);
            ex = top > 0.0f ? (ex < -100 ? -100 : ex) : 14;
            const float up = __builtin_ldexpf(1.0f, 14 - ex);
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[j][e] *= up;
            factor = __builtin_ldexpf(factor, ex - 14);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            v8 part[NP];
            Split<T, NP>::parts(x[j], part);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                f[p][j] = part[p];
        }
    }
    return factor;
}

// A row's place in a piece: its D sums, and its maximum and sum of weights.
struct Part {
    float *sums;
    float2 *stats;
};
// Few rows: row `row` of piece `piece` (2 few.items of them per key head).
__device__ __forceinline__ Part few_part(const AttnArgs &g, int dim, int kh, int piece, int row)
{
    const int64_t at = ((int64_t)kh * 2 * g.p.few.items + piece) * g.p.few.cols + row;
    char *w = static_cast<char *>(g.a.work);
    return Part{reinterpret_cast<float *>(w) + at * dim, reinterpret_cast<float2 *>(w + g.p.few_stats) + at};
}
// Many rows: row `row` of a tile, the sums chunk by chunk, a row's statistics
// next to each other (one lane reads all of them).
__device__ __forceinline__ Part many_part(const AttnArgs &g, int dim, int kh, int tile, int chunk, int row)
{
    const int64_t tiles = (int64_t)kh * g.p.many.tiles + tile;
    char *w = static_cast<char *>(g.a.work);
    return Part{reinterpret_cast<float *>(w + g.p.many_sums) + ((tiles * g.p.many.chunks + chunk) * g.p.many.cols + row) * dim,
                reinterpret_cast<float2 *>(w + g.p.many_stats) + (tiles * g.p.many.cols + row) * g.p.many.chunks + chunk};
}
// What the kernels leave for the joins: the units of a piece of few rows' keys,
// the first piece of each split request of few rows, and the first tile of
// each request of many rows.
__device__ __forceinline__ int32_t *note_units(const AttnArgs &g)
{
    return reinterpret_cast<int32_t *>(static_cast<char *>(g.a.work) + g.p.notes);
}
__device__ __forceinline__ int32_t *note_piece(const AttnArgs &g, int b) { return note_units(g) + 4 + b; }
__device__ __forceinline__ int32_t *note_tile(const AttnArgs &g, int b) { return note_units(g) + 4 + g.a.requests + b; }

hipError_t launch_attn_tiles(const AttnArgs &g, hipStream_t st);

}  // namespace bq
