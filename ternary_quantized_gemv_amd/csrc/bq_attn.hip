// bq_attn.hip -- attention of new tokens over the paged cache (bq_paged_attn).
//
// o_r = sum_j exp(scale q_r.k_j - m_r) v_j / sum_j exp(scale q_r.k_j - m_r) in
// one pass over the keys, with a running maximum m_r and sum l_r per row.  The
// rows of one key head are its G query heads of each new token, row r = i G + g
// of token i: all of them see nearly the same keys, so a key is read once for
// up to 16 nt rows.
//
// A wavefront takes 32 keys at a time and computes the transposed products
// S^T = K Q^T and O^T = V^T P^T, rows of the result along keys (values), columns
// along rows r.  Result row r' = 4 g + i of 16-key tile t is assigned key
// 8 g + 4 t + i (g = lane / 16): a lane then holds the scores of keys 8 g .. 8 g
// + 7 of its column, which is exactly the second product's B operand, and the
// transposed value pages give its A operand as one 16-byte load.  So scores,
// weights and sums never leave the lane's registers, and m, l are two values
// per lane.
//
// f32 rows: q and the weights are split into 16-bit parts whose products with
// the cache are exact and add up in f32 (three of bf16, 24 bits; two of f16, 22
// bits, q scaled by a power of two per row).  f16 weights are scaled by 2^14 in
// either case, so that small ones stay clear of f16's subnormals.
#include "bq_half.h"
#include "bq_layer.h"

namespace bq {

constexpr int kAttnWaves = 4;
constexpr int kAttnKeys = 32;  // keys of a wavefront at a time
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

// The keys and rows of one request, bounded by what the launch was given.
struct Request {
    int row0, n, keys;
};
__device__ __forceinline__ Request request_at(const bq_attn &a, int b)
{
    Request r;
    const int lo = a.cu[b], hi = a.cu[b + 1];
    r.row0 = lo < 0 ? 0 : lo;
    const int end = hi > a.tokens ? (int)a.tokens : hi;
    r.n = lo < 0 ? 0 : end - lo;  // a request that starts before the rows is none
    const int64_t most = (int64_t)a.table_cols * a.cache.page;
    const int len = a.lens[b];
    r.keys = len < 0 ? 0 : len > most ? (int)most : len;
    return r;
}

// Page of key block `key` (a multiple of 8) of a request, -1 where there is none.
__device__ __forceinline__ int page_at(const AttnArgs &g, const int32_t *table, int key, int end)
{
    if (key >= end)
        return -1;
    const int p = table[key >> g.page_log2];
    return (unsigned)p < (unsigned)g.a.cache.pages ? p : -1;
}

template <int CT, int D, int NT, bool F32>
__global__ __launch_bounds__(64 * kAttnWaves) void attn_kernel(const AttnArgs g)
{
    typedef typename Num<CT>::t T;
    typedef typename Num<CT>::v8 v8;
    constexpr int NP = F32 ? Parts<T>::n : 1;
    constexpr int DJ = D / 32, DT = D / 16;
    __shared__ float sm[kAttnWaves][NT][16], sl[kAttnWaves][NT][16];
    __shared__ float so[NT * 16][D + 4];

    const bq_attn &a = g.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c16 = lane & 15, q4 = lane >> 4;
    const int b = blockIdx.z, kh = blockIdx.y;
    const int tile = blockIdx.x / g.p.chunks, chunk = blockIdx.x % g.p.chunks;
    const Request rq = request_at(a, b);
    if (rq.n <= 0)
        return;
    const int rows = rq.n * g.group;
    const int64_t page_elems = (int64_t)a.cache.heads << g.page_log2;
    const T *kbase = static_cast<const T *>(a.cache.k), *vbase = static_cast<const T *>(a.cache.v);
    const int32_t *table = a.table + (int64_t)b * a.ld_table;
    const int P = a.cache.page, pmask = P - 1;

    for (int r0 = tile * 16 * NT; r0 < rows; r0 += g.p.tiles * 16 * NT) {
        // ---- the rows: this lane's columns are rows r0 + 16 t + c16
        v8 qf[NT][NP][DJ];
        float qs[NT], m[NT], l[NT];
        int last[NT];  // the last key the column sees
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 16 * t + c16;
            const bool live = r < rows;
            const int i = live ? r / g.group : 0, hq = kh * g.group + (live ? r % g.group : 0);
            const int64_t at = (rq.row0 + i) * a.ld_q + (int64_t)hq * D + 8 * q4;
            last[t] = live ? rq.keys - rq.n + i : -1;
            m[t] = kNone;
            l[t] = 0.0f;
            qs[t] = a.scale * kLog2e;
            if constexpr (!F32) {
#pragma unroll
                for (int j = 0; j < DJ; ++j)
                    qf[t][0][j] = *reinterpret_cast<const v8 *>(static_cast<const T *>(a.q) + at + 32 * j);
            } else {
                float x[DJ][8], top = 0.0f;
#pragma unroll
                for (int j = 0; j < DJ; ++j) {
                    load8(static_cast<const float *>(a.q) + at + 32 * j, x[j]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        top = fmaxf(top, fabsf(x[j][e]));
                }
                if constexpr (NP == 2) {
                    top = fmaxf(top, __shfl_xor(top, 16, 64));
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    int ex;
                    (void)__builtin_frexpf(top, &ex);
                    ex = top > 0.0f ? ex : 0;
                    ex = ex < -100 ? -100 : ex;  // the largest value becomes 2^13 .. 2^14
                    const float up = __builtin_ldexpf(1.0f, 14 - ex > 120 ? 120 : 14 - ex);
#pragma unroll
                    for (int j = 0; j < DJ; ++j)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[j][e] *= up;
                    qs[t] /= up;
                }
#pragma unroll
                for (int j = 0; j < DJ; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float rest = x[j][e];
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            qf[t][p][j][e] = (T)rest;
                            rest -= (float)qf[t][p][j][e];
                        }
                    }
            }
        }
        f32x4 o[NT][DT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[t][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        // ---- the keys: those that the tile's last row sees, this workgroup's chunk of them
        const int last_row = min(r0 + 16 * NT, rows) - 1;
        const int seen = min(rq.keys, rq.keys - rq.n + last_row / g.group + 1);
        const int begin = chunk * g.p.chunk;
        const int end = chunk == g.p.chunks - 1 ? seen : min(seen, begin + g.p.chunk);
        const int first_last = rq.keys - rq.n + r0 / g.group;  // the last key that the tile's first row sees

        for (int k0 = begin + kAttnKeys * wave; k0 < end; k0 += kAttnKeys * kAttnWaves) {
            const int kk = k0 + 8 * (c16 >> 2), vk = k0 + 8 * q4;
            const int kp = page_at(g, table, kk, end), vp = page_at(g, table, vk, end);
            const bool whole = k0 + kAttnKeys - 1 <= first_last && k0 + kAttnKeys <= end && !__any(kp < 0);
            const T *kr = kbase + (int64_t)max(kp, 0) * page_elems * D + ((int64_t)kh * P + (kk & pmask) + (c16 & 3)) * D +
                          8 * q4;
            const T *vr = vbase + (int64_t)max(vp, 0) * page_elems * D + ((int64_t)kh * D + c16) * P + (vk & pmask);
            v8 kf[2][DJ], vf[DT];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < DJ; ++j)
                    kf[t][j] = *reinterpret_cast<const v8 *>(kr + 4 * t * D + 32 * j);
#pragma unroll
            for (int d = 0; d < DT; ++d)
                vf[d] = *reinterpret_cast<const v8 *>(vr + (int64_t)16 * d * P);
            if (!whole) {
                // places that no row sees may hold anything: their values must not meet a weight of 0
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        vf[d][e] = vk + e < end && vp >= 0 ? vf[d][e] : (T)0.0f;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 s[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int j = 0; j < DJ; ++j)
                            s[h] = Num<CT>::mfma16(kf[h][j], qf[t][p][j], s[h]);
                }
                float w[8], top = kNone;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = s[e >> 2][e & 3] * qs[t];
                    if (!whole)
                        w[e] = vk + e <= last[t] && vk + e < end && vp >= 0 ? w[e] : kNone;
                    top = fmaxf(top, w[e]);
                }
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float mn = fmaxf(m[t], top);
                // nothing seen yet: any finite number will do, all weights are 0
                const float mz = mn == kNone ? 0.0f : mn;
                const float f = __builtin_amdgcn_exp2f(m[t] - mz);
                m[t] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = __builtin_amdgcn_exp2f(w[e] - mz + Parts<T>::up);
                    sum += w[e];
                }
                l[t] = l[t] * f + sum;
                v8 pf[NP];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float rest = w[e];
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        pf[p][e] = (T)rest;
                        rest -= (float)pf[p][e];
                    }
                }
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    o[t][d] *= f;
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
                        o[t][d] = Num<CT>::mfma16(vf[d], pf[p], o[t][d]);
                }
            }
        }
        // ---- the four wavefronts' sums become one; l over the lane's key groups first
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            l[t] += __shfl_xor(l[t], 16, 64);
            l[t] += __shfl_xor(l[t], 32, 64);
            if (q4 == 0) {
                sm[wave][t][c16] = m[t];
                sl[wave][t][c16] = l[t];
            }
        }
        __syncthreads();
        float mt[NT], lt[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mt[t] = kNone;
            for (int w = 0; w < kAttnWaves; ++w)
                mt[t] = fmaxf(mt[t], sm[w][t][c16]);
            const float mz = mt[t] == kNone ? 0.0f : mt[t];
            lt[t] = 0.0f;
            for (int w = 0; w < kAttnWaves; ++w)
                lt[t] += sl[w][t][c16] * __builtin_amdgcn_exp2f(sm[w][t][c16] - mz);
            const float f = __builtin_amdgcn_exp2f(m[t] - mz);
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[t][d] *= f;
        }
        for (int w = 0; w < kAttnWaves; ++w) {
            if (wave == w) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        f32x4 *p = reinterpret_cast<f32x4 *>(&so[16 * t + c16][16 * d + 4 * q4]);
                        *p = w ? *p + o[t][d] : o[t][d];
                    }
            }
            __syncthreads();
        }
        // ---- out, or this chunk's part of it: [row][chunk][D] then [row][chunk] of (m, l)
        const int64_t all_rows = a.tokens * a.q_heads;
        float *po = static_cast<float *>(a.work);
        float2 *pm = reinterpret_cast<float2 *>(po + all_rows * g.p.chunks * D);
        for (int u = threadIdx.x; u < 16 * NT * (D / 8); u += 64 * kAttnWaves) {
            const int cr = u / (D / 8), d8 = u % (D / 8) * 8, r = r0 + cr;
            if (r >= rows)
                continue;
            const int64_t tok = rq.row0 + r / g.group;
            const int hq = kh * g.group + r % g.group;
            float v[8];
            load8(&so[cr][d8], v);
            if (g.p.chunks == 1) {
                float lt1 = 0.0f, mt1 = kNone;
                for (int w = 0; w < kAttnWaves; ++w)
                    mt1 = fmaxf(mt1, sm[w][cr >> 4][cr & 15]);
                const float mz = mt1 == kNone ? 0.0f : mt1;
                for (int w = 0; w < kAttnWaves; ++w)
                    lt1 += sl[w][cr >> 4][cr & 15] * __builtin_amdgcn_exp2f(sm[w][cr >> 4][cr & 15] - mz);
                const float inv = lt1 > 0.0f ? 1.0f / lt1 : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] *= inv;
                const int64_t at = tok * a.ld_out + (int64_t)hq * D + d8;
                if constexpr (F32)
                    store8(static_cast<float *>(a.out) + at, v);
                else
                    store8(static_cast<T *>(a.out) + at, v);
            } else {
                store8(po + ((tok * a.q_heads + hq) * g.p.chunks + chunk) * D + d8, v);
            }
        }
        if (g.p.chunks > 1 && wave == 0 && q4 == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int r = r0 + 16 * t + c16;
                if (r < rows) {
                    const int64_t at = (rq.row0 + r / g.group) * (int64_t)a.q_heads + kh * g.group + r % g.group;
                    pm[at * g.p.chunks + chunk] = make_float2(mt[t], lt[t]);
                }
            }
        }
        __syncthreads();
    }
}

// The chunks of a row added up: D / 8 lanes a row.
template <class OT, int D>
__global__ __launch_bounds__(256) void attn_join(const AttnArgs g)
{
    const bq_attn &a = g.a;
    constexpr int L = D / 8;
    const int64_t u = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
    const int d8 = threadIdx.x % L * 8;
    if (u >= a.tokens * a.q_heads)
        return;
    const int64_t tok = u / a.q_heads;
    const int hq = (int)(u % a.q_heads);
    const int b = request_of(a.cu, a.requests, (int)tok);
    if (b < 0)
        return;
    const float *po = static_cast<const float *>(a.work);
    const float2 *pm = reinterpret_cast<const float2 *>(po + a.tokens * a.q_heads * g.p.chunks * D);
    float m = kNone;
    for (int c = 0; c < g.p.chunks; ++c)
        m = fmaxf(m, pm[u * g.p.chunks + c].x);
    const float mz = m == kNone ? 0.0f : m;
    float l = 0.0f, o[8] = {};
    for (int c = 0; c < g.p.chunks; ++c) {
        const float2 ml = pm[u * g.p.chunks + c];
        const float f = __builtin_amdgcn_exp2f(ml.x - mz);
        float v[8];
        load8(po + (u * g.p.chunks + c) * D + d8, v);
        l = __builtin_fmaf(ml.y, f, l);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] = __builtin_fmaf(v[e], f, o[e]);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] *= inv;
    store8(static_cast<OT *>(a.out) + tok * a.ld_out + (int64_t)hq * D + d8, o);
}

AttnPlan attn_plan(const bq_attn &a)
{
    AttnPlan p;
    const int group = a.q_heads / a.cache.heads;
    const int64_t most = a.max_new < a.tokens ? a.max_new : a.tokens;
    const int64_t rows = most * group;
    p.nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.tiles = (int)((rows + 16 * p.nt - 1) / (16 * p.nt));
    // tiles that can have rows: no request has more than `tiles`, all together no more than the rows allow
    const int64_t all = a.tokens * group / (16 * p.nt) + a.requests;
    const int64_t busy = (p.tiles * (int64_t)a.requests < all ? p.tiles * (int64_t)a.requests : all) * a.cache.heads;
    int64_t chunks = (1024 + busy - 1) / busy;
    const int64_t step = kAttnKeys * kAttnWaves;
    const int64_t steps = (a.max_keys + step - 1) / step;
    chunks = chunks > steps ? steps : chunks;
    chunks = chunks < 1 ? 1 : chunks > 64 ? 64 : chunks;
    const int64_t each = (steps + chunks - 1) / chunks;
    p.chunk = (int)((each < 1 ? 1 : each) * step);
    p.chunks = (int)((steps + (each < 1 ? 1 : each) - 1) / (each < 1 ? 1 : each));
    p.chunks = p.chunks < 1 ? 1 : p.chunks;
    p.work_bytes = p.chunks > 1 ? a.tokens * a.q_heads * p.chunks * (4 * (int64_t)a.cache.dim + 8) : 0;
    return p;
}

template <int CT, int D, bool F32>
static void attn_nt(const AttnArgs &g, dim3 grid, hipStream_t st)
{
    switch (g.p.nt) {
    case 1: hipLaunchKernelGGL((attn_kernel<CT, D, 1, F32>), grid, dim3(64 * kAttnWaves), 0, st, g); break;
    case 2: hipLaunchKernelGGL((attn_kernel<CT, D, 2, F32>), grid, dim3(64 * kAttnWaves), 0, st, g); break;
    default: hipLaunchKernelGGL((attn_kernel<CT, D, 4, F32>), grid, dim3(64 * kAttnWaves), 0, st, g); break;
    }
}

template <int CT, int D>
static void attn_dim(const AttnArgs &g, dim3 grid, dim3 join, hipStream_t st)
{
    const bool f32 = g.a.type == BQ_F32;
    f32 ? attn_nt<CT, D, true>(g, grid, st) : attn_nt<CT, D, false>(g, grid, st);
    if (g.p.chunks > 1) {
        if (f32)
            hipLaunchKernelGGL((attn_join<float, D>), join, dim3(256), 0, st, g);
        else
            hipLaunchKernelGGL((attn_join<typename Num<CT>::t, D>), join, dim3(256), 0, st, g);
    }
}

hipError_t launch_attn(const bq_attn &a, const AttnPlan &p, hipStream_t st)
{
    AttnArgs g;
    g.a = a;
    g.p = p;
    g.group = a.q_heads / a.cache.heads;
    g.page_log2 = __builtin_ctz((unsigned)a.cache.page);
    const dim3 grid((unsigned)(p.tiles * p.chunks), (unsigned)a.cache.heads, (unsigned)a.requests);
    const dim3 join((unsigned)((a.tokens * a.q_heads * (a.cache.dim / 8) + 255) / 256));
    if (a.cache.type == BQ_F16)
        a.cache.dim == 64 ? attn_dim<BQ_F16, 64>(g, grid, join, st) : attn_dim<BQ_F16, 128>(g, grid, join, st);
    else
        a.cache.dim == 64 ? attn_dim<BQ_BF16, 64>(g, grid, join, st) : attn_dim<BQ_BF16, 128>(g, grid, join, st);
    return hipGetLastError();
}

}  // namespace bq
