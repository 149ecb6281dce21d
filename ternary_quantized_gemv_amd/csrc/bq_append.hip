// bq_append.hip -- new tokens into the paged cache (bq_kv_append): per-head
// norm, rotation by position, and the write of keys and transposed values.
//
// A rotation turns (v[i], v[i + rot/2]) by pos * freq[i].  The angle is formed
// in binary64 and reduced to a fraction of a turn there (a position of 10^6
// leaves 2^-32 of a turn), then sine and cosine of the remaining eighth turn
// either way are f32 series.  One workgroup computes them once for all heads
// of a token.  Memory bounds the prompt form (everything is read and written
// once), latency the single token.
#include "bq_half.h"
#include "bq_layer.h"

namespace bq {

constexpr int kAppendThreads = 256;

// cos and sin of pos * freq.  |x| <= pi/4 after the reduction; the first term
// left out of each series is below 2^-28 of the result.
__device__ __forceinline__ void cos_sin(int pos, float freq, float &c, float &s)
{
    const double turns = (double)pos * (double)freq * 0.15915494309189533577;  // 1 / (2 pi)
    const double part = turns - __builtin_rint(turns);                         // exact, in [-1/2, 1/2]
    const double quarter = __builtin_rint(4.0 * part);
    const float x = (float)((part - 0.25 * quarter) * 6.283185307179586477);
    const float z = x * x;
    float ps = __builtin_fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
    ps = __builtin_fmaf(z, ps, 1.0f / 120.0f);
    ps = __builtin_fmaf(z, ps, -1.0f / 6.0f);
    const float sx = __builtin_fmaf(x * z, ps, x);
    float pc = __builtin_fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    pc = __builtin_fmaf(z, pc, -1.0f / 720.0f);
    pc = __builtin_fmaf(z, pc, 1.0f / 24.0f);
    pc = __builtin_fmaf(z, pc, -0.5f);
    const float cx = __builtin_fmaf(z, pc, 1.0f);
    const int k = (int)quarter & 3;
    const float a = (k & 1) ? sx : cx, b = (k & 1) ? cx : sx;
    c = (k == 1 || k == 2) ? -a : a;
    s = (k & 2) ? -b : b;
}

struct AppendArgs {
    bq_append a;
    int qk_blocks;   // workgroups of the query and key heads, then those of the values
    int splits;      // workgroups per token of the former
    int v_cols;      // workgroups per eight tokens of the latter
};

// 8 values a lane, D / 8 neighbouring lanes a head.  T: type of the rows, C: of the cache.
template <class T, class C, int D>
__device__ __forceinline__ void append_qk(const AppendArgs &g, float *cs)
{
    const bq_append &a = g.a;
    constexpr int L = D / 8, HEADS = kAppendThreads / L;
    const int64_t t = blockIdx.x / g.splits;
    const int part = blockIdx.x % g.splits;
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += kAppendThreads)
        cos_sin(a.pos[t], a.freq[i], cs[i], cs[64 + i]);
    __syncthreads();
    const int li = threadIdx.x % L, hl = half / 8;
    const int64_t slot = a.slot[t];
    const bool cached = slot >= 0 && slot < a.cache.pages * a.cache.page;
    const int H = a.cache.heads, total = a.q_heads + H;
    for (int h0 = part * HEADS; h0 < total; h0 += g.splits * HEADS) {
        const int h = h0 + threadIdx.x / L;
        const bool live = h < total, is_q = h < a.q_heads;
        float v[8] = {};
        if (live) {
            const T *p = is_q ? static_cast<const T *>(a.q) + t * a.ld_q + (int64_t)h * D
                              : static_cast<const T *>(a.k) + t * a.ld_k + (int64_t)(h - a.q_heads) * D;
            load8(p + 8 * li, v);
        }
        const float *w = is_q ? a.q_norm : a.k_norm;
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            ss = __builtin_fmaf(v[e], v[e], ss);
#pragma unroll
        for (int off = 1; off < L; off <<= 1)
            ss += __shfl_xor(ss, off, 64);
        if (live && w) {
            const float r = 1.0f / __builtin_sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = v[e] * r * w[8 * li + e];
        }
        if (half) {
            const bool low = li < hl, turned = li < 2 * hl;
            const int other = (threadIdx.x & 63) + (low ? hl : turned ? -hl : 0);
            const int i0 = 8 * (low ? li : turned ? li - hl : 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl(v[e], other, 64);
                const float c = cs[i0 + e], s = cs[64 + i0 + e];
                // low: v1 c - v2 s; high: v2 c + v1 s
                const float n = __builtin_fmaf(v[e], c, low ? -(o * s) : o * s);
                v[e] = turned ? n : v[e];
            }
        }
        if (!live)
            continue;
        if (is_q) {
            const int64_t at = t * a.ld_qo + (int64_t)h * D + 8 * li;
            if (a.q_out_type == a.type)
                store8(static_cast<T *>(a.q_out) + at, v);
            else
                store8(static_cast<C *>(a.q_out) + at, v);
        } else if (cached) {
            const int64_t page = slot / a.cache.page, off = slot % a.cache.page;
            store8(static_cast<C *>(a.cache.k) + ((page * H + (h - a.q_heads)) * a.cache.page + off) * D + 8 * li, v);
        }
    }
}

// Eight tokens, 256 value columns: a thread owns one column (head, index).
// Eight tokens whose places are neighbours in a page, from a multiple of
// eight on, are one 16-byte store; the workgroup with the first of them makes
// it and those of the others leave them out.
template <class T, class C, int D>
__device__ __forceinline__ void append_v(const AppendArgs &g, int64_t block, int *how)
{
    const bq_append &a = g.a;
    const int64_t t0 = block / g.v_cols * 8;
    const int col = (int)(block % g.v_cols) * kAppendThreads + threadIdx.x;
    const int64_t places = a.cache.pages * a.cache.page;
    if (threadIdx.x < 8) {
        const int64_t t = t0 + threadIdx.x;
        int f = 0;  // nothing to store
        if (t < a.tokens) {
            const int64_t slot = a.slot[t];
            if (slot >= 0 && slot < places) {
                const int64_t first = t - (slot & 7);
                bool run = first >= 0 && first + 8 <= a.tokens;
                for (int i = 0; i < 8 && run; ++i)
                    run = a.slot[first + i] == (slot & ~(int64_t)7) + i;
                f = !run ? 1 : (slot & 7) == 0 ? 2 : 0;
            }
        }
        how[threadIdx.x] = f;
    }
    __syncthreads();
    if (col >= a.cache.heads * D)
        return;
    const int h = col / D, d = col % D;
    const T *src = static_cast<const T *>(a.v) + col;
    for (int i = 0; i < 8; ++i) {
        const int f = how[i];
        if (!f)
            continue;
        const int64_t t = t0 + i, slot = a.slot[t];
        const int64_t page = slot / a.cache.page, off = slot % a.cache.page;
        C *dst = static_cast<C *>(a.cache.v) + ((page * a.cache.heads + h) * D + d) * a.cache.page + off;
        if (f == 1) {
            *dst = (C)(float)src[t * a.ld_v];
        } else {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (float)src[(t + e) * a.ld_v];
            store8(dst, v);
        }
    }
}

template <class T, class C, int D>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(const AppendArgs g)
{
    __shared__ float cs[128];
    __shared__ int how[8];
    if ((int)blockIdx.x < g.qk_blocks)
        append_qk<T, C, D>(g, cs);
    else
        append_v<T, C, D>(g, (int64_t)blockIdx.x - g.qk_blocks, how);
}

template <class T, class C>
static void append_dim(const AppendArgs &g, unsigned blocks, hipStream_t st)
{
    if (g.a.cache.dim == 64)
        hipLaunchKernelGGL((append_kernel<T, C, 64>), dim3(blocks), dim3(kAppendThreads), 0, st, g);
    else
        hipLaunchKernelGGL((append_kernel<T, C, 128>), dim3(blocks), dim3(kAppendThreads), 0, st, g);
}

hipError_t launch_append(const bq_append &a, hipStream_t st)
{
    AppendArgs g;
    g.a = a;
    const int per_round = kAppendThreads / (a.cache.dim / 8);
    const int rounds = (a.q_heads + a.cache.heads + per_round - 1) / per_round;
    // few tokens: a workgroup per round of heads; many: all heads share one workgroup's angles
    g.splits = a.tokens < 512 ? rounds : 1;
    g.qk_blocks = (int)(a.tokens * g.splits);
    g.v_cols = (a.cache.heads * a.cache.dim + kAppendThreads - 1) / kAppendThreads;
    const unsigned blocks = (unsigned)(g.qk_blocks + (a.tokens + 7) / 8 * g.v_cols);
    if (a.type == BQ_F32)
        a.cache.type == BQ_F16 ? append_dim<float, _Float16>(g, blocks, st) : append_dim<float, __bf16>(g, blocks, st);
    else if (a.type == BQ_F16)
        append_dim<_Float16, _Float16>(g, blocks, st);
    else
        append_dim<__bf16, __bf16>(g, blocks, st);
    return hipGetLastError();
}

}  // namespace bq
