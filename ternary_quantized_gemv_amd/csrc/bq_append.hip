// bq_append.hip -- new tokens into the paged cache (bq_kv_append): per-head
// norm, rotation by position, and the write of keys and transposed values.
//
// A rotation turns (v[i], v[i + rot/2]) by pos * freq[i].  The angle is formed
// in binary64 and reduced to a fraction of a turn there (a position of 10^6
// leaves 2^-32 of a turn), then sine and cosine of the remaining eighth turn
// either way are f32 series.  One workgroup computes them once for all heads
// of a token.  Memory bounds the prompt form (everything is read and written
// once), latency the single token.
//
// Measured: 2049 f16 tokens of 32 + 8 heads of 128 (50.4 MB) 12.7 us, 4.0
// TB/s; 16 f32 tokens 3.6 us.
#include <type_traits>

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
    int v_cols;      // workgroups per 64 tokens of the latter
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

// About 64 tokens, 64 value columns: a lane owns a column (head, index), a
// wavefront eight tokens at a time.  Eight tokens whose places are neighbours
// in a page, from a multiple of eight on, are one 16-byte store a lane; so the
// tile starts up to seven tokens early, where its first token's run has such a
// place, and takes up to seven more tokens than the 64 that its neighbours
// leave (what two tiles both take they write alike).  64 tokens because a
// page's row of them is a whole cache line then: one L2 has all its parts.
constexpr int kValueTokens = 64, kValueCols = 64;

template <class T, class C, int D>
__device__ __forceinline__ void append_v(const AppendArgs &g, int64_t block)
{
    const bq_append &a = g.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tile = block / g.v_cols * kValueTokens;
    const int col = (int)(block % g.v_cols) * kValueCols + lane;
    const int64_t places = a.cache.pages * a.cache.page;
    const int64_t start = a.slot[tile];
    const int64_t from = tile - (start > 0 ? start & 7 : 0);
    const int h = col / D, d = col % D;
    const T *src = static_cast<const T *>(a.v) + col;
    C *dst = static_cast<C *>(a.cache.v) + (int64_t)(h * D + d) * a.cache.page;
    const int64_t page_elems = (int64_t)a.cache.heads * D * a.cache.page;
    const int log2 = __builtin_ctz((unsigned)a.cache.page);
    for (int i = wave; i < kValueTokens / 8 + 1; i += kAppendThreads / 64) {
        const int64_t t0 = from + 8 * i;
        if (t0 >= a.tokens)
            break;
        T v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t t = t0 + e < 0 ? 0 : t0 + e < a.tokens ? t0 + e : a.tokens - 1;
            v[e] = src[t * a.ld_v];
        }
        // lanes 0 .. 7 (and every eighth of them again): the place of token t0 + lane % 8
        const int64_t t = t0 + (lane & 7);
        int64_t slot = t >= 0 && t < a.tokens ? a.slot[t] : -1;
        slot = slot < places ? slot : -1;
        const int64_t first = __shfl(slot, 0, 64);
        if (__all(first >= 0 && (first & 7) == 0 && slot == first + (lane & 7))) {
            C *p = dst + (first >> log2) * page_elems + (first & (a.cache.page - 1));
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = (float)v[e];
            store8(p, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t to = __shfl(slot, e, 64);
                if (to >= 0)
                    dst[(to >> log2) * page_elems + (to & (a.cache.page - 1))] = (C)(float)v[e];
            }
        }
    }
}

template <class T, class C, int D>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(const AppendArgs g)
{
    __shared__ float cs[128];
    if ((int)blockIdx.x < g.qk_blocks)
        append_qk<T, C, D>(g, cs);
    else
        append_v<T, C, D>(g, (int64_t)blockIdx.x - g.qk_blocks);
}

template <class T, class C>
static void append_dim(const AppendArgs &g, unsigned blocks, hipStream_t st)
{
    if (g.a.cache.dim == 64)
        hipLaunchKernelGGL((append_kernel<T, C, 64>), dim3(blocks), dim3(kAppendThreads), 0, st, g);
    else
        hipLaunchKernelGGL((append_kernel<T, C, 128>), dim3(blocks), dim3(kAppendThreads), 0, st, g);
}

static void append_slice(const bq_append &a, hipStream_t st)
{
    AppendArgs g;
    g.a = a;
    const int per_round = kAppendThreads / (a.cache.dim / 8);
    const int rounds = (a.q_heads + a.cache.heads + per_round - 1) / per_round;
    // few tokens: a workgroup per round of heads; many: all heads share one workgroup's angles
    g.splits = a.tokens < 512 ? rounds : 1;
    g.qk_blocks = (int)(a.tokens * g.splits);
    g.v_cols = a.cache.heads * a.cache.dim / kValueCols;
    const unsigned blocks = (unsigned)(g.qk_blocks + (a.tokens + kValueTokens - 1) / kValueTokens * g.v_cols);
    if (a.type == BQ_F32)
        a.cache.type == BQ_F16 ? append_dim<float, _Float16>(g, blocks, st) : append_dim<float, __bf16>(g, blocks, st);
    else if (a.type == BQ_F16)
        append_dim<_Float16, _Float16>(g, blocks, st);
    else
        append_dim<__bf16, __bf16>(g, blocks, st);
}

hipError_t launch_append(const bq_append &a, hipStream_t st)
{
    // a grid holds fewer than 2^32 threads: 2^17 tokens have at most 2^17 + 2^11 * 2048 workgroups
    const int64_t most = int64_t(1) << 17;
    auto rows = [](auto *p, int64_t elems, int type) {
        typedef std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(p)>>, const char, char> byte;
        return p ? static_cast<byte *>(p) + elems * (type == BQ_F32 ? 4 : 2) : nullptr;
    };
    for (int64_t t = 0; t < a.tokens; t += most) {
        bq_append s = a;
        s.tokens = a.tokens - t < most ? a.tokens - t : most;
        s.q = rows(a.q, t * a.ld_q, a.type);
        s.k = rows(a.k, t * a.ld_k, a.type);
        s.v = rows(a.v, t * a.ld_v, a.type);
        s.q_out = rows(a.q_out, t * a.ld_qo, a.q_out_type);
        s.pos = a.pos + t;
        s.slot = a.slot + t;
        append_slice(s, st);
    }
    return hipGetLastError();
}

}  // namespace bq
