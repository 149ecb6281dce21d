// bq_attn_tiles.hip -- attention of many new tokens (whole prompts, long
// chunks) over the paged cache: the arithmetic of bq_attn.hip with the keys
// shared through LDS.
//
// A workgroup of four or eight wavefronts takes 128 or 256 rows (G query heads
// of each token) of one key head, 32 columns a wavefront, and 64 keys at a time.
// The products are v_mfma_f32_32x32x16, again S^T = K Q^T and O^T = V^T P^T:
// result register r of lane l holds row 8 (r / 4) + 4 (l / 32) + r % 4 of column
// l % 32, and operands hold k = 8 (l / 32) + e.  Row 8 a + 4 h + i of a 32-key
// tile is assigned key 16 (a / 2) + 8 h + 4 (a % 2) + i, so that a lane's
// registers 8 s .. 8 s + 7 are keys 16 s + 8 h .. + 7: the B operand of the
// second product as they stand.  Both tiles lie in LDS in 16-byte pieces, turned
// within their rows so that the 16 lanes that a read serves at a time (16
// neighbouring rows) touch all 64 banks once.
//
// The running maximum is only raised when a tile's exceeds it by 2^8: until
// then the weights are at most 2^8 times larger than they would be, which
// changes no relative error, and the D sums of a column are not rescaled.
// (f16 weights are scaled by 2^6, which leaves room for that below 2^16.)
//
// The matrix cores bound it, with the exponentials in turn: 4 D operations per
// row and key, and a key's 4 D bytes are read from LDS once for 32 rows and from
// memory once for 128 or 256.  Measured: 512 bf16 tokens, 32 + 8 heads of 128, over
// 30011 keys 283 to 293 us, 855-884 TFLOP/s (a large matrix product: 1386); a
// prompt of 16384 tokens 2.39 ms, 921.  f32 rows make three (bf16 cache) or two
// (f16) times the products: the same chunk 776 and 652 us.
#include "bq_attn.h"

namespace bq {

constexpr int kTileKeys = 64;
constexpr float kSlack = 8.0f;  // log2

// Piece c of row r lies at c ^ turn(r) of its row of PIECES (16: one row fills
// the banks; 8: two rows do).  (512 bf16 tokens over 30011 keys: no bank conflict in
// 38.1 M LDS cycles; with r % 8 for both 30.5 M in 68.6 M.)
template <int PIECES>
__device__ __forceinline__ int turn(int r) { return PIECES == 16 ? r & 15 : (r >> 1) & 7; }

template <int CT, int D, int WAVES, bool F32>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4) void attn_tiles(const AttnArgs g)
{
    typedef typename Num<CT>::t T;
    typedef typename Num<CT>::v8 v8;
    constexpr int NP = F32 ? Parts<T>::n : 1;
    constexpr float UP = CT == BQ_F16 ? 6.0f : 0.0f;
    constexpr int THREADS = 64 * WAVES, ROWS = 32 * WAVES;
    constexpr int DJ = D / 16, DT = D / 32, KC = D / 8;  // steps and tiles of D; 16-byte pieces of a key
    // the wavefront of a SIMD that has products to issue goes first, the other's exponentials fill the gaps
    // (+2%; 5% slower where the products are three times as many, or half as long)
    constexpr bool FIRST = !F32 && D == 128;
    constexpr int BLOCKS = kTileKeys / 16;               // of 16 keys: one page each
    constexpr int KL = kTileKeys * KC / THREADS, VL = D * 8 / THREADS;  // pieces a thread stages
    constexpr int KROWS = THREADS / KC, VROWS = THREADS / 8;            // rows that one piece of each thread covers
    static_assert(KROWS % 16 == 0 && KL >= 1 && VL >= 1, "a thread's piece of keys stays in one 16-key block per 16 rows");
    __shared__ v8 ks[2][kTileKeys * KC];
    __shared__ v8 vs[2][D * 8];

    const bq_attn &a = g.a;
    const auto &sp = g.p.many;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c32 = lane & 31, half = lane >> 5;
    const int kh = blockIdx.x;
    const int chunk = blockIdx.y % sp.chunks;
    const int P = a.cache.page, pmask = P - 1;
    const int64_t page_elems = ((int64_t)a.cache.heads << g.page_log2) * D;
    const T *kbase = static_cast<const T *>(a.cache.k) + (int64_t)kh * P * D;
    const T *vbase = static_cast<const T *>(a.cache.v) + (int64_t)kh * D * P;

    // staging: a thread's pieces are piece kc of rows kr + KROWS i (keys) and piece vc of rows vr + VROWS i (values)
    const int kc = threadIdx.x % KC, kr = threadIdx.x / KC;
    const int vc = threadIdx.x % 8, vr = threadIdx.x / 8;

    auto tiles_of = [&](int i, int &) {
        int rows, keys;
        lane_request(g, i, false, rows, keys);
        return (rows + ROWS - 1) / ROWS;
    };
    Walk walk;
    int b, within, front;
    for (int item = blockIdx.y / sp.chunks; find_item<false>(walk, a.requests, item, b, within, front, tiles_of); item += sp.tiles) {
        const Request rq = request_at(a, b);
        const int32_t *table = a.table + (int64_t)b * a.ld_table;
        const int rows = rq.n * g.group;
        // the last tile first: it sees the most keys
        const int r0 = ((rows + ROWS - 1) / ROWS - 1 - within) * ROWS;
        const int r = r0 + wave * 32 + c32;
        const bool live = r < rows;
        const int i_tok = live ? r / g.group : 0, hq = kh * g.group + (live ? r % g.group : 0);
        const int last = live ? rq.keys - rq.n + i_tok : -1;
        float m = kNone, l = 0.0f;
        v8 qf[NP][DJ];
        const float qs = load_query<T, v8, NP, DJ, F32>(a, (int64_t)(rq.row0 + i_tok) * a.ld_q + (int64_t)hq * D + 8 * half, 16,
                                                        qf, [](float x) { return across32(x, Max()); });
        f32x16 o[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                o[d][e] = 0.0f;

        const int last_row = min(r0 + ROWS, rows) - 1;
        const int seen = min(rq.keys, rq.keys - rq.n + last_row / g.group + 1);
        // tiles past those that the launch and its scratch were made for are not split
        const bool split = sp.chunks > 1 && item < sp.tiles;
        if (sp.chunks > 1 && kh == 0 && chunk == 0 && within == 0 && threadIdx.x == 0)
            *note_tile(g, b) = item;
        if (!split && chunk)
            continue;
        const int begin = chunk * sp.chunk;
        const int end = !split || chunk == sp.chunks - 1 ? seen : min(seen, begin + sp.chunk);
        const int first_last = rq.keys - rq.n + r0 / g.group;

        // ---- staging of one tile: pages (one tile ahead), memory to registers, registers to LDS
        v8 kreg[KL], vreg[VL];
        int page[BLOCKS];
        auto look_up = [&](int k0) {
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i)
                page[i] = page_at(g, table, k0 + 16 * i, end);
        };
        int holes = 0, bad = 0;  // 16-key blocks of this (the next) tile without a page of the cache
        int vpage = -1;
        auto fetch = [&](int k0) {
            bad = 0;
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i)
                bad |= (page[i] < 0) << i;
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const int row = kr + KROWS * i, ri = row & 31;
                // row 8 a + 4 h + i of 32 is key 16 (a / 2) + 8 h + 4 (a % 2) + i
                const int key = k0 + (row & ~15) + 8 * ((ri >> 2) & 1) + 4 * ((ri >> 3) & 1) + (ri & 3);
                int p;
                if constexpr (KROWS == 16)
                    p = page[i];
                else  // the thread's 16-key block of KROWS / 16 neighbours
                    p = kr < 16 ? page[i * (KROWS / 16)] : KROWS == 32 || kr < 32 ? page[i * (KROWS / 16) + 1]
                        : kr < 48 ? page[(i * (KROWS / 16) + 2) % BLOCKS] : page[(i * (KROWS / 16) + 3) % BLOCKS];
                kreg[i] = *reinterpret_cast<const v8 *>(kbase + (int64_t)max(p, 0) * page_elems + (key & pmask) * D + 8 * kc);
            }
            vpage = vc < 2 ? page[0] : vc < 4 ? page[1] : vc < 6 ? page[2] : page[3];
            const T *p = vbase + (int64_t)max(vpage, 0) * page_elems + ((k0 + 8 * vc) & pmask);
#pragma unroll
            for (int i = 0; i < VL; ++i)
                vreg[i] = *reinterpret_cast<const v8 *>(p + (vr + VROWS * i) * P);
        };
        auto stage = [&](int k0, int buf) {
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const int row = kr + KROWS * i;
                ks[buf][row * KC + (kc ^ turn<KC>(row))] = kreg[i];
            }
            if (k0 + kTileKeys > end || bad) {
                // places that no row sees may hold anything: their values must not meet a weight of 0
#pragma unroll
                for (int i = 0; i < VL; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        vreg[i][e] = k0 + 8 * vc + e < end && vpage >= 0 ? vreg[i][e] : (T)0.0f;
            }
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int row = vr + VROWS * i;
                vs[buf][row * 8 + (vc ^ turn<8>(row))] = vreg[i];
            }
        };

        int buf = 0;
        if (begin < end) {
            look_up(begin);
            fetch(begin);
            look_up(begin + kTileKeys);
            stage(begin, 0);
            holes = bad;
            __syncthreads();
        }
        for (int k0 = begin; k0 < end; k0 += kTileKeys) {
            const int next = k0 + kTileKeys;
            if (next < end) {
                fetch(next);
                look_up(next + kTileKeys);
            }
            const bool whole = k0 + kTileKeys - 1 <= first_last && k0 + kTileKeys <= end && !holes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // ---- scores
                f32x16 s;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    s[e] = 0.0f;
                const int krow = 32 * h + c32;
                if (FIRST)
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int j = 0; j < DJ; ++j) {
                    const v8 kf = ks[buf][krow * KC + ((2 * j + half) ^ turn<KC>(krow))];
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
                        s = Num<CT>::mfma32(kf, qf[p][j], s);
                }
                if (FIRST)
                    __builtin_amdgcn_s_setprio(0);
                // ---- weights
                float factor = qs, top = kNone;
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int key = k0 + 32 * h + 16 * (e >> 3) + 8 * half + (e & 7);
                        const bool sees = key <= last && key < end && !(holes >> (2 * h + (e >> 3)) & 1);
                        s[e] = sees ? s[e] * factor : kNone;
                    }
                    factor = 1.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    top = fmaxf(top, s[e]);
                top = across32(top, Max()) * factor;
                if (__any(top > m + kSlack)) {
                    const float mn = fmaxf(m, top);
                    const float f = __builtin_amdgcn_exp2f(m - (mn == kNone ? 0.0f : mn));
                    m = mn;
                    l *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        o[d] *= f;
                }
                const float shift = UP - (m == kNone ? 0.0f : m);
                float sum = 0.0f;
                v8 pf[NP][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + e], factor, shift));
                        sum += w[e];
                    }
                    v8 part[NP];
                    Split<T, NP>::parts(w, part);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        pf[p][k] = part[p];
                }
                l += sum;
                // ---- values
                if (FIRST)
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const int row = 32 * d + c32;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const v8 vf = vs[buf][row * 8 + ((4 * h + 2 * k + half) ^ turn<8>(row))];
#pragma unroll
                        for (int p = NP - 1; p >= 0; --p)
                            o[d] = Num<CT>::mfma32(vf, pf[p][k], o[d]);
                    }
                }
                if (FIRST)
                    __builtin_amdgcn_s_setprio(0);
            }
            if (next < end) {
                stage(next, buf ^ 1);
                holes = bad;
            }
            __syncthreads();
            buf ^= 1;
        }
        // ---- out, or this chunk's part of it
        l = across32(l, Add());
        const int64_t tok = rq.row0 + i_tok;
        const Part part = many_part(g, D, kh, split ? item : 0, chunk, wave * 32 + c32);
        const float f = split ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int at = 32 * d + 8 * q + 4 * half;
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = o[d][4 * q + e] * f;
                if (!live) {
                } else if (split) {
                    *reinterpret_cast<f32x4 *>(part.sums + at) = v;
                } else if constexpr (F32) {
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + tok * a.ld_out + (int64_t)hq * D + at) = v;
                } else {
                    typedef T tx4 __attribute__((ext_vector_type(4)));
                    tx4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = (T)v[e];
                    *reinterpret_cast<tx4 *>(static_cast<T *>(a.out) + tok * a.ld_out + (int64_t)hq * D + at) = x;
                }
            }
        if (live && split && half == 0)
            *part.stats = make_float2(m, l);
    }
}

template <int CT, int D>
static void tiles_dim(const AttnArgs &g, dim3 grid, hipStream_t st)
{
    if (g.a.type == BQ_F32)
        hipLaunchKernelGGL((attn_tiles<CT, D, 4, true>), grid, dim3(256), 0, st, g);
    else if (g.p.many.cols == 128)
        hipLaunchKernelGGL((attn_tiles<CT, D, 4, false>), grid, dim3(256), 0, st, g);
    else
        hipLaunchKernelGGL((attn_tiles<CT, D, 8, false>), grid, dim3(512), 0, st, g);
}

hipError_t launch_attn_tiles(const AttnArgs &g, hipStream_t st)
{
    const bq_attn &a = g.a;
    const dim3 grid((unsigned)a.cache.heads, (unsigned)(g.p.many.tiles * g.p.many.chunks));
    if (a.cache.type == BQ_F16)
        a.cache.dim == 64 ? tiles_dim<BQ_F16, 64>(g, grid, st) : tiles_dim<BQ_F16, 128>(g, grid, st);
    else
        a.cache.dim == 64 ? tiles_dim<BQ_BF16, 64>(g, grid, st) : tiles_dim<BQ_BF16, 128>(g, grid, st);
    return hipGetLastError();
}

}  // namespace bq
