// bq_attn.hip -- attention of few new tokens over the paged cache, and the join
// of split keys (bq_paged_attn; whole prompts and long chunks are in
// bq_attn_tiles.hip).
//
// o_r = sum_j exp(scale q_r.k_j - m_r) v_j / sum_j exp(scale q_r.k_j - m_r) in
// one pass over the keys, with a running maximum m_r and sum l_r per row.  The
// rows of one key head are its G query heads of each new token, row r = i G + g
// of token i: all of them see nearly the same keys, so a key is read once for
// up to 16 NT rows.
//
// A wavefront takes 32 keys at a time and computes the transposed products
// S^T = K Q^T and O^T = V^T P^T, rows of the result along keys (values), columns
// along rows r.  Result row 4 g + i of 16-key tile t is assigned key
// 8 g + 4 t + i (g = lane / 16): a lane then holds the scores of keys 8 g .. 8 g
// + 7 of its column, which is exactly the second product's B operand, and the
// transposed value pages give its A operand as one 16-byte load.  So scores,
// weights and sums never leave the lane's registers, m and l are two values
// per lane, and the keys go straight from memory to the matrix cores.
//
// f32 rows: q and the weights are split into 16-bit parts whose products with
// the cache are exact and add up in f32 (three of bf16, 24 bits; two of f16, 22
// bits, q scaled by a power of two per row).  f16 weights are scaled by 2^14 in
// either case, so that small ones stay clear of f16's subnormals.
//
// 16-bit rows: the weights are rounded to that type once, l sums them in f32
// before.  Each is off by half a step of the type at most, as out is by its own
// rounding, and over many keys they average out: relative to the formula in 64
// bits, in the mean square, bf16 decode rows 1.8e-3 and chunks 2.3e-3, of which
// out's rounding alone is 1.7e-3.  Two parts would double the second product.
//
// Memory bounds it: 2 D values a key and head, read once.  Measured with 8 key
// heads of 128: 64 requests of 8192 keys 329 us a call, 6.5 TB/s (a streaming
// read: 7.1); 32 bf16 requests of 3 to 8192 keys 52 us and the join 4.9; 16 bf16
// tokens over 16384 keys 22 + 5.2; one token of f32 rows over 8191 keys 12.5 +
// 4.5, of which the keys are 5: lengths, table, keys and sums come one behind
// the other.
#include "bq_attn.h"

namespace bq {

constexpr int kAttnKeys = 32;   // keys of a wavefront at a time
constexpr int kAttnStep = 128;  // keys that a workgroup's wavefronts take at most at a time
constexpr int kMaxChunks = 128; // pieces of a row's keys that the joins take

// ---- the split of the keys, from the lengths of all requests
//
// Requests of very different lengths would leave some compute units with long
// ones and others with none (pieces of a fixed number of keys, empty ones
// among them: 75 us against 61 for 32 requests of 3 to 8192 keys), so every
// workgroup derives the same equal cut from the lengths: units of 128 keys,
// `chunk` of them a piece, so that the pieces are about few.items per key head
// and at most kMaxChunks per row.

// Tiles of rows and units of keys; a request without keys has one piece, of zeros.
__device__ __forceinline__ int few_tiles(const AttnArgs &g, int rows) { return (rows + g.p.few.cols - 1) / g.p.few.cols; }
__device__ __forceinline__ int few_units(int keys) { return keys > kAttnStep ? (keys + kAttnStep - 1) / kAttnStep : 1; }

// Units of a piece: those of all requests over the pieces wanted, and, as every
// request rounds its pieces up, more where that made too many (twice: pieces
// that fill the GPU once and a third take as long as two fillings; not for so
// many requests that they even out).  The sums are f32, the same in every
// workgroup and within 2^-13 (at most 1024 + 6 additions): with at most 1536
// places, the split pieces stay below 2 few.items + 1/2, so within them.
__device__ __forceinline__ int few_chunk(const AttnArgs &g)
{
    const int lane = threadIdx.x & 63;
    const float want = (float)g.p.few.items;
    float total = 0.0f;
    int most = 1, tiles = 0, units = 1;
    if (g.a.requests == 1) {  // a single token waits for every load in a row: scalar ones, and few
        const Request rq = request_at(g.a, 0);
        tiles = rq.n > 0 && has_few(g.p, rq.n * g.group) ? few_tiles(g, rq.n * g.group) : 0;
        most = few_units(rq.keys);
        total = (float)tiles * (float)most;
    }
#pragma unroll 4
    for (int base = 0; base < g.a.requests && g.a.requests > 1; base += 64) {
        int rows = 0, keys = 0;
        if (base + lane < g.a.requests)
            lane_request(g, base + lane, true, rows, keys);
        tiles = few_tiles(g, rows);
        units = few_units(keys);
        total += (float)tiles * (float)units;
        most = max(most, tiles ? units : 1);
    }
    if (g.a.requests > 1) {
        total = wave_all(total, Add());
        most = (int)wave_all((float)most, Max());  // at most 2^24: exact
    }
    const int least = (most + kMaxChunks - 1) / kMaxChunks;
    int chunk = max((int)fminf(__builtin_ceilf(total / want), 16777216.0f), least);
    if (g.a.requests > 1 && g.a.requests <= 64 && total > want) {
        for (int again = 0; again < 2; ++again) {
            const float count = wave_all((float)(tiles * ((units + chunk - 1) / chunk)), Add());
            if (count > want)
                chunk = max(min((int)fminf(__builtin_ceilf((float)chunk * (count / want)), 16777216.0f), most), chunk);
        }
    }
    return __builtin_amdgcn_readfirstlane(g.p.few.split ? chunk : max(chunk, most));
}

// CW of the W wavefronts take 16 NT columns each, the others the same columns
// over other keys.
template <int CT, int D, int NT, int CW, int W, bool F32>
__global__ __launch_bounds__(64 * W, NT == 1 && !F32 ? 3 : 2) void attn_kernel(const AttnArgs g)
{
    typedef typename Num<CT>::t T;
    typedef typename Num<CT>::v8 v8;
    constexpr int NP = F32 ? Parts<T>::n : 1;
    constexpr int DJ = D / 32, DT = D / 16;
    constexpr int KW = W / CW, COLS = 16 * NT * CW;  // wavefronts along the keys, rows of a tile
    __shared__ float sm[KW][COLS], sl[KW][COLS];
    __shared__ float so[KW][COLS][D + 4];

    const bq_attn &a = g.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cw = wave % CW, kw = wave / CW;
    const int c16 = lane & 15, q4 = lane >> 4;
    const int kh = blockIdx.x;
    const int64_t page_elems = ((int64_t)a.cache.heads << g.page_log2) * D;
    const int P = a.cache.page, pmask = P - 1;
    // K: this lane reads key 8 (c16 / 4) + c16 % 4 (+ 4); V: keys 8 q4 .. 8 q4 + 7
    const int kofs = 8 * (c16 >> 2), vofs = 8 * q4;
    const T *kbase = static_cast<const T *>(a.cache.k) + (int64_t)kh * P * D + 8 * q4 + (c16 & 3) * D;
    const T *vbase = static_cast<const T *>(a.cache.v) + (int64_t)(kh * D + c16) * P;
    const int chunk_units = few_chunk(g);
    if (g.p.few.split && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *note_units(g) = chunk_units;
    // the pieces of all requests, and those of split ones, which have places in the scratch
    auto pieces = [&](int i, int &placed) {
        int rows, keys;
        lane_request(g, i, true, rows, keys);
        const int chunks = (few_units(keys) + chunk_units - 1) / chunk_units, n = few_tiles(g, rows) * chunks;
        placed = chunks > 1 ? n : 0;
        return n;
    };
    Walk walk;
    int b = 0, within = 0, front = 0;
    auto find = [&](int item) {
        if (a.requests > 1)
            return find_item<true>(walk, a.requests, item, b, within, front, pieces);
        const Request rq = request_at(a, 0);
        const int rows = rq.n > 0 && has_few(g.p, rq.n * g.group) ? rq.n * g.group : 0;
        within = item;
        return item < few_tiles(g, rows) * ((few_units(rq.keys) + chunk_units - 1) / chunk_units);
    };
    for (int item = blockIdx.y; find(item); item += gridDim.y) {
        const Request rq = request_at(a, b);
        const int rows = rq.n * g.group, tiles = few_tiles(g, rows), units = few_units(rq.keys);
        // a request's pieces are as even as its units allow
        const int chunks = (units + chunk_units - 1) / chunk_units, keys = (units + chunks - 1) / chunks * kAttnStep;
        const int chunk = within / tiles, r0 = (within - chunk * tiles) * COLS;
        if (chunks > 1 && kh == 0 && within == 0 && threadIdx.x == 0)
            *note_piece(g, b) = front;
        const int32_t *table = a.table + (int64_t)b * a.ld_table;
        // ---- the keys: those that the tile's last row sees, this workgroup's chunk of them
        const int last_row = min(r0 + COLS, rows) - 1;
        const int seen = min(rq.keys, rq.keys - rq.n + last_row / g.group + 1);
        const int begin = chunk * keys;
        const int end = min(seen, begin + keys);
        const int first_last = rq.keys - rq.n + r0 / g.group;  // the last key that the tile's first row sees

        // pages one step ahead of the keys, keys and values one product ahead of their use
        v8 kf[2][DJ], vf[DT];
        auto load_k = [&](int at, int page0, int page1) {
            const int page = max(c16 < 8 ? page0 : page1, 0);
            const T *p = kbase + (int64_t)page * page_elems + ((at + kofs) & pmask) * D;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < DJ; ++j)
                    kf[t][j] = stream8<v8, CW == 1>(p + 4 * t * D + 32 * j);
        };
        auto load_v = [&](int at, int page0, int page1) {
            const int page = max(q4 < 2 ? page0 : page1, 0);
            const T *p = vbase + (int64_t)page * page_elems + ((at + vofs) & pmask);
#pragma unroll
            for (int d = 0; d < DT; ++d)
                vf[d] = stream8<v8, CW == 1>(p + 16 * d * P);
        };
        int k0 = begin + kAttnKeys * kw;
        int p0 = page_at(g, table, k0, end), p1 = page_at(g, table, k0 + 16, end);
        constexpr int STEP = kAttnKeys * KW;
        int n0 = page_at(g, table, k0 + STEP, end), n1 = page_at(g, table, k0 + STEP + 16, end);
        if (k0 < end) {
            load_k(k0, p0, p1);
            load_v(k0, p0, p1);
        }
        // ---- the rows, behind the first keys in the queue of loads: this lane's columns are rows c0 + 16 t + c16
        const int c0 = r0 + 16 * NT * cw;
        v8 qf[NT][NP][DJ];
        float qs[NT], m[NT], l[NT];
        int last[NT];  // the last key the column sees
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = c0 + 16 * t + c16;
            const bool live = r < rows;
            const int i = live ? r / g.group : 0, hq = kh * g.group + (live ? r % g.group : 0);
            last[t] = live ? rq.keys - rq.n + i : -1;
            m[t] = kNone;
            l[t] = 0.0f;
            qs[t] = load_query<T, v8, NP, DJ, F32>(a, (int64_t)(rq.row0 + i) * a.ld_q + (int64_t)hq * D + 8 * q4, 32, qf[t],
                                                   [](float x) { return across32(across16(x, Max()), Max()); });
        }
        f32x4 o[NT][DT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[t][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        while (k0 < end) {
            const int next = k0 + STEP;
            const bool whole = k0 + kAttnKeys - 1 <= first_last && k0 + kAttnKeys <= end && p0 >= 0 && p1 >= 0;
            const bool here = (q4 < 2 ? p0 : p1) >= 0;  // this lane's keys have a page
            f32x4 s[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[t][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int j = 0; j < DJ; ++j)
                            s[t][h] = Num<CT>::mfma16(kf[h][j], qf[t][p][j], s[t][h]);
                }
            if (next < end)
                load_k(next, n0, n1);
            if (!whole) {
                // places that no row sees may hold anything: their values must not meet a weight of 0
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        vf[d][e] = k0 + vofs + e < end && here ? vf[d][e] : (T)0.0f;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float w[8], factor = qs[t], top = kNone;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = s[t][e >> 2][e & 3];
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int key = k0 + vofs + e;
                        w[e] = key <= last[t] && key < end && here ? w[e] * factor : kNone;
                    }
                    factor = 1.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, w[e]);
                top = across32(across16(top, Max()), Max()) * factor;
                if (__any(top > m[t])) {
                    const float mn = fmaxf(m[t], top);
                    const float f = __builtin_amdgcn_exp2f(m[t] - (mn == kNone ? 0.0f : mn));
                    m[t] = mn;
                    l[t] *= f;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        o[t][d] *= f;
                }
                // nothing seen yet: any finite number will do, all weights are 0
                const float shift = Parts<T>::up - (m[t] == kNone ? 0.0f : m[t]);
                v8 pf[NP];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[e], factor, shift));
                    l[t] += w[e];
                }
                Split<T, NP>::parts(w, pf);
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
                        o[t][d] = Num<CT>::mfma16(vf[d], pf[p], o[t][d]);
            }
            if (next < end)
                load_v(next, n0, n1);
            p0 = n0;
            p1 = n1;
            n0 = page_at(g, table, next + STEP, end);
            n1 = page_at(g, table, next + STEP + 16, end);
            k0 = next;
        }
        // ---- the sums of the wavefronts along the keys become one; l over the lane's key groups first
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            l[t] = across32(across16(l[t], Add()), Add());
            const int col = 16 * (NT * cw + t) + c16;
            if (q4 == 0) {
                sm[kw][col] = m[t];
                sl[kw][col] = l[t];
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
                *reinterpret_cast<f32x4 *>(&so[kw][col][16 * d + 4 * q4]) = o[t][d];
        }
        __syncthreads();
        // ---- out, or this chunk's part of it
        for (int u = threadIdx.x; u < COLS * (D / 8); u += 64 * W) {
            const int cr = u / (D / 8), d8 = u % (D / 8) * 8, r = r0 + cr;
            if (r >= rows)
                continue;
            const int64_t tok = rq.row0 + r / g.group;
            const int hq = kh * g.group + r % g.group;
            float v[8] = {}, mt = kNone, lt = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w)
                mt = fmaxf(mt, sm[w][cr]);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const float f = __builtin_amdgcn_exp2f(sm[w][cr] - (mt == kNone ? 0.0f : mt));
                float x[8];
                load8(&so[w][cr][d8], x);
                lt = __builtin_fmaf(sl[w][cr], f, lt);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = __builtin_fmaf(x[e], f, v[e]);
            }
            if (chunks == 1) {
                const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] *= inv;
                const int64_t at = tok * a.ld_out + (int64_t)hq * D + d8;
                if constexpr (F32)
                    store8(static_cast<float *>(a.out) + at, v);
                else
                    store8(static_cast<T *>(a.out) + at, v);
            } else {
                const Part part = few_part(g, D, kh, front + within, cr);
                store8(part.sums + d8, v);
                if (d8 == 0)
                    *part.stats = make_float2(mt, lt);
            }
        }
        __syncthreads();
    }
}

// The pieces of a request of few rows added up, a workgroup a row: the lanes of a wavefront
// hold the pieces' statistics, then D / 8 threads take every
// 256 / (D / 8)-th piece's sums and add up through LDS, always in that order.
template <class OT, int D>
__global__ __launch_bounds__(256) void attn_join_few(const AttnArgs g)
{
    const bq_attn &a = g.a;
    constexpr int L = D / 8, GROUPS = 256 / L, MOST = kMaxChunks / GROUPS;
    __shared__ float weight[kMaxChunks];
    __shared__ float so[GROUPS][D + 4];
    const int lane = threadIdx.x & 63;
    // all that the rest hangs on in one go (notes of a request that has none are not used)
    const int chunk_units = uniform_word(note_units(g)), first = uniform_word(note_piece(g, blockIdx.y));
    const Request rq = request_at(a, blockIdx.y);
    asm volatile("" ::"s"(chunk_units), "s"(first));
    if (rq.n <= 0 || !has_few(g.p, rq.n * g.group) || (int64_t)blockIdx.x >= (int64_t)rq.n * a.q_heads)
        return;
    const int chunks = (few_units(rq.keys) + chunk_units - 1) / chunk_units;
    if (chunks <= 1)
        return;
    const int tiles = few_tiles(g, rq.n * g.group);
    const int grp = threadIdx.x / L, d8 = threadIdx.x % L * 8;
    for (int64_t u = blockIdx.x; u < (int64_t)rq.n * a.q_heads; u += gridDim.x) {
        // row i G + g of key head kh: tile and row of the tile; its pieces are `tiles` apart
        const int i = (int)(u / a.q_heads), hq = (int)(u - (int64_t)i * a.q_heads), kh = hq / g.group;
        const int r = i * g.group + hq - kh * g.group, tile = r / g.p.few.cols, cr = r - tile * g.p.few.cols;
        const float2 none = make_float2(kNone, 0.0f);
        // all loads first: a single token waits for little else
        float v[MOST][8];
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[k][e] = 0.0f;
            if (grp + GROUPS * k < chunks)
                load8(few_part(g, D, kh, first + (grp + GROUPS * k) * tiles + tile, cr).sums + d8, v[k]);
        }
        const float2 s0 = lane < chunks ? *few_part(g, D, kh, first + lane * tiles + tile, cr).stats : none;
        const float2 s1 = lane + 64 < chunks ? *few_part(g, D, kh, first + (lane + 64) * tiles + tile, cr).stats : none;
        float m = wave_all(fmaxf(s0.x, s1.x), Max());
        m = m == kNone ? 0.0f : m;
        const float f0 = __builtin_amdgcn_exp2f(s0.x - m), f1 = __builtin_amdgcn_exp2f(s1.x - m);
        const float l = wave_all(s0.y * f0 + s1.y * f1, Add());
        if (threadIdx.x < 64) {
            weight[lane] = f0;
            weight[lane + 64] = f1;
        }
        __syncthreads();
        float o[8] = {};
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const float f = weight[grp + GROUPS * k];  // 0 where there is no piece
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = __builtin_fmaf(v[k][e], f, o[e]);
        }
        store8(&so[grp][d8], o);
        __syncthreads();
        if (grp == 0) {
            const int groups = min(GROUPS, chunks);
            for (int k = 1; k < groups; ++k) {
                float x[8];
                load8(&so[k][d8], x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] += x[e];
            }
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] *= inv;
            store8(static_cast<OT *>(a.out) + (int64_t)(rq.row0 + i) * a.ld_out + (int64_t)hq * D + d8, o);
        }
        __syncthreads();
    }
}

// The pieces of requests of many rows added up: D / 8 lanes a row.
template <class OT, int D>
__global__ __launch_bounds__(256) void attn_join_many(const AttnArgs g)
{
    const bq_attn &a = g.a;
    constexpr int L = D / 8;
    const int64_t row = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x) / L;
    const int d8 = threadIdx.x % L * 8, chunks = g.p.many.chunks;
    if (row >= a.tokens * a.q_heads)
        return;
    const int64_t tok = row / a.q_heads;
    const int b = request_of(a.cu, a.requests, (int)tok);
    if (b < 0)
        return;
    const Rows mine = rows_between(a.cu[b], a.cu[b + 1], a.tokens);
    const int n = mine.n;
    if (n <= 0 || has_few(g.p, n * g.group))
        return;
    // the row's tile, counted from the request's last, and its row there; tiles past the scratch are not split
    const int hq = (int)(row - tok * a.q_heads), kh = hq / g.group, cols = g.p.many.cols;
    const int r = (int)(tok - mine.first) * g.group + hq - kh * g.group, tiles = (n * g.group + cols - 1) / cols;
    const int tile = *note_tile(g, b) + tiles - 1 - r / cols;
    if (tile >= g.p.many.tiles)
        return;
    const Part first = many_part(g, D, kh, tile, 0, r % cols);  // the next chunk's sums are cols rows on
    const float *sums = first.sums + d8;
    const float2 *stats = first.stats;
    float m = kNone;
    for (int c = 0; c < chunks; ++c)
        m = fmaxf(m, stats[c].x);
    m = m == kNone ? 0.0f : m;
    float l = 0.0f, o[8] = {};
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
        const float2 st = stats[c];
        const float f = __builtin_amdgcn_exp2f(st.x - m);
        float v[8];
        load8(sums + (int64_t)c * cols * D, v);
        l = __builtin_fmaf(st.y, f, l);
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
    const int64_t group = a.q_heads / a.cache.heads, heads = a.cache.heads;
    const int64_t most = a.max_new < a.tokens ? a.max_new : a.tokens;
    const int64_t rows = most * group;
    p.few.cols = p.few.grid = p.few.items = p.few.split = 0;
    p.many.cols = p.many.tiles = p.many.chunk = 0;
    p.many.chunks = 1;
    const int64_t row_bytes = 4 * (int64_t)a.cache.dim;
    int64_t few_rows = 0, many_rows = 0;  // of the scratch
    if (rows <= kFewRows || a.requests > 1) {  // one request of many rows: one kernel
        p.few.cols = rows <= 16 || rows > kFewRows ? 16 : rows <= 32 ? 32 : 64;
        const int64_t tiles = ((rows > kFewRows ? kFewRows : rows) + p.few.cols - 1) / p.few.cols;
        const int64_t units = (a.max_keys + kAttnStep - 1) / kAttnStep;
        // as many pieces as workgroups fit the 256 compute units at once: one of eight wavefronts, two of four,
        // three of four where 170 registers are enough
        const int64_t want = p.few.cols == 64 ? 256 : p.few.cols == 16 && a.type != BQ_F32 ? 768 : 512;
        const int64_t items = want / heads < 1 ? 1 : want / heads;
        const int64_t cut = units < 1 ? 1 : units, each = tiles * a.requests;
        // a workgroup for every piece there can be; of more than 64 requests two fillings of the GPU, which look
        // the requests up once and walk their pieces
        int64_t grid = items + each < each * cut ? items + each : each * cut;
        if (a.requests > 64 && grid > 2 * items)
            grid = 2 * items;
        p.few.items = (int)items;
        p.few.grid = (int)(grid > 65535 ? 65535 : grid);
        p.few.split = cut > 1;
        few_rows = p.few.split ? heads * 2 * items * p.few.cols : 0;
    }
    if (rows > kFewRows) {
        p.many.cols = rows <= 128 || a.type == BQ_F32 ? 128 : 256;
        // tiles that can have rows: no request has more than its rows fill, all together no more than all rows do
        // and one for each request of many rows
        const int64_t all_rows = a.tokens * group, others = all_rows / kFewRows + 1;
        const int64_t all = all_rows / p.many.cols + (others < a.requests ? others : a.requests);
        const int64_t each = (rows + p.many.cols - 1) / p.many.cols * a.requests, tiles = each < all ? each : all;
        p.many.tiles = (int)(tiles < 32768 ? tiles : 32768);  // a grid dimension; the kernel walks on from there
        const int64_t busy = tiles * heads, least = 512;
        const int64_t steps = (a.max_keys + least - 1) / least;
        int64_t chunks = 256 / busy;  // one filling of the compute units
        chunks = chunks > steps ? steps : chunks;
        chunks = chunks < 1 ? 1 : chunks;
        const int64_t per = steps < 1 ? 1 : (steps + chunks - 1) / chunks;
        p.many.chunk = (int)(per * least);
        p.many.chunks = (int)(steps < 1 ? 1 : (steps + per - 1) / per);
        many_rows = p.many.chunks > 1 ? heads * p.many.tiles * p.many.chunks * p.many.cols : 0;
    }
    p.few_stats = few_rows * row_bytes;
    p.many_sums = p.few_stats + few_rows * 8;
    p.many_stats = p.many_sums + many_rows * row_bytes;
    p.notes = p.many_stats + many_rows * 8;
    p.work_bytes = few_rows || many_rows ? p.notes + 16 + 8 * (int64_t)a.requests : 0;
    return p;
}

template <int CT, int D, bool F32>
static void attn_nt(const AttnArgs &g, dim3 grid, hipStream_t st)
{
    switch (g.p.few.cols) {
    case 16: hipLaunchKernelGGL((attn_kernel<CT, D, 1, 1, 4, F32>), grid, dim3(256), 0, st, g); break;
    case 32: hipLaunchKernelGGL((attn_kernel<CT, D, 1, 2, 4, F32>), grid, dim3(256), 0, st, g); break;
    default:
        // three parts of 128 values for 32 columns a wavefront do not fit its registers: 16 columns, the keys
        // shared by twice as many (16 tokens over 16384 keys 39.7 -> 37.4 us, 32 x 2048 123 -> 117).  Two parts
        // need all 256 and 3 more, which are spilled, and are faster so all the same (31.6 against 38.7 and 85
        // against 120)
        if constexpr (F32 && CT == BQ_BF16 && D == 128)
            hipLaunchKernelGGL((attn_kernel<CT, D, 1, 4, 8, F32>), grid, dim3(512), 0, st, g);
        else
            hipLaunchKernelGGL((attn_kernel<CT, D, 2, 2, 8, F32>), grid, dim3(512), 0, st, g);
    }
}

template <int CT, int D>
static void attn_dim(const AttnArgs &g, dim3 grid, hipStream_t st)
{
    const bool f32 = g.a.type == BQ_F32;
    f32 ? attn_nt<CT, D, true>(g, grid, st) : attn_nt<CT, D, false>(g, grid, st);
}

template <class OT, int D>
static void join_type(const AttnArgs &g, hipStream_t st)
{
    const bq_attn &a = g.a;
    if (g.p.few.split) {
        const int64_t rows = (a.max_new < a.tokens ? a.max_new : a.tokens) * (a.q_heads / a.cache.heads);
        const int64_t most = (rows < kFewRows ? rows : kFewRows) * a.cache.heads;
        hipLaunchKernelGGL((attn_join_few<OT, D>), dim3((unsigned)most, (unsigned)a.requests), dim3(256), 0, st, g);
    }
    if (g.p.many.chunks > 1) {
        const int64_t blocks = (a.tokens * a.q_heads * (D / 8) + 255) / 256;
        const int64_t x = blocks < (1 << 20) ? blocks : 1 << 20, y = (blocks + x - 1) / x;  // fewer than 2^32 threads along x
        hipLaunchKernelGGL((attn_join_many<OT, D>), dim3((unsigned)x, (unsigned)y), dim3(256), 0, st, g);
    }
}

template <int CT, int D>
static void join_dim(const AttnArgs &g, hipStream_t st)
{
    g.a.type == BQ_F32 ? join_type<float, D>(g, st) : join_type<typename Num<CT>::t, D>(g, st);
}

hipError_t launch_attn(const bq_attn &a, const AttnPlan &p, hipStream_t st)
{
    AttnArgs g;
    g.a = a;
    g.p = p;
    g.group = a.q_heads / a.cache.heads;
    g.page_log2 = __builtin_ctz((unsigned)a.cache.page);
    const bool wide = a.cache.dim == 128, f16 = a.cache.type == BQ_F16;
    if (p.many.tiles) {
        const hipError_t e = launch_attn_tiles(g, st);
        if (e != hipSuccess)
            return e;
    }
    if (p.few.cols) {
        const dim3 grid((unsigned)a.cache.heads, (unsigned)p.few.grid);
        if (f16)
            wide ? attn_dim<BQ_F16, 128>(g, grid, st) : attn_dim<BQ_F16, 64>(g, grid, st);
        else
            wide ? attn_dim<BQ_BF16, 128>(g, grid, st) : attn_dim<BQ_BF16, 64>(g, grid, st);
    }
    if (p.few.split || p.many.chunks > 1) {
        if (f16)
            wide ? join_dim<BQ_F16, 128>(g, st) : join_dim<BQ_F16, 64>(g, st);
        else
            wide ? join_dim<BQ_BF16, 128>(g, st) : join_dim<BQ_BF16, 64>(g, st);
    }
    return hipGetLastError();
}

}  // namespace bq
