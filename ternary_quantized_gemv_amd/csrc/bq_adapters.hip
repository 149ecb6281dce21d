// bq_adapters.hip -- low-rank updates of many requests beside a shared
// projection (bq_adapters_add): out = y + gain B (A x), row by row, each
// request with its own A (rank x n) and B (rows x rank).
//
// Two launches: u = gain A x, split along n where the requests are few (pieces
// in the scratch, added up by the second launch in a fixed order), then out = y +
// B u.  Both are v_mfma_f32_16x16x32 products with the adapter's rows along the
// result's rows and up to 16 tokens of one request along its columns; a decode
// step uses one column, which costs nothing: the adapters' weights bound it
// (read once a request), or for prompts x, y and out.
//
// f32 values (x, and u) enter as three bf16 parts that hold their 24 bits
// exactly; f16 weights beside them as two (8 and 3 bits, exact), all products
// but the smallest (2^-24 of the largest, at most) on the matrix cores.
#include "bq_attn.h"

namespace bq {

constexpr int kDownStep = 128;    // values of n that a workgroup's four wavefronts take at a time
constexpr int kMaxPieces = 16;    // of n
constexpr int kUpRows = 256;      // rows of B per workgroup

struct AdapterArgs {
    bq_adapters a;
    int64_t piece;    // values of n in each of the pieces: up to 2^31
    int pieces;       // of n
    int down_items;   // items along the grid: of 16 or 32 tokens, and of 16
    int up_items;
    int direct;       // item i is request i (few tokens each), else the items of all requests are counted through
};

// Item `item` of TOKENS tokens each: request b, its rows and where they start.
// With `direct` a request is one item, which walks its rows.
template <int TOKENS>
__device__ __forceinline__ bool adapter_item(const AdapterArgs &g, Walk &w, int item, int &b, int &first, int &end)
{
    const bq_adapters &a = g.a;
    int within = 0, front;
    if (g.direct) {
        if (item >= a.requests)
            return false;
        b = item;
    } else if (!find_item<false>(w, a.requests, item, b, within, front, [&](int i, int &) {
                   return (rows_between(a.cu[i], a.cu[i + 1], a.tokens).n + TOKENS - 1) / TOKENS;
               })) {
        return false;
    }
    const Rows rows = rows_between(uniform_word(a.cu + b), uniform_word(a.cu + b + 1), a.tokens);
    first = rows.first;
    end = first + rows.n;
    if (!g.direct) {
        first += within * TOKENS;
        end = min(end, first + TOKENS);
    }
    return true;
}

// c += W X^T for 32 values of k: weights w (16 bits), values x as f32 or of the weights' type.
template <class T, class X> struct Step;
template <class T> struct Step<T, T> {
    typedef T t8 __attribute__((ext_vector_type(8)));
    typedef t8 raw;
    t8 x;
    __device__ __forceinline__ void set(raw v) { x = v; }
    __device__ __forceinline__ f32x4 add(t8 w, f32x4 c) const
    {
        return Num<sizeof(T) == 2 && __is_same(T, _Float16) ? BQ_F16 : BQ_BF16>::mfma16(w, x, c);
    }
};
template <class T> struct Step<T, float> {
    typedef T t8 __attribute__((ext_vector_type(8)));
    typedef float raw __attribute__((ext_vector_type(8), aligned(16)));
    bf16x8 x[3];
    __device__ __forceinline__ void set(raw r)
    {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = r[e];
        Split<__bf16, 3>::parts(v, x);
    }
    __device__ __forceinline__ f32x4 add(t8 w, f32x4 c) const
    {
        typedef Num<BQ_BF16> N;
        if constexpr (__is_same(T, __bf16)) {
            c = N::mfma16(w, x[2], c);
            c = N::mfma16(w, x[1], c);
            return N::mfma16(w, x[0], c);
        } else {
            // an f16's 11 bits as 8 and 3
            u32x4 hi, lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t p = __builtin_bit_cast(uint32_t, (float)w[2 * i]), q = __builtin_bit_cast(uint32_t, (float)w[2 * i + 1]);
                const float pr = (float)w[2 * i] - __builtin_bit_cast(float, p & 0xFFFF0000u);
                const float qr = (float)w[2 * i + 1] - __builtin_bit_cast(float, q & 0xFFFF0000u);
                hi[i] = upper_halves(p, q);
                lo[i] = upper_halves(__builtin_bit_cast(uint32_t, pr), __builtin_bit_cast(uint32_t, qr));
            }
            const bf16x8 h = __builtin_bit_cast(bf16x8, hi), l = __builtin_bit_cast(bf16x8, lo);
            c = N::mfma16(h, x[2], c);
            c = N::mfma16(l, x[1], c);
            c = N::mfma16(h, x[1], c);
            c = N::mfma16(l, x[0], c);
            return N::mfma16(h, x[0], c);
        }
    }
};

// u[piece][t][r] = gain A[r] . x[t] over a piece of n: ranks along the result's
// rows (RT tiles of 16, a grid row for every 64), tokens along its columns (NT
// tiles).  The four wavefronts take turns along n and add up in LDS.  Latency
// bounds the small calls (16 requests of rank 16, n 4096: 4.2 us), x's reading
// the large (1000 tokens of rank 64: 11 us).
template <class T, class X, int RT, int NT>
__global__ __launch_bounds__(256) void adapters_down(const AdapterArgs g)
{
    typedef T t8 __attribute__((ext_vector_type(8)));
    constexpr int U = RT * NT <= 4 ? 4 : 2;
    __shared__ float red[4][NT][RT][16][17];
    const bq_adapters &a = g.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, q4 = lane >> 4;
    const int piece = blockIdx.x % g.pieces, rank0 = blockIdx.y * 16 * RT;
    const int64_t from = piece * g.piece, to = min(from + g.piece, a.n);
    Walk walk;
    int b, first, end;
    for (int item = blockIdx.x / g.pieces; adapter_item<16 * NT>(g, walk, item, b, first, end); item += gridDim.x / g.pieces) {
        const int id = uniform_word(a.ids + b);
        if ((unsigned)id >= (unsigned)a.count)
            continue;
        const float gain = a.gain[id];
        const T *w[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            w[r] = static_cast<const T *>(a.a) + ((int64_t)id * a.rank + min(rank0 + 16 * r + c16, a.rank - 1)) * a.n + 8 * q4;
        for (int t0 = first; t0 < end; t0 += 16 * NT) {
            f32x4 acc[NT][RT];
            const X *x[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                x[t] = static_cast<const X *>(a.x) + (int64_t)min(t0 + 16 * t + c16, end - 1) * a.ld_x + 8 * q4;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[t][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            for (int64_t i0 = from + 32 * wave; i0 < to; i0 += U * kDownStep) {
                // the loads of U steps, then their products
                typename Step<T, X>::raw x8[U][NT];
                t8 v[U][RT];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int64_t i = i0 + j * kDownStep;
                    const bool in = i + 8 * q4 < to;  // n is a multiple of 8: the last lanes may have none
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        v[j][r] = in ? *reinterpret_cast<const t8 *>(w[r] + i) : t8{};
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        x8[j][t] = in ? *reinterpret_cast<const typename Step<T, X>::raw *>(x[t] + i) : typename Step<T, X>::raw{};
                }
#pragma unroll
                for (int j = 0; j < U; ++j)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        Step<T, X> s;
                        s.set(x8[j][t]);
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            acc[t][r] = s.add(v[j][r], acc[t][r]);
                    }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        red[wave][t][r][c16][4 * q4 + e] = acc[t][r][e];
            __syncthreads();
            for (int u = threadIdx.x; u < NT * 16 * RT * 16; u += 256) {
                const int r = u % (16 * RT), t = u / (16 * RT);
                if (rank0 + r < a.rank && t0 + t < end) {
                    float sum = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sum += red[k][t >> 4][r >> 4][t & 15][r & 15];
                    static_cast<float *>(a.work)[((int64_t)piece * a.tokens + t0 + t) * a.rank + rank0 + r] = sum * gain;
                }
            }
            __syncthreads();
        }
    }
}

// out[t][row] = y[t][row] + B[row] . u[t]: 64 rows of B a wavefront, in
// registers, along the result's rows; 16 tokens along its columns.  The pieces
// of u are added up once for the workgroup's wavefronts, in LDS.  (32 tokens an
// item read B and u half as often, but leave two wavefronts a SIMD where four
// fit: 19.3 against 17.1 us for 1000 tokens x 4096 rows of rank 64.)
template <class T, int KS>
__global__ __launch_bounds__(256) void adapters_up(const AdapterArgs g)
{
    typedef T t8 __attribute__((ext_vector_type(8)));
    __shared__ float us[16][32 * KS + 4];
    const bq_adapters &a = g.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, q4 = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.y * kUpRows + 64 * wave;
    // four rows at a time, at any multiple of 4 bytes; the matrix's last rows one by one
    typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
    const bool full = row0 + 64 <= a.rows;
    Walk walk;
    int b, first, end;
    for (int item = blockIdx.x; adapter_item<16>(g, walk, item, b, first, end); item += gridDim.x) {
        const int id = uniform_word(a.ids + b);
        const bool has = (unsigned)id < (unsigned)a.count;
        if (!has && a.y == a.out)
            continue;
        t8 w[4][KS];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t row = min(row0 + 16 * r + c16, a.rows - 1);
#pragma unroll
            for (int k = 0; k < KS; ++k)
                w[r][k] = has && 32 * k + 8 * q4 < a.rank
                              ? *reinterpret_cast<const t8 *>(static_cast<const T *>(a.b) + ((int64_t)id * a.rows + row) * a.rank + 32 * k + 8 * q4)
                              : t8{};
        }
        for (int t0 = first; t0 < end; t0 += 16) {
            const int t = t0 + c16;
            const float *y = a.y + (int64_t)min(t, end - 1) * a.ld_y + row0 + 4 * q4;
            float *out = a.out + (int64_t)t * a.ld_out + row0 + 4 * q4;
            f32x4 sum[4];
            if (full) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sum[r] = *reinterpret_cast<const f32x4u *>(y + 16 * r);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[r][e] = row0 + 16 * r + 4 * q4 + e < a.rows ? y[16 * r + e] : 0.0f;
            }
            if (has) {
                // four ranks of a token at a time; the loads of four pieces, for all that a thread has, before their sums
                constexpr int QUADS = 16 * 8 * KS, MINE = (QUADS + 255) / 256;
                f32x4 u[MINE];
#pragma unroll
                for (int i = 0; i < MINE; ++i)
                    u[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                for (int j = 0; j < g.pieces; j += 4) {
                    f32x4 x[MINE][4];
#pragma unroll
                    for (int i = 0; i < MINE; ++i) {
                        const int q = threadIdx.x + 256 * i, r = q % (8 * KS) * 4, tok = t0 + q / (8 * KS);
                        const float *p = static_cast<const float *>(a.work) + (int64_t)tok * a.rank + r;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[i][k] = q < QUADS && r < a.rank && tok < end && j + k < g.pieces
                                          ? *reinterpret_cast<const f32x4 *>(p + (int64_t)(j + k) * a.tokens * a.rank)
                                          : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
#pragma unroll
                    for (int i = 0; i < MINE; ++i)
                        u[i] += (x[i][0] + x[i][1]) + (x[i][2] + x[i][3]);
                }
#pragma unroll
                for (int i = 0; i < MINE; ++i) {
                    const int q = threadIdx.x + 256 * i;
                    if (q < QUADS)
                        *reinterpret_cast<f32x4 *>(&us[q / (8 * KS)][q % (8 * KS) * 4]) = u[i];
                }
                __syncthreads();
                f32x4 acc[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    Step<T, float> s;
                    s.set(*reinterpret_cast<const typename Step<T, float>::raw *>(&us[c16][32 * k + 8 * q4]));
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[r] = s.add(w[r][k], acc[r]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sum[r] += acc[r];
                __syncthreads();
            }
            if (t < end && full) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<f32x4u *>(out + 16 * r) = sum[r];
            } else if (t < end) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (row0 + 16 * r + 4 * q4 + e < a.rows)
                            out[16 * r + e] = sum[r][e];
            }
        }
    }
}

static AdapterArgs adapters_plan(const bq_adapters &a)
{
    AdapterArgs g;
    g.a = a;
    const int64_t most = a.max_new < a.tokens ? a.max_new : a.tokens;
    g.direct = most <= 16;
    // items: no request has more tiles than its tokens fill, all together no more than all tokens do
    auto items = [&](int tokens) {
        const int64_t all = a.tokens / tokens + a.requests, each = (most + tokens - 1) / tokens * a.requests;
        return g.direct ? (int64_t)a.requests : all < each ? all : each;
    };
    const int64_t down = items(g.direct ? 16 : 32), up = items(16);
    // pieces of n until a workgroup a compute unit runs, none of fewer than 512 values
    int64_t pieces = 256 / down, cap = a.n / 512;
    pieces = pieces > cap ? cap : pieces;
    pieces = pieces > kMaxPieces ? kMaxPieces : pieces < 1 ? 1 : pieces;
    const int64_t steps = (a.n + kDownStep - 1) / kDownStep, per = (steps + pieces - 1) / pieces;
    g.piece = per * kDownStep;
    g.pieces = (int)((steps + per - 1) / per);
    // a grid holds fewer than 2^32 threads along x; the kernels walk on from there
    g.down_items = (int)(down < (1 << 22) ? down : 1 << 22);
    g.up_items = (int)(up < (1 << 22) ? up : 1 << 22);
    return g;
}

int64_t adapters_work(const bq_adapters &a) { return adapters_plan(a).pieces * a.tokens * a.rank * 4; }

template <class T, class X, int RT>
static void down_nt(const AdapterArgs &g, hipStream_t st)
{
    const dim3 grid((unsigned)(g.down_items * g.pieces), (unsigned)((g.a.rank + 16 * RT - 1) / (16 * RT)));
    if (g.direct)
        hipLaunchKernelGGL((adapters_down<T, X, RT, 1>), grid, dim3(256), 0, st, g);
    else
        hipLaunchKernelGGL((adapters_down<T, X, RT, 2>), grid, dim3(256), 0, st, g);
}

template <class T, class X>
static void down_rank(const AdapterArgs &g, hipStream_t st)
{
    const int rank = g.a.rank;
    rank <= 16 ? down_nt<T, X, 1>(g, st) : rank <= 32 ? down_nt<T, X, 2>(g, st) : down_nt<T, X, 4>(g, st);
}

template <class T, int KS>
static void up_rank(const AdapterArgs &g, hipStream_t st)
{
    const dim3 grid((unsigned)g.up_items, (unsigned)((g.a.rows + kUpRows - 1) / kUpRows));
    hipLaunchKernelGGL((adapters_up<T, KS>), grid, dim3(256), 0, st, g);
}

template <class T>
static void adapters_type(const AdapterArgs &g, hipStream_t st)
{
    g.a.x_type == BQ_F32 ? down_rank<T, float>(g, st) : down_rank<T, T>(g, st);
    g.a.rank <= 32 ? up_rank<T, 1>(g, st) : g.a.rank <= 64 ? up_rank<T, 2>(g, st) : up_rank<T, 4>(g, st);
}

hipError_t launch_adapters(const bq_adapters &a, hipStream_t st)
{
    const AdapterArgs g = adapters_plan(a);
    a.type == BQ_F16 ? adapters_type<_Float16>(g, st) : adapters_type<__bf16>(g, st);
    return hipGetLastError();
}

}  // namespace bq
