// bq_sample.hip -- the next token of each row of logits (bq_sample).
//
// Weights are exp((l - m) / T) in binary64, rounded to multiples of 2^-b and added
// as integers: sums are exact, so their order (and the atomics') changes nothing.
// A token whose weight rounds to 0 can be neither drawn nor felt, and is skipped.
//
// The three filters keep a prefix of the descending order, and so does the draw
// end at a place of it: each is "the first token at which the running sum (of
// weights, or of ones) reaches a target".  One pass finds the row's largest
// logit; one more counts tokens and weights in 1024 buckets of (m - l) / T, whose
// running sums say in which bucket a target is reached; a third collects the tokens of
// the few buckets that the filters and the draw can need, ordered by (logit, -index).
//
// Up to 256 rows the first two passes are launches over slices of the rows, sixteen at
// most; the third is one workgroup a row (with more rows, all three are).  Measured: one
// row of 151936 f32 27 to 44 us by the filters' places (4.6, 7.3 and 22 in the kernels: one workgroup reads 600 KB),
// 192 rows 128 us (21, 53, 58: 117 MB three times at up to 5.4 TB/s; the middle one is
// bound by its weights in binary64 and by LDS atomics), 33 rows of 32001 bf16 35 us.
#include "bq_half.h"
#include "bq_model.h"

namespace bq {

constexpr int kSampleThreads = 1024;
constexpr int kBuckets = 1024;  // one a thread
constexpr int kList = 4096;     // tokens of a bucket kept in LDS

typedef unsigned long long u64;

// Logits as integers of the same order; 0 for what has no weight (NaN, -infinity).
__device__ __forceinline__ uint32_t key_of(float l)
{
    if (!(l > -__builtin_inff()))
        return 0;
    const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);  // -0 as +0
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __builtin_bit_cast(float, key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

// What turns a logit into its weight and bucket.
struct Scale {
    double top;     // the largest logit
    double per;     // 32 log2(e) / T
    float topf;
    float unit;     // of a difference of logits, for bucket_of: half, or 2^100 where T is tiny
    float back;     // 1 / unit
    float buckets;  // a unit
    int bits;       // weights are multiples of 2^-bits
    bool greedy;
};

__device__ __forceinline__ Scale scale_of_row(uint32_t top, float t, int vocab)
{
    Scale s;
    s.topf = logit_of(top);
    s.top = (double)s.topf;
    s.greedy = !(t > 0.0f);
    s.per = 32.0 * 1.44269504088896340736 / (double)t;
    const int wide = 32 - __builtin_clz((unsigned)vocab);
    s.bits = 62 - wide < 50 ? 62 - wide : 50;
    // kBuckets of them hold bits + 2 halvings: behind the last one every weight rounds to 0 (bits + 1 would do; f32
    // is off by far less than that).  Half a difference: the whole one may be past f32's range.  2^100 of it under a T
    // whose buckets a unit would be; not with a largest logit of 2^27 and more, which so much of would be infinite
    // (any logit below it is by 8, past the last bucket with infinitely many a unit too).
    const bool tiny = t < 0x1p-100f && fabsf(s.topf) < 0x1p27f;
    s.unit = tiny ? 0x1p100f : 0.5f;
    s.back = tiny ? 0x1p-100f : 2.0f;
    s.buckets = (float)(kBuckets / 32.0 * s.per * (double)s.back / (double)(s.bits + 2));
    return s;
}

// Never falling as the logit falls; kBuckets and more: no weight.  (+infinity minus itself: 0.)
__device__ __forceinline__ int bucket_of(const Scale &s, float l)
{
    if (l == s.topf)
        return 0;
    const float x = __builtin_fmaf(l, -s.unit, s.unit * s.topf) * s.buckets;
    return !s.greedy && x < (float)kBuckets ? (int)x : kBuckets;
}
// Every logit of buckets 0 .. b is at least this (the slack is far above what bucket_of's roundings come to; a NaN, from
// infinite operands, is above nothing).
__device__ __forceinline__ float least_logit(const Scale &s, int b)
{
    if (s.greedy)
        return s.topf;
    return s.topf - (float)(b + 1) * s.back / s.buckets * 1.0001f - fabsf(s.topf) * 0x1p-20f;
}
// exp((l - top) / T) in units of 2^-bits, before it is rounded: 2^(y / 32) with y = n + f, |f| <= 1/2, of which 2^(f / 32)
// is exp(f ln 2 / 32) by its series (the first term left out is below 2^-48 of it), and 2^(n % 32 / 32) from a table.
__device__ __forceinline__ double weight_at(const Scale &s, const double *table, float l)
{
    if (l == s.topf)
        return __builtin_ldexp(1.0, s.bits);
    const double y = ((double)l - s.top) * s.per, n = __builtin_rint(y), f = (y - n) * (0.69314718055994530942 / 32.0);
    double p = 1.0 / 120.0;
    p = __builtin_fma(p, f, 1.0 / 24.0);
    p = __builtin_fma(p, f, 1.0 / 6.0);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    const int i = (int)n;
    return __builtin_ldexp(p * table[i & 31], (i >> 5) + s.bits);
}
// Rounded to nearest: below 2^52, so that in the sum with 2^52 the low bits hold the number.
__device__ __forceinline__ u64 rounded(double w) { return __builtin_bit_cast(u64, w + 0x1p52) & 0xFFFFFFFFFFFFFull; }

// A token's place in the order: larger is earlier.
__device__ __forceinline__ u64 token_of(float l, int i) { return (u64)key_of(l) << 32 | (uint32_t)~i; }

__device__ __forceinline__ u64 lane_u64(u64 x, int lane)
{
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)x, lane), hi = __builtin_amdgcn_readlane((uint32_t)(x >> 32), lane);
    return (u64)hi << 32 | lo;
}

// LDS of a workgroup.
struct Room {
    uint32_t count[kBuckets];   // running counts and weights of the row's buckets
    u64 mass[kBuckets];
    uint32_t count2[kBuckets];  // of parts of one bucket
    u64 mass2[kBuckets];
    u64 list[kList];            // (key, ~index)
    double table[32];           // 2^(i / 32)
    u64 waves[2][kSampleThreads / 64];
    uint32_t found;
    u64 before_count, before_mass, low, high, answer;
    uint32_t listed, gathered;
};

// Running sums over all threads' count and mass (inclusive); every thread gets its own.
__device__ __forceinline__ void scan(Room &r, uint32_t &count, u64 &mass)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t c = __shfl_up(count, off, 64);
        const u64 m = __shfl_up(mass, off, 64);
        if (lane >= off) {
            count += c;
            mass += m;
        }
    }
    if (lane == 63) {
        r.waves[0][wave] = count;
        r.waves[1][wave] = mass;
    }
    __syncthreads();
    u64 c = 0, m = 0;
    for (int w = 0; w < wave; ++w) {
        c += r.waves[0][w];
        m += r.waves[1][w];
    }
    count += (uint32_t)c;
    mass += m;
    __syncthreads();
}

template <int V, class VEC>
__device__ __forceinline__ float largest(const VEC &v)
{
    float m = (float)v[0];
#pragma unroll
    for (int e = 1; e < V; ++e)
        m = fmaxf(m, (float)v[e]);
    return m;
}

// Calls f(index, logit) once for each token from lo to hi of a row: 16 bytes a load, LOADS of them under way.  Where all
// of a load's logits are below `least`, they may be left out.
template <int LOADS, class T, class F>
__device__ __forceinline__ void each_token(const T *row, int lo, int hi, float least, F f)
{
    constexpr int V = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(V)));
    const int tid = threadIdx.x;
    int head = (int)((16 - ((uintptr_t)(row + lo) & 15)) & 15) / (int)sizeof(T);
    head = head < hi - lo ? head : hi - lo;
    if (tid < head)
        f(lo + tid, (float)row[lo + tid]);
    const int from = lo + head, n = (hi - from) / V;
    const vec *p = reinterpret_cast<const vec *>(row + from);
    int c = tid;
    for (; c + (LOADS - 1) * kSampleThreads < n; c += LOADS * kSampleThreads) {
        vec v[LOADS];
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            v[j] = p[c + j * kSampleThreads];
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            if (!(largest<V>(v[j]) < least))
#pragma unroll
                for (int e = 0; e < V; ++e)
                    f(from + (c + j * kSampleThreads) * V + e, (float)v[j][e]);
    }
    for (; c < n; c += kSampleThreads) {
        const vec v = p[c];
#pragma unroll
        for (int e = 0; e < V; ++e)
            f(from + c * V + e, (float)v[e]);
    }
    const int rest = from + n * V + tid;
    if (rest < hi)
        f(rest, (float)row[rest]);
}

// Calls f(index, logit) for the tokens of a row whose logit is not below `least`, and maybe others; few of them: what a
// load brings is only compared, and read again where there is one.
template <class T, class F>
__device__ __forceinline__ void each_above(const T *row, int vocab, float least, F f)
{
    constexpr int V = 16 / sizeof(T), LOADS = 8;
    typedef T vec __attribute__((ext_vector_type(V)));
    const int tid = threadIdx.x;
    int head = (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T);
    head = head < vocab ? head : vocab;
    const int n = (vocab - head) / V, ends = vocab - n * V;
    const vec *p = reinterpret_cast<const vec *>(row + head);
    for (int c = tid; c < n; c += LOADS * kSampleThreads) {
        vec v[LOADS];
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            v[j] = p[c + j * kSampleThreads < n ? c + j * kSampleThreads : c];
        uint32_t some = 0;
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            some |= c + j * kSampleThreads < n && !(largest<V>(v[j]) < least) ? 1u << j : 0;
        while (some) {
            const int j = __builtin_ctz(some), first = head + (c + j * kSampleThreads) * V;
            some &= some - 1;
#pragma unroll 1
            for (int e = 0; e < V; ++e)
                f(first + e, (float)row[first + e]);
        }
    }
    // what no whole load holds, at both ends
    if (tid < ends) {
        const int i = tid < head ? tid : n * V + tid;
        f(i, (float)row[i]);
    }
}

// A place of the descending order: the sum of weights up to and with its token.
struct Place {
    u64 mass;
    u64 token;  // (key, ~index)
};

// The bucket in which the running count (by_count) or weight reaches target, and the sums in front of it.
struct Found {
    int bucket;
    u64 count, mass;
};
__device__ __forceinline__ Found find(Room &r, bool by_count, u64 target)
{
    const int tid = threadIdx.x;
    const u64 upto = by_count ? r.count[tid] : r.mass[tid], before = tid ? (by_count ? r.count[tid - 1] : r.mass[tid - 1]) : 0;
    if (before < target && target <= upto)
        r.found = tid;
    __syncthreads();
    const int b = (int)r.found;
    const Found f{b, b ? r.count[b - 1] : 0, b ? r.mass[b - 1] : 0};
    __syncthreads();
    return f;
}

// The first token at which the running count (by_count) or weight reaches target, which
// the whole row does (1 <= target).  gathered: the list holds all tokens of its bucket.
template <class T>
__device__ __forceinline__ Place reach(Room &r, const Scale &s, const T *row, int vocab, bool by_count, u64 target, bool gathered)
{
    const int tid = threadIdx.x;
    const Found found = find(r, by_count, target);
    const int bucket = found.bucket;
    u64 before_count = found.count, before_mass = found.mass, n = r.count[bucket] - before_count;
    // tokens low <= (key, ~index) <= high of the bucket: n of them, the target among them
    u64 low = 0, high = ~0ull;
    bool from_list = gathered;
    int listed = gathered ? (int)r.gathered : 0;
    auto weight = [&](u64 token) { return rounded(weight_at(s, r.table, logit_of((uint32_t)(token >> 32)))); };
    auto member = [&](u64 token) {
        return token >= low && token <= high && bucket_of(s, logit_of((uint32_t)(token >> 32))) == bucket;
    };
    auto each = [&](auto f) {
        if (from_list) {
            for (int i = tid; i < listed; i += kSampleThreads)
                if (member(r.list[i]))
                    f(r.list[i]);
        } else {
            each_above(row, vocab, least_logit(s, bucket), [&](int i, float l) {
                if (l > -__builtin_inff() && bucket_of(s, l) == bucket) {
                    const u64 token = token_of(l, i);
                    if (token >= low && token <= high)
                        f(token);
                }
            });
        }
    };
    // (the bound only holds back logits that something changes meanwhile)
    auto put = [&](u64 *to, uint32_t size, u64 token) {
        const uint32_t i = atomicAdd(&r.listed, 1u);
        if (i < size)
            to[i] = token;
    };
    for (;;) {
        if (!from_list && n <= kList) {
            if (tid == 0)
                r.listed = 0;
            __syncthreads();
            each([&](u64 token) { put(r.list, kList, token); });
            __syncthreads();
            listed = (int)n;
            from_list = true;
        }
        if (n <= 64)
            break;
        // the members' range, in 1024 parts from its upper end
        if (tid == 0) {
            r.low = ~0ull;
            r.high = 0;
        }
        r.count2[tid] = 0;
        r.mass2[tid] = 0;
        __syncthreads();
        {
            u64 lo = ~0ull, hi = 0;
            each([&](u64 token) {
                lo = token < lo ? token : lo;
                hi = token > hi ? token : hi;
            });
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const u64 l = __shfl_xor(lo, off, 64), h = __shfl_xor(hi, off, 64);
                lo = l < lo ? l : lo;
                hi = h > hi ? h : hi;
            }
            if ((tid & 63) == 0 && lo <= hi) {
                atomicMin(&r.low, lo);
                atomicMax(&r.high, hi);
            }
        }
        __syncthreads();
        const u64 top = r.high, span = top - r.low;
        int shift = 0;
        while (span >> shift >= kBuckets)
            ++shift;
        each([&](u64 token) {
            const int part = (int)((top - token) >> shift);
            atomicAdd(&r.count2[part], 1u);
            atomicAdd(&r.mass2[part], weight(token));
        });
        __syncthreads();
        uint32_t c = r.count2[tid];
        u64 m = r.mass2[tid];
        const uint32_t own = c;
        const u64 own_mass = m;
        scan(r, c, m);
        const u64 upto = by_count ? before_count + c : before_mass + m, mine = by_count ? own : own_mass;
        if (upto - mine < target && target <= upto) {
            r.found = tid;
            r.before_count = before_count + c - own;
            r.before_mass = before_mass + m - own_mass;
        }
        __syncthreads();
        n = r.count2[r.found];
        before_count = r.before_count;
        before_mass = r.before_mass;
        high = top - ((u64)r.found << shift);
        low = high - ((1ull << shift) - 1);
        __syncthreads();
    }
    // at most 64 members, one a lane of the first wavefront
    if (tid == 0)
        r.listed = 0;
    __syncthreads();
    u64 *last = r.mass2;
    each([&](u64 token) { put(last, 64, token); });
    __syncthreads();
    if (tid < 64) {
        const bool live = tid < (int)n;
        const u64 token = live ? last[tid] : 0;
        const u64 w = live ? weight(token) : 0;
        u64 count = before_count, mass = before_mass;
        for (int i = 0; i < (int)n; ++i) {
            const bool ahead = lane_u64(token, i) >= token;
            count += ahead;
            mass += ahead ? lane_u64(w, i) : 0;
        }
        const u64 upto = by_count ? count : mass, mine = by_count ? 1 : w;
        if (live && upto - mine < target && target <= upto) {
            r.answer = token;
            r.before_mass = mass;
        }
    }
    __syncthreads();
    const Place p{r.before_mass, r.answer};
    __syncthreads();
    return p;
}

// The largest key of a slice, in every thread.
template <class T>
__device__ __forceinline__ uint32_t slice_top(Room &r, const T *row, int lo, int hi)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float top = -__builtin_inff();
    each_token<4>(row, lo, hi, -__builtin_inff(), [&](int, float l) { top = fmaxf(top, l); });  // (the number of a number and a NaN)
    top = wave_all(top, Max());
    if (lane == 0)
        r.waves[0][wave] = key_of(top);
    __syncthreads();
    uint32_t key = 0;
    for (int w = 0; w < kSampleThreads / 64; ++w)
        key = (uint32_t)r.waves[0][w] > key ? (uint32_t)r.waves[0][w] : key;
    __syncthreads();
    return key;
}

// Counts and weights of a slice's tokens by bucket into r.count and r.mass; the weight of those that weigh at least
// `least` (of 1), of the whole workgroup, in thread 0's return value.
template <class T>
__device__ __forceinline__ u64 slice_buckets(Room &r, const Scale &s, const T *row, int lo, int hi, double least)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    r.count[tid] = 0;
    r.mass[tid] = 0;
    __syncthreads();
    const double bound = __builtin_ldexp(least, s.bits);
    u64 over = 0;
    each_token<2>(row, lo, hi, least_logit(s, kBuckets - 1), [&](int, float l) {
        if (!(l > -__builtin_inff()))
            return;
        const int b = bucket_of(s, l);
        if (b >= kBuckets)
            return;
        const double w = weight_at(s, r.table, l);
        const u64 units = rounded(w);
        atomicAdd(&r.count[b], 1u);
        atomicAdd(&r.mass[b], units);
        over += w >= bound ? units : 0;
    });
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        over += __shfl_xor(over, off, 64);
    if (lane == 0)
        r.waves[0][wave] = over;
    __syncthreads();
    over = 0;
    for (int w = 0; w < kSampleThreads / 64; ++w)
        over += r.waves[0][w];
    __syncthreads();
    return over;
}

__device__ __forceinline__ void fill_table(Room &r)
{
    if (threadIdx.x < 32)
        r.table[threadIdx.x] = exp2((double)threadIdx.x / 32.0);
}

// The rest of a row, whose counts and weights by bucket are in r.count and r.mass (`over`: the weight that min_p keeps).
template <class T>
__device__ void pick(Room &r, const bq_draw &a, const Scale &s, const T *row, int64_t at, u64 over)
{
    const int tid = threadIdx.x, vocab = (int)a.vocab;
    uint32_t c = r.count[tid];
    u64 m = r.mass[tid];
    scan(r, c, m);
    r.count[tid] = c;
    r.mass[tid] = m;
    __syncthreads();
    const u64 total = r.mass[kBuckets - 1];
    const uint32_t weighty = r.count[kBuckets - 1];
    const int k = !s.greedy && a.top_k ? a.top_k[at] : 0;
    const float p = !s.greedy && a.top_p ? a.top_p[at] : 1.0f;
    const bool limit_k = k > 0 && (uint32_t)k < weighty, limit_p = p < 1.0f;
    const double share = limit_p ? (double)p : 1.0;
    // How far each filter's place, and the draw's, can lie apart follows from the buckets: their tokens are collected
    // in one pass over the row, where the list has room for them (else each place is looked for in a pass of its own).
    auto share_of = [&](u64 mass) {
        const double want = share * (double)mass;
        const u64 target = want > 0.0 ? (u64)__builtin_ceil(want) : 1;
        return target > mass && mass ? mass : target < 1 ? 1 : target;
    };
    const double u = s.greedy ? 0.0 : (double)a.u[at];
    auto drawn_of = [&](u64 mass) {
        const double want = u * (double)mass;
        const u64 target = want >= 1.0 ? (want >= (double)mass ? mass : (u64)want + 1) : 1;
        return target > mass && mass ? mass : target;
    };
    u64 lo = total, hi = total;  // bounds of the kept weight
    int k0 = 0, k1 = -1, p0 = 0, p1 = -1;
    if (limit_k) {
        const Found f = find(r, true, (u64)k);
        k0 = k1 = f.bucket;
        lo = f.mass;
        hi = r.mass[k0];
    }
    if (limit_p) {
        const Found f = find(r, false, share_of(lo)), g = find(r, false, share_of(hi));
        p0 = f.bucket;
        p1 = g.bucket;
        lo = f.mass < lo ? f.mass : lo;
        hi = r.mass[p1] < hi ? r.mass[p1] : hi;
    }
    if (!s.greedy) {
        lo = over < lo ? over : lo;
        hi = over < hi ? over : hi;
    }
    const int d0 = find(r, false, drawn_of(lo)).bucket, d1 = find(r, false, drawn_of(hi)).bucket;
    auto counted = [&](int from, int to) { return from > to ? 0u : r.count[to] - (from ? r.count[from - 1] : 0u); };
    const bool gather = counted(k0, k1) + counted(p0, p1) + counted(d0, d1) <= kList;
    if (gather) {
        if (tid == 0)
            r.gathered = 0;
        __syncthreads();
        const int most = d1 > p1 ? d1 > k1 ? d1 : k1 : p1 > k1 ? p1 : k1;
        auto collect = [&](int i, float l) {
            if (!(l > -__builtin_inff()))
                return;
            const int b = bucket_of(s, l);
            if ((b >= d0 && b <= d1) || (b >= p0 && b <= p1) || b == k1) {
                const uint32_t to = atomicAdd(&r.gathered, 1u);
                if (to < kList)
                    r.list[to] = token_of(l, i);
            }
        };
        // few tokens that far up in the order: most loads hold none of them
        if (r.count[most] < (uint32_t)vocab / 64)
            each_above(row, vocab, least_logit(s, most), collect);
        else
            each_token<16 / sizeof(T)>(row, 0, vocab, -__builtin_inff(), collect);
        __syncthreads();
        if (tid == 0 && r.gathered > kList)  // (only if something changes the logits meanwhile)
            r.gathered = kList;
        __syncthreads();
    }
    // the places in turn: the k-th token, the end of top_p, the draw
    u64 mass = total, target = 1;
    Place place;
    for (int what = limit_k ? 0 : limit_p ? 1 : 2;; what = what == 0 && limit_p ? 1 : 2) {
        if (what == 1)
            target = share_of(mass);
        if (what == 2) {
            if (!s.greedy)
                mass = over < mass ? over : mass;
            target = drawn_of(mass);
        }
        place = reach(r, s, row, vocab, what == 0, what == 0 ? (u64)k : target, gather);
        if (what == 2)
            break;
        mass = place.mass < mass ? place.mass : mass;
    }
    if (tid == 0) {
        a.token[at] = (uint32_t)~(uint32_t)place.token;
        if (a.logprob) {
            const double w = weight_at(s, r.table, logit_of((uint32_t)(place.token >> 32)));
            a.logprob[at] = s.greedy ? 0.0f : (float)log(w / (double)total);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ double least_of(const bq_draw &a, const Scale &s, int64_t at)
{
    const float least = a.min_p && !s.greedy ? a.min_p[at] : 0.0f;
    return least > 0.0f ? (double)least : 0.0;
}
__device__ __forceinline__ void no_token(const bq_draw &a, int64_t at)
{
    if (threadIdx.x == 0) {
        a.token[at] = -1;
        if (a.logprob)
            a.logprob[at] = -__builtin_inff();
    }
}

// Whole rows, one a workgroup at a time.
template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_rows(const bq_draw a)
{
    __shared__ Room r;
    fill_table(r);
    for (int64_t at = blockIdx.x; at < a.rows; at += gridDim.x) {
        const T *row = static_cast<const T *>(a.logits) + at * a.ld_logits;
        const uint32_t top = slice_top(r, row, 0, (int)a.vocab);
        if (top == 0) {
            no_token(a, at);
            continue;
        }
        const Scale s = scale_of_row(top, a.temperature ? a.temperature[at] : 1.0f, (int)a.vocab);
        const u64 over = slice_buckets(r, s, row, 0, (int)a.vocab, least_of(a, s, at));
        pick(r, a, s, row, at, over);
    }
}

// Few rows: their slices in three launches, with what the launches hand on in scratch: a key a slice, then a slice's
// 1024 weights, 1024 counts and what min_p keeps.
struct Slices {
    bq_draw a;
    int n, len;  // slices a row, tokens a slice
};
constexpr int64_t kSliceBytes = kBuckets * 12 + 16;
__device__ __forceinline__ uint32_t *slice_keys(const Slices &g, int64_t at) { return static_cast<uint32_t *>(g.a.work) + at * g.n; }
__device__ __forceinline__ u64 *slice_sums(const Slices &g, int64_t at, int i)
{
    const int64_t keys = (g.a.rows * g.n * 4 + 15) / 16 * 16;
    return reinterpret_cast<u64 *>(static_cast<char *>(g.a.work) + keys + (at * g.n + i) * kSliceBytes);
}
__device__ __forceinline__ uint32_t row_top(const Slices &g, int64_t at)
{
    uint32_t top = 0;
    for (int i = 0; i < g.n; ++i)
        top = slice_keys(g, at)[i] > top ? slice_keys(g, at)[i] : top;
    return top;
}

template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_tops(const Slices g)
{
    __shared__ Room r;
    const int64_t at = blockIdx.x / g.n;
    const int i = blockIdx.x % g.n, lo = i * g.len, hi = lo + g.len < g.a.vocab ? lo + g.len : (int)g.a.vocab;
    const uint32_t top = slice_top(r, static_cast<const T *>(g.a.logits) + at * g.a.ld_logits, lo, hi);
    if (threadIdx.x == 0)
        slice_keys(g, at)[i] = top;
}

template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_buckets(const Slices g)
{
    __shared__ Room r;
    fill_table(r);
    const bq_draw &a = g.a;
    const int tid = threadIdx.x;
    const int64_t at = blockIdx.x / g.n;
    const int i = blockIdx.x % g.n, lo = i * g.len, hi = lo + g.len < a.vocab ? lo + g.len : (int)a.vocab;
    const uint32_t top = row_top(g, at);
    if (top == 0)
        return;
    const Scale s = scale_of_row(top, a.temperature ? a.temperature[at] : 1.0f, (int)a.vocab);
    const u64 over = slice_buckets(r, s, static_cast<const T *>(a.logits) + at * a.ld_logits, lo, hi, least_of(a, s, at));
    u64 *sums = slice_sums(g, at, i);
    sums[tid] = r.mass[tid];
    reinterpret_cast<uint32_t *>(sums + kBuckets)[tid] = r.count[tid];
    if (tid == 0)
        sums[kBuckets + kBuckets / 2] = over;
}

template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_pick(const Slices g)
{
    __shared__ Room r;
    fill_table(r);
    const bq_draw &a = g.a;
    const int tid = threadIdx.x;
    const int64_t at = blockIdx.x;
    const uint32_t top = row_top(g, at);
    if (top == 0) {
        no_token(a, at);
        return;
    }
    const Scale s = scale_of_row(top, a.temperature ? a.temperature[at] : 1.0f, (int)a.vocab);
    u64 mass = 0, over = 0;
    uint32_t count = 0;
#pragma unroll 8
    for (int i = 0; i < g.n; ++i) {
        const u64 *sums = slice_sums(g, at, i);
        mass += sums[tid];
        count += reinterpret_cast<const uint32_t *>(sums + kBuckets)[tid];
        over += sums[kBuckets + kBuckets / 2];
    }
    r.mass[tid] = mass;
    r.count[tid] = count;
    __syncthreads();
    pick(r, a, s, static_cast<const T *>(a.logits) + at * a.ld_logits, at, over);
}

// Slices a row: enough workgroups for two a compute unit, each with 4096 tokens or more; 1: whole rows.
static Slices slices_of(const bq_draw &a)
{
    Slices g;
    g.a = a;
    int64_t n = 512 / a.rows;
    const int64_t most = (a.vocab + 4095) / 4096 < 16 ? (a.vocab + 4095) / 4096 : 16;
    n = n < 1 ? 1 : n > most ? most : n;
    g.len = (int)((a.vocab + n - 1) / n);
    g.n = (int)((a.vocab + g.len - 1) / g.len);
    return g;
}

int64_t sample_work(const bq_draw &a)
{
    const Slices g = slices_of(a);
    return g.n == 1 ? 0 : (a.rows * g.n * 4 + 15) / 16 * 16 + a.rows * g.n * kSliceBytes;
}

template <class T>
static void sample_type(const bq_draw &a, hipStream_t st)
{
    const Slices g = slices_of(a);
    const dim3 block(kSampleThreads);
    if (g.n == 1) {
        const int64_t most = int64_t(1) << 21;
        hipLaunchKernelGGL((sample_rows<T>), dim3((unsigned)(a.rows < most ? a.rows : most)), block, 0, st, a);
        return;
    }
    const dim3 grid((unsigned)(a.rows * g.n));
    hipLaunchKernelGGL((sample_tops<T>), grid, block, 0, st, g);
    hipLaunchKernelGGL((sample_buckets<T>), grid, block, 0, st, g);
    hipLaunchKernelGGL((sample_pick<T>), dim3((unsigned)a.rows), block, 0, st, g);
}

hipError_t launch_sample(const bq_draw &a, hipStream_t st)
{
    switch (a.type) {
    case BQ_F16: sample_type<_Float16>(a, st); break;
    case BQ_BF16: sample_type<__bf16>(a, st); break;
    default: sample_type<float>(a, st); break;
    }
    return hipGetLastError();
}

}  // namespace bq
