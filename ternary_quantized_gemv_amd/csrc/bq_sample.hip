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
// running sums say in which bucket a target is reached; only that bucket's tokens
// are then looked at, ordered by (logit, -index).
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
    double top;      // the largest logit
    double per;      // log2(e) / T
    float buckets;   // buckets a unit of log2 weight
    int bits;        // weights are multiples of 2^-bits
    bool greedy;
};

// log2 of the weight, at most 0.
__device__ __forceinline__ double log2_weight(const Scale &s, float l)
{
    const double x = (double)l - s.top;
    if ((double)l == s.top)
        return 0.0;
    return s.greedy ? -__builtin_inf() : x * s.per;
}
// 2^y in units of 2^-bits, rounded to nearest: y = n + f, |f| <= 1/2, 2^f = exp(f ln 2) by
// its series (the first term left out is below 2^-52 of it); 0 where it is below half a unit.
__device__ __forceinline__ u64 weight_of(const Scale &s, double y)
{
    if (!(y > -(double)(s.bits + 1)))
        return 0;
    const double n = __builtin_rint(y), f = (y - n) * 0.69314718055994530942;
    double p = 1.0 / 479001600.0;
    p = __builtin_fma(p, f, 1.0 / 39916800.0);
    p = __builtin_fma(p, f, 1.0 / 3628800.0);
    p = __builtin_fma(p, f, 1.0 / 362880.0);
    p = __builtin_fma(p, f, 1.0 / 40320.0);
    p = __builtin_fma(p, f, 1.0 / 5040.0);
    p = __builtin_fma(p, f, 1.0 / 720.0);
    p = __builtin_fma(p, f, 1.0 / 120.0);
    p = __builtin_fma(p, f, 1.0 / 24.0);
    p = __builtin_fma(p, f, 1.0 / 6.0);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    // weights are below 2^52 units: added to 2^52, the low bits hold the rounded number
    const double w = __builtin_ldexp(p, (int)n + s.bits) + 0x1p52;
    return __builtin_bit_cast(u64, w) & 0xFFFFFFFFFFFFFull;
}
// y > -(bits + 1) - 1/2: never more than kBuckets - 1, and never falling as the logit falls.
__device__ __forceinline__ int bucket_of(const Scale &s, double y)
{
    const int b = (int)((float)-y * s.buckets);
    return b < kBuckets ? b : kBuckets - 1;
}

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
    u64 waves[2][kSampleThreads / 64];
    uint32_t found;
    u64 before_count, before_mass, low, high, answer;
    uint32_t listed;
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

// The tokens of a row.  Calls f(index, logit) for all of them, each once.
template <class T, class F>
__device__ __forceinline__ void each_token(const T *row, int vocab, F f)
{
    for (int i = threadIdx.x; i < vocab; i += kSampleThreads)
        f(i, (float)row[i]);
}

// A place of the descending order: the sum of weights up to and with its token.
struct Place {
    u64 mass;
    u64 token;  // (key, ~index)
};

// The first token at which the running count (by_count) or weight reaches target, which
// the whole row does (1 <= target).
template <class T>
__device__ Place reach(Room &r, const Scale &s, const T *row, int vocab, bool by_count, u64 target)
{
    const int tid = threadIdx.x;
    {
        const u64 upto = by_count ? r.count[tid] : r.mass[tid], before = tid ? (by_count ? r.count[tid - 1] : r.mass[tid - 1]) : 0;
        if (before < target && target <= upto) {
            r.found = tid;
            r.before_count = tid ? r.count[tid - 1] : 0;
            r.before_mass = tid ? r.mass[tid - 1] : 0;
        }
    }
    __syncthreads();
    const int bucket = (int)r.found;
    u64 n = r.count[bucket] - (uint32_t)r.before_count, before_count = r.before_count, before_mass = r.before_mass;
    // tokens low <= (key, ~index) <= high of the bucket: n of them, the target among them
    u64 low = 0, high = ~0ull;
    bool from_list = false;
    int listed = 0;
    auto member = [&](u64 token) { return token >= low && token <= high; };
    auto each = [&](auto f) {
        if (from_list) {
            for (int i = tid; i < listed; i += kSampleThreads)
                if (member(r.list[i]))
                    f(r.list[i]);
        } else {
            each_token(row, vocab, [&](int i, float l) {
                const uint32_t key = key_of(l);
                const u64 token = (u64)key << 32 | (uint32_t)~i;
                if (!key || !member(token))
                    return;
                const double y = log2_weight(s, l);
                if (weight_of(s, y) && bucket_of(s, y) == bucket)
                    f(token);
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
            if (lo <= hi) {
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
            atomicAdd(&r.mass2[part], weight_of(s, log2_weight(s, logit_of((uint32_t)(token >> 32)))));
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
        const u64 w = live ? weight_of(s, log2_weight(s, logit_of((uint32_t)(token >> 32)))) : 0;
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

template <class T>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(const bq_draw a)
{
    __shared__ Room r;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, vocab = (int)a.vocab;
    for (int64_t at = blockIdx.x; at < a.rows; at += gridDim.x) {
        const T *row = static_cast<const T *>(a.logits) + at * a.ld_logits;
        uint32_t top = 0;
        each_token(row, vocab, [&](int, float l) {
            const uint32_t k = key_of(l);
            top = k > top ? k : top;
        });
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_xor(top, off, 64);
            top = o > top ? o : top;
        }
        if (lane == 0)
            r.waves[0][wave] = top;
        r.count[tid] = 0;
        r.mass[tid] = 0;
        __syncthreads();
        for (int w = 0; w < kSampleThreads / 64; ++w)
            top = (uint32_t)r.waves[0][w] > top ? (uint32_t)r.waves[0][w] : top;
        __syncthreads();
        if (top == 0) {
            if (tid == 0) {
                a.token[at] = -1;
                if (a.logprob)
                    a.logprob[at] = -__builtin_inff();
            }
            continue;
        }
        const float t = a.temperature ? a.temperature[at] : 1.0f;
        Scale s;
        s.top = (double)logit_of(top);
        s.greedy = !(t > 0.0f);
        s.per = 1.44269504088896340736 / (double)t;
        const int wide = 32 - __builtin_clz((unsigned)vocab);
        s.bits = 62 - wide < 50 ? 62 - wide : 50;
        s.buckets = (float)kBuckets / (float)(s.bits + 2);
        const double least = a.min_p ? (double)a.min_p[at] : 0.0;
        u64 over = 0;
        each_token(row, vocab, [&](int, float l) {
            if (!key_of(l))
                return;
            const double y = log2_weight(s, l);
            const u64 w = weight_of(s, y);
            if (!w)
                return;
            const int b = bucket_of(s, y);
            atomicAdd(&r.count[b], 1u);
            atomicAdd(&r.mass[b], w);
            if (least > 0.0 && exp2(y) >= least)
                over += w;
        });
        __syncthreads();
        uint32_t c = r.count[tid];
        u64 m = r.mass[tid];
        scan(r, c, m);
        r.count[tid] = c;
        r.mass[tid] = m;
        if (tid == 0)
            r.answer = 0;
        __syncthreads();
        if (over)
            atomicAdd(&r.answer, over);
        __syncthreads();
        over = r.answer;
        const u64 total = r.mass[kBuckets - 1];
        const uint32_t weighty = r.count[kBuckets - 1];
        u64 mass = total;
        if (!s.greedy) {
            const int k = a.top_k ? a.top_k[at] : 0;
            if (k > 0 && (uint32_t)k < weighty)
                mass = reach(r, s, row, vocab, true, (u64)k).mass;
            const float p = a.top_p ? a.top_p[at] : 1.0f;
            if (p < 1.0f) {
                const double want = (double)p * (double)mass;
                u64 target = want > 0.0 ? (u64)__builtin_ceil(want) : 1;
                target = target < 1 ? 1 : target > mass ? mass : target;
                const u64 kept = reach(r, s, row, vocab, false, target).mass;
                mass = kept < mass ? kept : mass;
            }
            if (least > 0.0)
                mass = over < mass ? over : mass;
        }
        u64 target = 1;
        if (!s.greedy && mass) {
            const double want = (double)a.u[at] * (double)mass;
            target = want >= 1.0 ? (want >= (double)mass ? mass : (u64)want + 1) : 1;
            target = target > mass ? mass : target;
        }
        const Place p = reach(r, s, row, vocab, false, target);
        if (tid == 0) {
            a.token[at] = (uint32_t)~(uint32_t)p.token;
            if (a.logprob) {
                const double y = log2_weight(s, logit_of((uint32_t)(p.token >> 32)));
                a.logprob[at] = s.greedy ? 0.0f
                                         : (float)(y * 0.69314718055994530942 - log(__builtin_ldexp((double)total, -s.bits)));
            }
        }
        __syncthreads();
    }
}

int64_t sample_work(const bq_draw &) { return 0; }

hipError_t launch_sample(const bq_draw &a, hipStream_t st)
{
    const int64_t most = int64_t(1) << 21;
    const dim3 grid((unsigned)(a.rows < most ? a.rows : most)), block(kSampleThreads);
    switch (a.type) {
    case BQ_F16: hipLaunchKernelGGL((sample_kernel<_Float16>), grid, block, 0, st, a); break;
    case BQ_BF16: hipLaunchKernelGGL((sample_kernel<__bf16>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((sample_kernel<float>), grid, block, 0, st, a); break;
    }
    return hipGetLastError();
}

}  // namespace bq
