/*
 * bq.h -- C ABI of libbq: 1-bit (Q1_0) and ternary (Q2_0) quantized
 * matrix-vector products on AMD Instinct MI355X (gfx950).
 *
 * The operation (bankML "gpu/ -- the video-card component", section
 * "kernels.rs -- the Q1_0 kernels"): a weight matrix stored as blocks of
 * packed sign bits or ternary codes with one f16 scale per block, times an
 * activation vector quantized to int8 with one f32 scale per block of qa
 * values, gives one f32 dot product per output row.  Every output element is
 * produced in one fixed order:
 *
 *   for each weight block b (Q1_0: 128 weights = 4 sub-blocks of 32;
 *                            Q2_0:  64 weights = 2 sub-blocks of 32):
 *     for each lane L in 0..7 and sub-block j:
 *       s   = exact int32 sum over weights 32j+4L .. 32j+4L+3 of w * q
 *             (Q1_0: w = +1 / -1, and -1 times -128 gives -128 as in an int8
 *              negation; Q2_0: w = code - 1)
 *       ab  = d1(j) * s        (first sub-block)
 *       ab  = fma(d1(j), s, ab) (later sub-blocks)
 *     acc[L] = fma(d0(b), ab, acc[L])        (acc starts at +0)
 *   y = ((acc0+acc4) + (acc2+acc6)) + ((acc1+acc5) + (acc3+acc7))
 *
 * with d0 the block's f16 scale widened exactly and d1(j) the activation
 * scale that covers the first value of sub-block j; every step is one
 * binary32 operation rounded to nearest-even (no flush of subnormals).  The
 * results do not depend on the grid, on how rows are split, or on which call
 * (matvec or sweep) computes them.
 *
 * Conventions for every entry point:
 *   - Return BQ_OK (0) on success or a BQ_E* code; the text of the last
 *     error of the calling thread, naming the call and the argument, is
 *     returned by bq_last_error().  No exception crosses this boundary, no
 *     call aborts, and there is no CPU fallback: a call that cannot run on
 *     the GPU fails.
 *   - Arguments are validated before anything is launched.  A GPU fault
 *     inside a kernel is reported by the caller's next synchronisation of
 *     the stream, not by the launching call.
 *   - "device" pointers are HIP device allocations (for example the
 *     data_ptr() of a torch tensor on a ROCm device); "host" pointers are
 *     ordinary process memory.  The caller allocates and owns every buffer;
 *     the library keeps no pointer after a call returns, except that a sweep
 *     plan keeps the pointers it was created with until it is destroyed.
 *   - GPU work is enqueued on the given stream (a hipStream_t, NULL = the
 *     null stream) and runs asynchronously; calls are reentrant and are
 *     ordered only by their streams.
 */
#ifndef BQ_H
#define BQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BQ_ABI_VERSION 8

/* Weight formats (one canonical block = 18 bytes: f16 scale, little-endian,
 * then 16 payload bytes).
 *   BQ_Q1_0: 128 weights; weight k is bit (k & 7) of payload byte (k >> 3);
 *            bit 1 means +1, bit 0 means -1.
 *   BQ_Q2_0: 64 weights; weight k is bits 2(k&3)..2(k&3)+1 of payload byte
 *            (k >> 2); code c means weight c - 1 (codes 0, 1, 2 are -1, 0, +1;
 *            code 3 decodes as +2 on both the CPU and the GPU). */
#define BQ_Q1_0 1
#define BQ_Q2_0 2

/* Return codes. */
#define BQ_OK 0
#define BQ_EARG 1   /* null pointer, bad shape, unsupported qa / ncols / format */
#define BQ_EALIGN 2 /* a pointer or a leading dimension is not aligned as required */
#define BQ_EHIP 3   /* the HIP runtime reported an error (its text is kept) */
#define BQ_ENOMEM 4 /* a plan could not allocate its device table */

typedef void *bq_stream; /* hipStream_t */

/* A packed weight matrix as laid out by bq_pack (device pointers). */
typedef struct bq_weights {
    int32_t fmt;            /* BQ_Q1_0 or BQ_Q2_0 */
    int32_t reserved;       /* must be 0 */
    int64_t rows;           /* M >= 1 */
    int64_t cols;           /* K >= 1, a multiple of the block length (128 or 64) */
    const void *bits;       /* device, 16-byte aligned: payload plane from bq_pack */
    const uint16_t *scales; /* device, 16-byte aligned: scale plane from bq_pack */
} bq_weights;

/* ncols quantized activation vectors (device pointers), as written by
 * bq_quantize_act_q8: column c is q[c*ld_q .. c*ld_q + n) with scales
 * d[c*ld_d .. c*ld_d + n/qa). */
typedef struct bq_act {
    const int8_t *q; /* device, 16-byte aligned */
    const float *d;  /* device, 4-byte aligned */
    int64_t n;       /* values per column; must equal the weights' cols */
    int32_t qa;      /* values per scale: 32, 64 or 128 (n % qa == 0) */
    int32_t ncols;   /* number of activation columns, 1..16 */
    int64_t ld_q;    /* int8 elements between columns, >= n, multiple of 16 */
    int64_t ld_d;    /* floats between columns, >= n / qa */
} bq_act;

/* One product of a sweep: y = W x for one activation vector. */
typedef struct bq_gemv {
    bq_weights w;
    bq_act a; /* a.ncols must be 1 */
    float *y; /* device, 4-byte aligned: w.rows floats */
} bq_gemv;

/* One product of a sweep that quantizes in the launch: y = W q(x), with q
 * the activation quantizer's output for the f32 vector x. */
typedef struct bq_gemv_x {
    bq_weights w;
    const float *x; /* device, 16-byte aligned: w.cols floats */
    float *y;       /* device, 4-byte aligned: w.rows floats */
} bq_gemv_x;

typedef struct bq_sweep bq_sweep; /* opaque plan */

/* BQ_ABI_VERSION of the loaded library, so that a binding can refuse a
 * library built for another version of this interface instead of passing it
 * structs of another layout (bankML "gpu/ -- the video-card component",
 * section "Advantages and efficiency": checks fail closed).  Host only. */
int bq_abi_version(void);

/* Text of the calling thread's last error ("" if none): the failing call,
 * the argument and why (bankML "gpu/ -- the video-card component", section
 * "Advantages and efficiency": errors name the failing call; OneModel GPU
 * docs, section "Errors": a failure names what was being done).  Owned by
 * the library, thread-local, valid until the thread's next failing call.
 * Host only. */
const char *bq_last_error(void);

/* Sizes in bytes of the two device planes that bq_pack writes for a packed
 * rows x cols matrix of format fmt (bankML "gpu/ -- the video-card
 * component", section "kernels.rs -- the Q1_0 kernels": weights are
 * repacked once into the card's layout, bits as 32-bit words).  Writes
 * *bits_bytes and *scale_bytes (host pointers) and returns BQ_OK, or BQ_EARG
 * (unknown fmt; rows or cols not in [1, 2^31); cols not a multiple of the
 * block length; a 64-row tile's payload above 2^31 - 16 bytes; a null output
 * pointer) with nothing written.  The sizes come back through pointers so
 * that the result is a return code like every other call.  The planes'
 * layout belongs to the library and changes with BQ_ABI_VERSION (the
 * payload plane may hold unused zero padding between groups of row tiles):
 * size buffers with this call, not with a formula.  Host only; touches no
 * GPU. */
int bq_packed_bytes(int32_t fmt, int64_t rows, int64_t cols, size_t *bits_bytes, size_t *scale_bytes);

/* Repack canonical blocks into the device layout (bankML "gpu/", section
 * "kernels.rs": weights are repacked once, numbers unchanged, only
 * re-ordered).  Host only: canon (host) holds rows x (cols / block length)
 * canonical 18-byte blocks, row-major; bits_out and scales_out (host) must
 * hold the sizes bq_packed_bytes reports.  The caller copies both planes to
 * the device once.  Padding is written as zeros. */
int bq_pack(int32_t fmt, const uint8_t *canon, int64_t rows, int64_t cols, void *bits_out,
            uint16_t *scales_out);

/* Inverse of bq_pack: bits and scales (host, the planes bq_pack wrote for
 * the same fmt, rows, cols) give back the canonical blocks in canon_out
 * (host, rows x (cols / block length) x 18 bytes), byte for byte -- the
 * repacking changes no number, it only re-orders them (bankML "gpu/ -- the
 * video-card component", section "kernels.rs -- the Q1_0 kernels").
 * Returns BQ_OK, or BQ_EARG (shape as bq_packed_bytes, null pointer).
 * Host only. */
int bq_unpack(int32_t fmt, const void *bits, const uint16_t *scales, int64_t rows, int64_t cols,
              uint8_t *canon_out);

/* The activation quantizer: the int8 activation with one scale per block
 * that the products read (bankML "gpu/ -- the video-card component",
 * section "kernels.rs -- the Q1_0 kernels": the activation binding holds
 * f32 scales, one per 32 values, and int8 quants, and the activation is
 * repacked per call; here the block length qa is a parameter, 128 in the
 * configured workloads).  Quantize n floats x (device, 16-byte aligned) in
 * blocks of qa values: d = amax / 127 (f32, correctly rounded), q = x / d
 * (correctly rounded) rounded half away from zero into [-127, 127]; an
 * all-zero block gives d = 0 and q = 0.  q (device, 4-byte aligned)
 * receives n int8 values and d (device, 4-byte aligned) n / qa floats.  qa
 * is 32, 64 or 128; n % qa == 0 (n = 0 does nothing).  Non-finite inputs are
 * outside the contract.  Returns BQ_EARG / BQ_EALIGN before any launch, or
 * BQ_EHIP if the launch fails.  Allocates nothing.  Asynchronous on s. */
int bq_quantize_act_q8(const float *x, int64_t n, int32_t qa, int8_t *q, float *d, bq_stream s);

/* The same quantizer with f16-valued scales, the flavour of the pages' q8_0
 * activation (bankML "gpu/", section "kernels.rs -- the Q1_0 kernels": the
 * activation binding holds one scale per 32 values; section "Advantages and
 * efficiency": d1*s is exact in f32, which holds when d1 has at most 11
 * significant bits).  Per block of qa values: d = amax / 127 (correctly
 * rounded), then narrowed to the nearest f16 value (ties to even) and stored
 * widened in d; q = x / d (correctly rounded) rounded half away from zero,
 * clamped to [-127, 127] -- the clamp can bind when d falls in the f16
 * subnormal range (amax < 127 * 2^-14).  d == 0 (also when amax / 127
 * narrows to 0) gives q = 0.  Blocks with amax / 127 >= 65520 (d = +inf)
 * are outside the contract, as are non-finite inputs.  Arguments, alignment
 * and errors as bq_quantize_act_q8.  Asynchronous on s. */
int bq_quantize_act_q8_f16(const float *x, int64_t n, int32_t qa, int8_t *q, float *d, bq_stream s);

/* The product itself (bankML "gpu/ -- the video-card component", section
 * "kernels.rs -- the Q1_0 kernels": one f32 dot product per row, in the
 * order given at the top of this file; Q2_0 by the same order, readings of
 * the format noted above).  y (device, 4-byte aligned, a.ncols * w->rows
 * floats; column c at y + c * rows) = W times each activation column.
 * w (host struct, device planes) must have fmt BQ_Q1_0 (resp. BQ_Q2_0 for
 * the second call); a (host struct, device arrays) must have a->n ==
 * w->cols.  Returns BQ_EARG / BQ_EALIGN before any launch, or BQ_EHIP if the
 * launch fails.  Allocates nothing.  Asynchronous on s. */
int bq_q1_0_matvec(const bq_weights *w, const bq_act *a, float *y, bq_stream s);
int bq_q2_0_matvec(const bq_weights *w, const bq_act *a, float *y, bq_stream s);

/* Which kernels compute the lane-group sums of bq_q1_0_matvec /
 * bq_q2_0_matvec for 2 to 16 activation columns: BQ_BATCH_AUTO (the path
 * measured faster for the shape and column count), BQ_BATCH_TABLES (LDS
 * lookup tables of the activation, the VALU path) or BQ_BATCH_MFMA (exact
 * integer sums on the matrix cores, as products with a block-diagonal
 * activation matrix; the f32 chain of the order above stays on the VALU).  Both paths give the same
 * bits; the choice affects only speed.  The sums are the integer part of
 * bankML "gpu/ -- the video-card component", section "kernels.rs -- the
 * Q1_0 kernels" (exact lane-group sums before the chain).  Process-wide,
 * atomic; calls already launched keep their path.  Returns the previous
 * setting, or -1 (with BQ_EARG's message) for an unknown path.  Host only. */
#define BQ_BATCH_AUTO 0
#define BQ_BATCH_TABLES 1
#define BQ_BATCH_MFMA 2
int bq_set_batch_path(int path);

/* One group of a dependency-ordered decode step in ONE launch: the count
 * products (1..4) that read the same activation -- bankML "gpu/ -- the
 * video-card component", section "Limitations": Q/K/V, and gate/up, are
 * submitted together with one wait per group.  x (device, 16-byte aligned)
 * holds the f32 activation of length w[0].cols; it is quantized in blocks of
 * qa exactly as bq_quantize_act_q8 would (the quants stay on chip) and
 * y[i] (device, 4-byte aligned, w[i].rows floats) receives what
 * bq_q1_0_matvec / bq_q2_0_matvec would write for w[i] and those quants.
 * Every w[i] must share w[0]'s format and cols (a multiple of qa); qa is
 * 32, 64 or 128.  No y[i] may overlap x.  w and y are host arrays of count
 * entries, read during the call.  Allocates nothing.  Asynchronous on s. */
int bq_group_matvec(const bq_weights *w, int32_t count, const float *x, int32_t qa, float *const *y,
                    bq_stream s);

/* A plan for many independent products run by ONE kernel launch (the 253
 * products of one decode token: bankML "par.rs -- the persistent thread pool
 * and row scheduler", section "Summary").  All entries must share one format
 * and one qa, with ncols == 1.  Validates every entry, balances the work
 * over the GPU and copies a descriptor table to the device (the plan's only
 * allocation, freed by bq_sweep_destroy).  Must be called with the device of
 * the pointers current.  *plan receives the plan, or NULL on failure. */
int bq_sweep_create(const bq_gemv *list, int32_t count, bq_sweep **plan);

/* As bq_sweep_create, for products whose activations are f32 vectors that
 * the launch itself quantizes: every workgroup quantizes the blocks of x it
 * needs into on-chip memory, with bq_quantize_act_q8's rule and block length
 * qa (32, 64 or 128; every w.cols a multiple of qa), before building its
 * tables, so a decode token's products run from their f32 inputs in one
 * launch and the int8 vectors never go to memory (bankML "par.rs -- the
 * persistent thread pool and row scheduler", section "Summary": one token's
 * 253 products; bankML "gpu/ -- the video-card component", section
 * "kernels.rs -- the Q1_0 kernels": the activation is quantized per call).
 * Each y equals what bq_quantize_act_q8 followed by bq_q1_0_matvec /
 * bq_q2_0_matvec would give.  No y may overlap an x.  Allocation, errors and
 * ownership as bq_sweep_create; run and release the plan with
 * bq_token_sweep and bq_sweep_destroy. */
int bq_sweep_create_x(const bq_gemv_x *list, int32_t count, int32_t qa, bq_sweep **plan);

/* Enqueue the whole plan on s as ONE kernel launch (bankML "gpu/ -- the
 * video-card component", section "Limitations": each of the token's 253
 * matrix calls paid one submit and wait there; here the token is one
 * submission).  Each entry's y equals what bq_q1_0_matvec / bq_q2_0_matvec
 * would write for it; the plan's pointers must still be valid.  Returns
 * BQ_EARG (null plan) or BQ_EHIP if the launch fails.  Allocates nothing.
 * Asynchronous on s. */
int bq_token_sweep(const bq_sweep *plan, bq_stream s);

/* The sweep of bq_sweep_create + bq_token_sweep in ONE call that allocates
 * nothing, for callers that cannot allocate memory: code under HIP graph
 * capture, tight serving loops, and harnesses that forbid hipMalloc.  The
 * list (host array of count bq_gemv, rules as bq_sweep_create) is validated
 * and planned on fixed host storage, and the plan (descriptors and work
 * items) is copied on s into a fixed device array of the library: 320 KiB
 * per GPU, held until the process ends, room for up to 1024 products and
 * 16384 work items (the 253 products of a decode token need 1,743 in Q1_0,
 * 2,029 in Q2_0).
 * Larger lists are refused with BQ_EARG, as is every invalid entry, before
 * anything is copied or launched.  The copy is from pageable memory, so the
 * call returns once the table is staged; it may wait for earlier work on s.
 * Each entry's y equals what bq_token_sweep of a bq_sweep_create plan of the
 * same list writes.  All calls on one GPU share that GPU's array: calls on
 * one stream are ordered, but calls that overlap on one GPU (several streams
 * or threads with launches in flight together) race on it.  Calls from
 * several host threads are serialised while they plan.  Returns BQ_OK,
 * BQ_EARG / BQ_EALIGN, or BQ_EHIP if the copy or the launch fails.
 * Asynchronous on s. */
int bq_token_sweep_noalloc(const bq_gemv *list, int32_t count, bq_stream s);

/* Release a plan and its device table (NULL is allowed): resources are
 * released only by an explicit call, never behind the caller's back (bankML
 * "gpu/ -- the video-card component", section "compute.rs -- Vulkan
 * compute": a buffer is released only by the free call).  Synchronises the
 * device first, so launches of the plan still in flight finish. */
void bq_sweep_destroy(bq_sweep *plan);

/* The streaming-read floor, a measurement aid and not a step of the
 * product (bankML "par.rs -- the persistent thread pool and row scheduler",
 * sections "How it is verified" and "Advantages and efficiency": the memory
 * floor a token's weight stream is compared against).  Reads every byte of
 * p (device, 16-byte aligned, bytes a positive multiple of 16) once with
 * plain 16-byte loads from a fixed grid and writes BQ_FLOOR_SINK_WORDS
 * uint32 to sink (device, 4-byte aligned): the XOR of all of them equals
 * the XOR of all 32-bit words of the buffer.  Time it with events to get
 * the read bandwidth a kernel can reach on this GPU.  Allocates nothing.
 * Asynchronous on s. */
#define BQ_FLOOR_SINK_WORDS 8192
int bq_read_floor(const void *p, int64_t bytes, uint32_t *sink, bq_stream s);

/* ------------------------------------------------------------------------
 * Between the products: the operators that turn the outputs of one group of
 * products into the activation of the next, for 1 to many tokens at once
 * (bankML "par.rs -- the persistent thread pool and row scheduler", section
 * "Summary", counts the 253 products of a token; a decode or prompt step
 * runs these between them).  All conventions above hold.  Every argument
 * block is a host struct read during the call; `reserved` fields must be 0.
 *
 * Tensors of these calls hold one of three types; a 16-bit result is rounded
 * once, to nearest even, from f32. */
#define BQ_F32 0
#define BQ_F16 1
#define BQ_BF16 2

/* Residual addition, root-mean-square norm and activation quantizer in one
 * pass: for each of `tokens` rows of n values,
 *   h    = x + res, rounded to `type` (x itself where res is NULL)
 *   r    = 1 / sqrt(sum(h^2) / n + eps), summed and evaluated in binary64
 *          and rounded once to binary32
 *   v    = (h * r) * w, each product rounded to binary32
 *   d    = max|v| * (1 / 127) over each block of qa, both in binary32 (with
 *          f16_scale narrowed to f16, nearest even, as bq_quantize_act_q8_f16
 *          does), within one unit in the last place of amax / 127
 *   q    = v / d (correctly rounded) rounded half away from zero, clamped to
 *          [-127, 127]; d = 0 gives 0
 *   y    = v rounded to `type`
 * so q and d are the same bits whatever order the sum is taken in (but for a
 * sum within 2^-50 of where r rounds the other way), the bits that elementwise
 * tensor operations on the GPU give, which divide by a constant as a product
 * with its reciprocal.  They feed the products
 * as bq_act {q, d, n, qa, ncols = tokens, ld_q, ld_d}.
 * x, res, h, w and y hold `type`; rows are ld_* elements apart.  res, h and
 * y may be NULL (absent); h and y may each be x or res (same pointer and
 * leading dimension), and not otherwise overlap them.  n is a multiple of
 * qa, at most BQ_NORM_MAX; qa is 32, 64 or 128; eps >= 1e-30.  x, res, h, y and w
 * are 16-byte aligned, their leading dimensions (and ld_q) multiples of 16
 * bytes; q is 8-byte aligned with ld_q a multiple of 16, d 4-byte.  tokens =
 * 0 does nothing.  Non-finite values are outside the contract, as in the
 * quantizer.  Returns BQ_EARG / BQ_EALIGN before any launch, or BQ_EHIP.
 * Allocates nothing.  Asynchronous on s. */
#define BQ_NORM_MAX 65536
typedef struct bq_norm {
    int32_t type;      /* BQ_F32, BQ_F16 or BQ_BF16 */
    int32_t qa;        /* values per scale */
    int32_t f16_scale; /* 0, or 1: f16-valued scales */
    int32_t reserved;
    double eps;
    int64_t tokens;
    int64_t n;
    const void *x;
    int64_t ld_x;
    const void *res;
    int64_t ld_res;
    void *h;
    int64_t ld_h;
    const void *w;
    int8_t *q;
    int64_t ld_q;
    float *d;
    int64_t ld_d;
    void *y;
    int64_t ld_y;
} bq_norm;
int bq_rmsnorm_q8(const bq_norm *a, bq_stream s);

/* A paged cache of keys and values (device, 16-byte aligned, owned by the
 * caller).  Place p of the cache is offset p % page of page p / page.  Keys
 * lie as [pages][heads][page][dim]; values as [pages][heads][dim][page], the
 * tokens of a page side by side for each value index, because the attention
 * sums over tokens and reads the operand of its matrix products so without
 * moving it.  Nothing reads a place before a token was written there. */
typedef struct bq_kv_cache {
    int32_t type;  /* BQ_F16 or BQ_BF16 */
    int32_t heads; /* key heads, 1..1024 */
    int32_t dim;   /* values per head: 64 or 128 */
    int32_t page;  /* tokens per page: a power of two, 16..256 */
    int64_t pages; /* 1 <= pages, pages * page < 2^31 */
    void *k;
    void *v;
} bq_kv_cache;

/* New tokens into the cache: for each of `tokens` rows t, every query and
 * key head is normed (v * (1 / sqrt(mean(v^2) + eps)) * norm weight, where
 * q_norm / k_norm is not NULL) and rotated by the token's position: for
 * i < rot / 2 the pair (v[i], v[i + rot/2]) turns by the angle pos[t] *
 * freq[i] (the angle in binary64, so that far positions keep their phase);
 * values from rot on stay.  The key row goes to place slot[t] of the cache,
 * the value row there too (neither normed nor rotated), both rounded to the
 * cache's type; the query row goes to q_out, in `type` or, with q_out_type,
 * in the cache's.  A token whose slot is not in [0, pages * page) (-1: padding of the
 * batch) is not cached; its query row is still written.  Slots that occur
 * twice in a call leave either token's values there, element by element.
 * q, k, v and q_out rows hold their heads end to end, rows ld_* elements
 * apart (q and q_out NULL, q_heads 0: keys and values only); `type` is
 * BQ_F32 or the cache's type.  rot is 0 or a multiple of 16, at most dim.
 * pos (int32) and slot (int64) are device arrays of `tokens`, freq (rot / 2
 * floats), q_norm and k_norm (dim floats) device arrays.  q_out may be q.
 * Pointers are 16-byte aligned (pos, slot, freq and the weights by their
 * element), leading dimensions multiples of 16 bytes.  tokens = 0 does
 * nothing.  Returns BQ_EARG / BQ_EALIGN before any launch, or BQ_EHIP.
 * Allocates nothing.  Asynchronous on s. */
typedef struct bq_append {
    bq_kv_cache cache;
    int32_t type;       /* of q, k and v */
    int32_t q_out_type; /* of q_out: `type` or the cache's type */
    int32_t q_heads;    /* 0..1024 */
    int32_t rot;
    float eps; /* > 0 where a norm weight is given */
    int32_t reserved;
    int64_t tokens;
    const void *q;
    int64_t ld_q;
    const void *k;
    int64_t ld_k;
    const void *v;
    int64_t ld_v;
    void *q_out;
    int64_t ld_qo;
    const int32_t *pos;
    const int64_t *slot;
    const float *freq;
    const float *q_norm;
    const float *k_norm;
} bq_append;
int bq_kv_append(const bq_append *a, bq_stream s);

/* Causal attention of the new tokens of several requests over the paged
 * cache that already holds them.  Request b has rows cu[b] .. cu[b+1] - 1 of
 * q (n of them, any number from 0) and lens[b] = L keys, key j at place
 * table[b][j / page] * page + j % page; its row i sees the keys j <= L - n + i:
 *   o = sum_j exp(scale q.k_j - m) v_j / sum_j exp(scale q.k_j - m)
 * per query head, the q_heads / heads query heads of a key head together.
 * A row that sees no key (L < n) is 0.  Rows of out at or behind
 * cu[requests] are left as they were.  One token per request is a decode
 * step, n = L a whole prompt, anything between a chunk of one.
 * q and out (q_heads heads of dim end to end, rows ld_* elements apart) hold
 * `type`: BQ_F32 or the cache's type.  With f32 rows the matrix products run
 * on the cache's 16-bit type with q and the weights exp(..) split into parts
 * that carry 22 bits or more, so out is good to f32 sums; with 16-bit rows
 * the weights are rounded to that type once, which costs as much as rounding
 * out does.  Softmax statistics and sums are f32.
 * cu (requests + 1), lens and table (requests rows, ld_table entries apart,
 * table_cols of them each) are int32 device arrays, so that a captured graph
 * can be replayed with other lengths; max_new and max_keys (host) bound the
 * new tokens and keys of any request, and only affect how the work is split
 * (larger counts are still computed).  cu ascends from 0 or more.  What the
 * device arrays say is bounded in the kernel: rows past `tokens`, keys past
 * table_cols * page and pages outside the cache are not read (keys of such a
 * page count as unseen), and a request that starts below 0, at or past
 * `tokens`, or at or past its end has no rows.
 * Places of keys below L must hold finite values; others may hold anything.
 * q is finite: the result of a row and head whose query is not has no defined
 * value; the others' are not touched by it.
 * work (device, 16-byte aligned, bq_paged_attn_work_bytes bytes -- some tens
 * of megabytes at most, whatever the tokens and keys -- may be NULL if that is
 * 0) is scratch of this call until it has run: calls that may run at the same
 * time need one each.  out must not overlap q.  tokens = 0 or
 * requests = 0 does nothing.  Returns BQ_EARG / BQ_EALIGN before any launch,
 * or BQ_EHIP.  Allocates nothing.  Asynchronous on s. */
typedef struct bq_attn {
    bq_kv_cache cache;
    int32_t type;    /* of q and out */
    int32_t q_heads; /* a multiple of cache.heads, at most 16 query heads per key head */
    int32_t requests;
    int32_t table_cols;
    int64_t ld_table;
    int64_t tokens; /* rows of q and out, < 2^31 */
    int64_t max_new;
    int64_t max_keys;
    const void *q;
    int64_t ld_q;
    void *out;
    int64_t ld_out;
    const int32_t *cu;
    const int32_t *lens;
    const int32_t *table;
    float scale;
    int32_t reserved;
    void *work;
    int64_t work_bytes;
} bq_attn;
int bq_paged_attn(const bq_attn *a, bq_stream s);

/* Bytes of `work` that bq_paged_attn needs for this argument block (its
 * pointers are not read).  Host only. */
int bq_paged_attn_work_bytes(const bq_attn *a, int64_t *bytes);

/* Low-rank adapters of many requests beside a shared projection: request b
 * has rows cu[b] .. cu[b+1] - 1 of x, y and out, and adapter ids[b]:
 *   out = y + gain[id] * B_id (A_id x)
 * with A_id (rank x n) at a + id * rank * n and B_id (rows x rank) at
 * b + id * rows * rank.  A request whose id is not in [0, count) (-1: none)
 * gets out = y.  Rows at or behind cu[requests] are left as they were.
 * y and out are f32, as the products write them (column c of
 * bq_q1_0_matvec's y is row c here); out may be y.  x holds x_type: BQ_F32
 * or the adapters' type.  Sums are f32; f32 values enter the matrix products
 * in parts that carry 22 bits or more.  x, A and B are finite, and so are A x
 * and the results: a row of x that is not, or whose A x is not, has NaN where
 * the formula may have an infinity; the other rows are not touched by it.
 * cu (requests + 1, ascending from 0 or more) and ids are int32 device
 * arrays, gain f32; rows past `tokens` are not touched, a request that ends in
 * front of its start has none; max_new (host) bounds the rows of any request
 * and only affects how the work is split.  tokens is at most 2^31 - 64, n a
 * multiple of 8 below 2^31, rank a multiple of 8 up to 128, requests at most
 * 2^30, rows below 2^23.  x, a, b and work are 16-byte aligned, ld_x a multiple
 * of 16 bytes; y and out 4-byte.  work (bq_adapters_work_bytes bytes) is scratch
 * of this call until it has run: calls that may run at the same time need one
 * each.  tokens = 0 or requests = 0 does nothing.  Returns BQ_EARG / BQ_EALIGN
 * before any launch, or BQ_EHIP.  Allocates nothing.  Asynchronous on s. */
typedef struct bq_adapters {
    int32_t type;   /* of a and b: BQ_F16 or BQ_BF16 */
    int32_t x_type; /* BQ_F32 or type */
    int32_t rank;
    int32_t count;
    int32_t requests;
    int32_t reserved;
    int64_t n;
    int64_t rows;
    int64_t tokens;
    int64_t max_new;
    const void *a;
    const void *b;
    const float *gain;
    const void *x;
    int64_t ld_x;
    const int32_t *cu;
    const int32_t *ids;
    const float *y;
    int64_t ld_y;
    float *out;
    int64_t ld_out;
    void *work;
    int64_t work_bytes;
} bq_adapters;
int bq_adapters_add(const bq_adapters *a, bq_stream s);
int bq_adapters_work_bytes(const bq_adapters *a, int64_t *bytes);

/* ------------------------------------------------------------------------
 * Around the layers: what a step of generation runs besides the products of
 * 1 to 16 columns and the operators above -- the rows of its tokens, the
 * products of a prompt, the gated activation, the next token.  The
 * conventions of the section above hold. */

/* Activation functions, evaluated on x:
 *   BQ_NONE   x
 *   BQ_SILU   x / (1 + exp(-x))
 *   BQ_GELU   x / (1 + exp(-2 z)), z = sqrt(2 / pi) (x + 0.044715 x^3), which is
 *             x (1 + tanh(z)) / 2
 *   BQ_RELU2  max(x, 0)^2 */
#define BQ_NONE 0
#define BQ_SILU 1
#define BQ_GELU 2
#define BQ_RELU2 3

/* Rows of a token table, scaled: out[t] = scale * table[ids[t]], each product
 * rounded once to f32 (a packed weight times its block scale is exact) and
 * then to `type`.  The table has w.rows rows of w.cols values: packed as the
 * products' weights (w.fmt BQ_Q1_0 or BQ_Q2_0; the LM head's planes serve
 * both), or, with w.fmt 0, dense values of dense_type, rows ld_dense elements
 * apart (w.bits, w.scales NULL; dense NULL where w.fmt is not 0).  A token
 * whose id is not in [0, w.rows) (-1: padding) gets a row of zeros.  ids is
 * an int64 device array.  Dense rows and rows of out are 16-byte aligned
 * (leading dimensions multiples of 16 bytes), w.cols a multiple of 8 below
 * 2^31, and of a packed table as in bq_pack: a multiple of the block length,
 * at most 268,435,328 (Q1_0) or 134,217,664 (Q2_0).  scale is finite.
 * out must not overlap the table or ids.  tokens = 0 does nothing.  Returns
 * BQ_EARG / BQ_EALIGN before any launch, or BQ_EHIP.  Allocates nothing.
 * Asynchronous on s. */
typedef struct bq_table {
    bq_weights w;
    const void *dense;
    int64_t ld_dense;
    int32_t dense_type;
    int32_t type; /* of out */
    float scale;
    int32_t reserved;
    int64_t tokens;
    const int64_t *ids;
    void *out;
    int64_t ld_out;
} bq_table;
int bq_embed(const bq_table *a, bq_stream s);

/* Activation, gate and activation quantizer in one pass: for each of `tokens`
 * rows of n values,
 *   v = act(gate) * up, evaluated in binary64 and rounded once to f32
 *   d, q as bq_rmsnorm_q8 forms them from v (blocks of qa, f16_scale)
 *   y = v rounded to `type`
 * so q and d do not hang on how exp is computed, but for a v that lies within
 * 2^-50 of its size (BQ_GELU: within (1 + 2 |z|) 2^-50, z as above at the gate,
 * whose rounding exp magnifies) of where it rounds the other way.  gate, up
 * and y hold `type`, rows ld_* elements apart; y may be NULL, gate or up (same
 * leading dimension), and not otherwise overlap them.  n is a multiple of qa
 * below 2^31, qa 32, 64 or 128.  gate, up and y rows are 16-byte aligned, q
 * 8-byte with ld_q a multiple of 16, d 4-byte.  Values are finite, act(gate) *
 * up too.
 * tokens = 0 does nothing.  Returns BQ_EARG / BQ_EALIGN before any launch, or
 * BQ_EHIP.  Allocates nothing.  Asynchronous on s. */
typedef struct bq_gated {
    int32_t type;
    int32_t act; /* BQ_NONE .. BQ_RELU2 */
    int32_t qa;
    int32_t f16_scale; /* 0 or 1 */
    int64_t tokens;
    int64_t n;
    const void *gate;
    int64_t ld_gate;
    const void *up;
    int64_t ld_up;
    int8_t *q;
    int64_t ld_q;
    float *d;
    int64_t ld_d;
    void *y;
    int64_t ld_y;
} bq_gated;
int bq_gated_q8(const bq_gated *a, bq_stream s);

/* A packed matrix times the quantized activations of any number of tokens:
 *   y[t, r] = act(sum_k W[r, k] x[t, k] + bias[r]) * mul[t, r] + res[t, r]
 * with x[t, k] = q[t, k] d[t, k / qa] as the quantizers write it (a.ncols
 * tokens, 1 to 2^31 - 2^16 of them).  For every block of weights and its
 * activation scale the sum of w * q is an exact integer; each is scaled by d0
 * (rounded to f32) and added with d1 by one fma, in f32, in no promised order
 * over the blocks: the numbers of bq_q1_0_matvec / bq_q2_0_matvec to f32
 * sums, not their bits.  (A quant of -128, which no quantizer writes, times
 * -1 gives +128 here.)  Epilogue in f32: bias (f32, w.rows of them), act, mul
 * and res (both of `type`, as y), each where it is not NULL / BQ_NONE; y is
 * rounded once.  y may be mul or res (same leading dimension), and not
 * otherwise overlap an input.  Scales and results are finite.
 * a.q, w's planes and work are 16-byte aligned (a.ld_q a multiple of 16); the
 * other arrays by their elements, with any leading dimension of at least
 * w.rows.  w.cols is at most 268,435,328 (Q1_0) or 134,217,664 (Q2_0).
 * work (bq_matmul_work_bytes bytes; may be NULL if that is 0) is scratch of
 * this call until it has run: calls that may run at the same time need one
 * each.  a.ncols = 0 does nothing.  Returns BQ_EARG / BQ_EALIGN before any
 * launch, or BQ_EHIP.  Allocates nothing.  Asynchronous on s. */
typedef struct bq_product {
    bq_weights w;
    bq_act a;
    int32_t type; /* of y, mul and res */
    int32_t act;
    const float *bias;
    const void *mul;
    int64_t ld_mul;
    const void *res;
    int64_t ld_res;
    void *y;
    int64_t ld_y;
    void *work;
    int64_t work_bytes;
} bq_product;
int bq_matmul(const bq_product *a, bq_stream s);

/* Bytes of `work` that bq_matmul needs for this argument block (its pointers
 * are not read).  Host only. */
int bq_matmul_work_bytes(const bq_product *a, int64_t *bytes);

/* The next token of each of `rows` rows of vocab logits.  With m the row's
 * largest logit and T its temperature, token i weighs exp((logit[i] - m) / T);
 * the tokens stand in descending order of their logits, equal ones by index.
 * Kept are the first of that order, as many as the shortest of these:
 *   top_k  the first top_k                    (top_k <= 0: all)
 *   top_p  the fewest whose weights add up to at least top_p times the weight
 *          of those that top_k keeps          (top_p >= 1: all)
 *   min_p  those that weigh at least min_p, the largest weight being 1
 *                                             (min_p <= 0: all)
 * but at least one.  token is the first of the kept ones at which the running
 * sum of the weights passes u times their sum (u in [0, 1); others are taken
 * as the nearer end), logprob the logarithm of its weight over that of all
 * tokens before the filters.  temperature <= 0 (or NaN) takes the first of the
 * largest logits, with logprob 0.
 * Weights are evaluated in binary64 and rounded to multiples of 2^-b (b =
 * 62 minus the bits of vocab, 39 at least, at most 50), and added up exactly: the
 * result is the same on any split of the work.
 * A logit that is NaN or -infinity has no weight; with +infinities only those
 * weigh.  A row without weight gives token -1 and logprob -infinity.
 * logits hold `type`, rows ld_logits elements apart (any, at least vocab);
 * vocab is 1 to 2^22.  u, temperature, top_p, min_p (f32) and top_k (int32)
 * are device arrays of `rows`; all but u may be NULL (temperature 1, no
 * filter).  token is an int64, logprob an f32 device array (may be NULL).
 * Arrays are aligned by their elements, work 16-byte.
 * work (bq_sample_work_bytes bytes; may be NULL if that is 0) is scratch of
 * this call until it has run: calls that may run at the same time need one
 * each.  rows = 0 does nothing.  Returns BQ_EARG / BQ_EALIGN before any
 * launch, or BQ_EHIP.  Allocates nothing.  Asynchronous on s. */
#define BQ_VOCAB_MAX (1 << 22)
typedef struct bq_draw {
    int32_t type;
    int32_t reserved;
    int64_t rows;
    int64_t vocab;
    const void *logits;
    int64_t ld_logits;
    const float *u;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    int64_t *token;
    float *logprob;
    void *work;
    int64_t work_bytes;
} bq_draw;
int bq_sample(const bq_draw *a, bq_stream s);

/* Bytes of `work` that bq_sample needs for this argument block (its pointers
 * are not read).  Host only. */
int bq_sample_work_bytes(const bq_draw *a, int64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* BQ_H */
