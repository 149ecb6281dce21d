// bq_layer.cpp -- the entry points of the operators between the products
// (include/bq.h): argument checks, before anything is launched, and the launch.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>

#include "bq_check.h"
#include "bq_layer.h"
#include "bq_layout.h"

using namespace bq;

namespace {

constexpr int64_t kKeysMax = (int64_t(1) << 31) - (1 << 16);
// the adapters' kernels count rows in 32 bits up to a tile of 32 past the last one
constexpr int64_t kAdapterTokens = kRowsMax - 64;

int check_cache(const char *fn, const bq_kv_cache &c)
{
    if (c.type != BQ_F16 && c.type != BQ_BF16)
        return set_error(BQ_EARG, "%s: cache type %d is not BQ_F16 or BQ_BF16", fn, (int)c.type);
    if (c.heads < 1 || c.heads > 1024)
        return set_error(BQ_EARG, "%s: cache heads %d not in [1, 1024]", fn, (int)c.heads);
    if (c.dim != 64 && c.dim != 128)
        return set_error(BQ_EARG, "%s: cache dim %d is not 64 or 128", fn, (int)c.dim);
    if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1)))
        return set_error(BQ_EARG, "%s: page %d is not a power of two in [16, 256]", fn, (int)c.page);
    if (c.pages < 1 || c.pages >= kRowsMax || c.pages * c.page >= kRowsMax)
        return set_error(BQ_EARG, "%s: pages %lld of %d tokens: not in [1, 2^31) tokens", fn, (long long)c.pages,
                         (int)c.page);
    return BQ_OK;
}

int check_planes(const char *fn, const bq_kv_cache &c)
{
    if (!c.k || !c.v)
        return set_error(BQ_EARG, "%s: null cache plane", fn);
    if (!aligned(c.k, 16) || !aligned(c.v, 16))
        return set_error(BQ_EALIGN, "%s: cache planes must be 16-byte aligned", fn);
    return BQ_OK;
}

// The checks of bq_paged_attn that read no pointer, enough to plan the call.
int check_attn(const char *fn, const bq_attn *a)
{
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    int rc = check_cache(fn, a->cache);
    if (!rc)
        rc = check_tokens(fn, a->tokens);
    if (rc)
        return rc;
    if (a->reserved != 0)
        return set_error(BQ_EARG, "%s: reserved must be 0", fn);
    if (a->type != BQ_F32 && a->type != a->cache.type)
        return set_error(BQ_EARG, "%s: type %d is neither BQ_F32 nor the cache's type %d", fn, (int)a->type,
                         (int)a->cache.type);
    if (a->q_heads < 1 || a->q_heads % a->cache.heads || a->q_heads / a->cache.heads > 16)
        return set_error(BQ_EARG, "%s: q_heads %d is not 1 to 16 times the cache's heads %d", fn, (int)a->q_heads,
                         (int)a->cache.heads);
    if (a->requests < 0 || a->requests > 65535)
        return set_error(BQ_EARG, "%s: requests %d not in [0, 65535]", fn, (int)a->requests);
    if (a->table_cols < 1 || (int64_t)a->table_cols * a->cache.page > kKeysMax)
        return set_error(BQ_EARG, "%s: table_cols %d: not in [1, 2^31 - 2^16] keys", fn, (int)a->table_cols);
    if (a->max_new < 1 || a->max_new >= kRowsMax)
        return set_error(BQ_EARG, "%s: max_new %lld not in [1, 2^31)", fn, (long long)a->max_new);
    if (a->max_keys < 0 || a->max_keys > kKeysMax)
        return set_error(BQ_EARG, "%s: max_keys %lld not in [0, 2^31 - 2^16]", fn, (long long)a->max_keys);
    if (a->tokens * a->q_heads >= kRowsMax)
        return set_error(BQ_EARG, "%s: tokens %lld times q_heads %d not below 2^31", fn, (long long)a->tokens,
                         (int)a->q_heads);
    return BQ_OK;
}

int check_adapters(const char *fn, const bq_adapters *a)
{
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    if (a->tokens < 0 || a->tokens > kAdapterTokens)
        return set_error(BQ_EARG, "%s: tokens %lld not in [0, 2^31 - 64]", fn, (long long)a->tokens);
    if (a->reserved != 0)
        return set_error(BQ_EARG, "%s: reserved must be 0", fn);
    if (a->type != BQ_F16 && a->type != BQ_BF16)
        return set_error(BQ_EARG, "%s: type %d is not BQ_F16 or BQ_BF16", fn, (int)a->type);
    if (a->x_type != BQ_F32 && a->x_type != a->type)
        return set_error(BQ_EARG, "%s: x_type %d is neither BQ_F32 nor the adapters' type %d", fn, (int)a->x_type,
                         (int)a->type);
    if (a->rank < 8 || a->rank > 128 || a->rank % 8)
        return set_error(BQ_EARG, "%s: rank %d is not a multiple of 8 in [8, 128]", fn, (int)a->rank);
    if (a->count < 1)
        return set_error(BQ_EARG, "%s: count %d below 1", fn, (int)a->count);
    if (a->requests < 0 || a->requests > (1 << 30))
        return set_error(BQ_EARG, "%s: requests %d not in [0, 2^30]", fn, (int)a->requests);
    if (a->n < 8 || a->n % 8 || a->n >= kRowsMax)
        return set_error(BQ_EARG, "%s: n %lld is not a multiple of 8 in [8, 2^31)", fn, (long long)a->n);
    if (a->rows < 1 || a->rows >= (int64_t(1) << 23))
        return set_error(BQ_EARG, "%s: rows %lld not in [1, 2^23)", fn, (long long)a->rows);
    if (a->max_new < 1 || a->max_new >= kRowsMax)
        return set_error(BQ_EARG, "%s: max_new %lld not in [1, 2^31)", fn, (long long)a->max_new);
    return BQ_OK;
}

}  // namespace

BQ_EXPORT int bq_rmsnorm_q8(const bq_norm *a, bq_stream s)
{
    const char *fn = "bq_rmsnorm_q8";
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    if (!known(a->type))
        return set_error(BQ_EARG, "%s: type %d unknown", fn, (int)a->type);
    if (a->qa != 32 && a->qa != 64 && a->qa != 128)
        return set_error(BQ_EARG, "%s: qa %d not in {32, 64, 128}", fn, (int)a->qa);
    if (a->f16_scale != 0 && a->f16_scale != 1)
        return set_error(BQ_EARG, "%s: f16_scale %d is not 0 or 1", fn, (int)a->f16_scale);
    if (a->reserved != 0)
        return set_error(BQ_EARG, "%s: reserved must be 0", fn);
    // below that, a zero row's 1 / sqrt(eps) would come near f32's range
    if (!(a->eps >= 1e-30) || !isfinite(a->eps))
        return set_error(BQ_EARG, "%s: eps %g is not a number of at least 1e-30", fn, a->eps);
    int rc = check_tokens(fn, a->tokens);
    if (rc)
        return rc;
    if (a->n < 1 || a->n > BQ_NORM_MAX || a->n % a->qa)
        return set_error(BQ_EARG, "%s: n %lld is not a multiple of qa %d in [1, %d]", fn, (long long)a->n, (int)a->qa,
                         BQ_NORM_MAX);
    if (a->tokens == 0)
        return BQ_OK;
    const int size = size_of(a->type);
    if ((rc = check_rows(fn, "x", a->x, a->ld_x, a->tokens, a->n, size)) ||
        (a->res && (rc = check_rows(fn, "res", a->res, a->ld_res, a->tokens, a->n, size))) ||
        (a->h && (rc = check_rows(fn, "h", a->h, a->ld_h, a->tokens, a->n, size))) ||
        (a->y && (rc = check_rows(fn, "y", a->y, a->ld_y, a->tokens, a->n, size))) ||
        (rc = check_rows(fn, "w", a->w, a->n, 1, a->n, size)))
        return rc;
    const void *const outs[2] = {a->h, a->y}, *const ins[2] = {a->x, a->res};
    const int64_t ld_out[2] = {a->ld_h, a->ld_y}, ld_in[2] = {a->ld_x, a->ld_res};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 2; ++i)
            if (outs[o] && outs[o] == ins[i] && a->tokens > 1 && ld_out[o] != ld_in[i])
                return set_error(BQ_EARG, "%s: h or y in place of x or res needs its leading dimension", fn);
    if (a->h && a->h == a->y)
        return set_error(BQ_EARG, "%s: h and y must not be the same", fn);
    if (!a->q || !a->d)
        return set_error(BQ_EARG, "%s: null q or d", fn);
    if (a->tokens > 1 && (a->ld_q < a->n || a->ld_q > kLdMax || a->ld_d < a->n / a->qa || a->ld_d > kLdMax))
        return set_error(BQ_EARG, "%s: leading dimensions of q or d too small, or above 2^40", fn);
    if (!aligned(a->q, 8) || !aligned(a->d, 4) || (a->tokens > 1 && a->ld_q % 16))
        return set_error(BQ_EALIGN, "%s: q must be 8-byte aligned (ld_q a multiple of 16), d 4-byte aligned", fn);
    NormArgs g;
    g.x = a->x;
    g.res = a->res;
    g.w = a->w;
    g.h = a->h;
    g.y = a->y;
    g.q = a->q;
    g.d = a->d;
    g.ld_x = a->ld_x;
    g.ld_res = a->ld_res;
    g.ld_h = a->ld_h;
    g.ld_y = a->ld_y;
    g.ld_q = a->ld_q;
    g.ld_d = a->ld_d;
    g.n = (int32_t)a->n;
    g.qa = a->qa;
    g.f16_scale = a->f16_scale;
    g.eps = a->eps;
    return launched(fn, launch_norm(a->type, g, a->tokens, static_cast<hipStream_t>(s)));
}

BQ_EXPORT int bq_kv_append(const bq_append *a, bq_stream s)
{
    const char *fn = "bq_kv_append";
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    int rc = check_cache(fn, a->cache);
    if (!rc)
        rc = check_planes(fn, a->cache);
    if (!rc)
        rc = check_tokens(fn, a->tokens);
    if (rc)
        return rc;
    if (a->reserved != 0)
        return set_error(BQ_EARG, "%s: reserved must be 0", fn);
    if (a->type != BQ_F32 && a->type != a->cache.type)
        return set_error(BQ_EARG, "%s: type %d is neither BQ_F32 nor the cache's type %d", fn, (int)a->type,
                         (int)a->cache.type);
    if (a->q_out_type != a->type && a->q_out_type != a->cache.type)
        return set_error(BQ_EARG, "%s: q_out_type %d is neither type %d nor the cache's type %d", fn,
                         (int)a->q_out_type, (int)a->type, (int)a->cache.type);
    if (a->q_heads < 0 || a->q_heads > 1024)
        return set_error(BQ_EARG, "%s: q_heads %d not in [0, 1024]", fn, (int)a->q_heads);
    if (a->rot < 0 || a->rot > a->cache.dim || a->rot % 16)
        return set_error(BQ_EARG, "%s: rot %d is not a multiple of 16 in [0, %d]", fn, (int)a->rot,
                         (int)a->cache.dim);
    if ((a->q_norm || a->k_norm) && (!(a->eps > 0.0f) || !isfinite(a->eps)))
        return set_error(BQ_EARG, "%s: eps %g is not a positive number", fn, (double)a->eps);
    if (a->tokens == 0)
        return BQ_OK;
    const int size = size_of(a->type);
    const int64_t nk = (int64_t)a->cache.heads * a->cache.dim, nq = (int64_t)a->q_heads * a->cache.dim;
    if (a->q_heads) {
        if ((rc = check_rows(fn, "q", a->q, a->ld_q, a->tokens, nq, size)) ||
            (rc = check_rows(fn, "q_out", a->q_out, a->ld_qo, a->tokens, nq, size_of(a->q_out_type))))
            return rc;
        if (a->q == a->q_out && (a->q_out_type != a->type || (a->tokens > 1 && a->ld_q != a->ld_qo)))
            return set_error(BQ_EARG, "%s: q_out in place of q needs its type and leading dimension", fn);
    } else if (a->q || a->q_out) {
        return set_error(BQ_EARG, "%s: q or q_out without q_heads", fn);
    }
    if ((rc = check_rows(fn, "k", a->k, a->ld_k, a->tokens, nk, size)) ||
        (rc = check_rows(fn, "v", a->v, a->ld_v, a->tokens, nk, size)))
        return rc;
    if (!a->pos || !a->slot || (a->rot && !a->freq))
        return set_error(BQ_EARG, "%s: null pos, slot or freq", fn);
    if (!aligned(a->pos, 4) || !aligned(a->slot, 8) || !aligned(a->freq, 4) || !aligned(a->q_norm, 4) ||
        !aligned(a->k_norm, 4))
        return set_error(BQ_EALIGN, "%s: pos, freq and norm weights must be 4-byte aligned, slot 8-byte", fn);
    return launched(fn, launch_append(*a, static_cast<hipStream_t>(s)));
}

BQ_EXPORT int bq_paged_attn_work_bytes(const bq_attn *a, int64_t *bytes)
{
    const char *fn = "bq_paged_attn_work_bytes";
    if (!bytes)
        return set_error(BQ_EARG, "%s: null bytes", fn);
    const int rc = check_attn(fn, a);
    if (rc)
        return rc;
    *bytes = a->tokens && a->requests ? attn_plan(*a).work_bytes : 0;
    return BQ_OK;
}

BQ_EXPORT int bq_paged_attn(const bq_attn *a, bq_stream s)
{
    const char *fn = "bq_paged_attn";
    int rc = check_attn(fn, a);
    if (!rc)
        rc = check_planes(fn, a->cache);
    if (rc)
        return rc;
    if (a->tokens == 0 || a->requests == 0)
        return BQ_OK;
    const int64_t n = (int64_t)a->q_heads * a->cache.dim;
    if ((rc = check_rows(fn, "q", a->q, a->ld_q, a->tokens, n, size_of(a->type))) ||
        (rc = check_rows(fn, "out", a->out, a->ld_out, a->tokens, n, size_of(a->type))))
        return rc;
    if (a->q == a->out)
        return set_error(BQ_EARG, "%s: out must not be q", fn);
    if (!a->cu || !a->lens || !a->table)
        return set_error(BQ_EARG, "%s: null cu, lens or table", fn);
    if (!aligned(a->cu, 4) || !aligned(a->lens, 4) || !aligned(a->table, 4))
        return set_error(BQ_EALIGN, "%s: cu, lens and table must be 4-byte aligned", fn);
    if (a->requests > 1 && (a->ld_table < a->table_cols || a->ld_table > kLdMax))
        return set_error(BQ_EARG, "%s: ld_table %lld below table_cols %d, or above 2^40", fn, (long long)a->ld_table,
                         (int)a->table_cols);
    if (!isfinite(a->scale))
        return set_error(BQ_EARG, "%s: scale is not finite", fn);
    const AttnPlan p = attn_plan(*a);
    if ((rc = check_work(fn, a->work, a->work_bytes, p.work_bytes)))
        return rc;
    return launched(fn, launch_attn(*a, p, static_cast<hipStream_t>(s)));
}

BQ_EXPORT int bq_adapters_work_bytes(const bq_adapters *a, int64_t *bytes)
{
    const char *fn = "bq_adapters_work_bytes";
    if (!bytes)
        return set_error(BQ_EARG, "%s: null bytes", fn);
    const int rc = check_adapters(fn, a);
    if (rc)
        return rc;
    *bytes = a->tokens && a->requests ? adapters_work(*a) : 0;
    return BQ_OK;
}

BQ_EXPORT int bq_adapters_add(const bq_adapters *a, bq_stream s)
{
    const char *fn = "bq_adapters_add";
    int rc = check_adapters(fn, a);
    if (rc)
        return rc;
    if (a->tokens == 0 || a->requests == 0)
        return BQ_OK;
    if (!a->a || !a->b || !a->gain)
        return set_error(BQ_EARG, "%s: null a, b or gain", fn);
    if (!aligned(a->a, 16) || !aligned(a->b, 16) || !aligned(a->gain, 4))
        return set_error(BQ_EALIGN, "%s: a and b must be 16-byte aligned, gain 4-byte", fn);
    if ((rc = check_rows(fn, "x", a->x, a->ld_x, a->tokens, a->n, size_of(a->x_type))))
        return rc;
    if (!a->cu || !a->ids || !a->y || !a->out)
        return set_error(BQ_EARG, "%s: null cu, ids, y or out", fn);
    if (a->tokens > 1 && (a->ld_y < a->rows || a->ld_out < a->rows || a->ld_y > kLdMax || a->ld_out > kLdMax))
        return set_error(BQ_EARG, "%s: leading dimensions of y or out below rows, or above 2^40", fn);
    if (a->y == a->out && a->tokens > 1 && a->ld_y != a->ld_out)
        return set_error(BQ_EARG, "%s: out in place of y needs its leading dimension", fn);
    if (!aligned(a->cu, 4) || !aligned(a->ids, 4) || !aligned(a->y, 4) || !aligned(a->out, 4))
        return set_error(BQ_EALIGN, "%s: cu, ids, y and out must be 4-byte aligned", fn);
    if ((rc = check_work(fn, a->work, a->work_bytes, adapters_work(*a))))
        return rc;
    return launched(fn, launch_adapters(*a, static_cast<hipStream_t>(s)));
}
