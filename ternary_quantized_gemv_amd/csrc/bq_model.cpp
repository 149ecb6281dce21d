// bq_model.cpp -- the entry points of the operators around the layers
// (include/bq.h): argument checks, before anything is launched, and the launch.
#include <hip/hip_runtime_api.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "bq_check.h"
#include "bq_layout.h"
#include "bq_model.h"

using namespace bq;

namespace {

// a.ncols is an int32; some tiles of tokens below its end
constexpr int64_t kMatmulTokens = kRowsMax - (1 << 16);

bool known_act(int act) { return act == BQ_NONE || act == BQ_SILU || act == BQ_GELU || act == BQ_RELU2; }

// A matrix of `rows` rows of n elements with any alignment but its elements'.
int check_loose(const char *fn, const char *what, const void *p, int64_t ld, int64_t rows, int64_t n, int size)
{
    if (!p)
        return set_error(BQ_EARG, "%s: null %s", fn, what);
    if (rows > 1 && (ld < n || ld > kLdMax))
        return set_error(BQ_EARG, "%s: leading dimension %lld of %s below its row length %lld, or above 2^40", fn,
                         (long long)ld, what, (long long)n);
    if (!aligned(p, size))
        return set_error(BQ_EALIGN, "%s: %s must be %d-byte aligned", fn, what, size);
    return BQ_OK;
}

// The checks of bq_matmul that read no pointer, enough to size its scratch.
int check_product(const char *fn, const bq_product *a)
{
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    if (a->w.fmt != BQ_Q1_0 && a->w.fmt != BQ_Q2_0)
        return set_error(BQ_EARG, "%s: weights format %d unknown", fn, (int)a->w.fmt);
    if (!known(a->type))
        return set_error(BQ_EARG, "%s: type %d unknown", fn, (int)a->type);
    if (!known_act(a->act))
        return set_error(BQ_EARG, "%s: act %d unknown", fn, (int)a->act);
    if (a->a.ncols < 0 || a->a.ncols > kMatmulTokens)
        return set_error(BQ_EARG, "%s: %d activation columns: not in [0, 2^31 - 2^16]", fn, (int)a->a.ncols);
    if (a->a.qa != 32 && a->a.qa != 64 && a->a.qa != 128)
        return set_error(BQ_EARG, "%s: qa %d not in {32, 64, 128}", fn, (int)a->a.qa);
    if (a->w.rows < 1 || a->w.rows >= kMaxDim || a->w.cols < 1 || a->w.cols >= kMaxDim)
        return set_error(BQ_EARG, "%s: rows %lld / cols %lld out of range", fn, (long long)a->w.rows,
                         (long long)a->w.cols);
    if (a->w.cols % block_len(a->w.fmt) || a->w.cols % a->a.qa)
        return set_error(BQ_EARG, "%s: cols %lld not a multiple of %d and of qa %d", fn, (long long)a->w.cols,
                         block_len(a->w.fmt), (int)a->a.qa);
    if (!tile_fits(a->w.cols / block_len(a->w.fmt)))
        return set_error(BQ_EARG, "%s: cols %lld: a 64-row tile's payload would exceed %lld bytes", fn,
                         (long long)a->w.cols, (long long)kMaxTileBytes);
    return BQ_OK;
}

int check_draw(const char *fn, const bq_draw *a)
{
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    if (!known(a->type))
        return set_error(BQ_EARG, "%s: type %d unknown", fn, (int)a->type);
    if (a->reserved != 0)
        return set_error(BQ_EARG, "%s: reserved must be 0", fn);
    if (a->rows < 0 || a->rows >= kRowsMax)
        return set_error(BQ_EARG, "%s: rows %lld not in [0, 2^31)", fn, (long long)a->rows);
    if (a->vocab < 1 || a->vocab > BQ_VOCAB_MAX)
        return set_error(BQ_EARG, "%s: vocab %lld not in [1, %d]", fn, (long long)a->vocab, BQ_VOCAB_MAX);
    return BQ_OK;
}

}  // namespace

BQ_EXPORT int bq_embed(const bq_table *a, bq_stream s)
{
    const char *fn = "bq_embed";
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    if (!known(a->type))
        return set_error(BQ_EARG, "%s: type %d unknown", fn, (int)a->type);
    if (a->reserved != 0)
        return set_error(BQ_EARG, "%s: reserved must be 0", fn);
    if (!isfinite(a->scale))
        return set_error(BQ_EARG, "%s: scale is not finite", fn);
    int rc = check_tokens(fn, a->tokens);
    if (rc)
        return rc;
    const bool dense = a->w.fmt == 0;
    if (dense) {
        if (a->w.bits || a->w.scales || a->w.reserved)
            return set_error(BQ_EARG, "%s: a dense table (w.fmt 0) has no packed planes", fn);
        if (!known(a->dense_type))
            return set_error(BQ_EARG, "%s: dense_type %d unknown", fn, (int)a->dense_type);
        if (a->w.rows < 1 || a->w.rows >= kMaxDim || a->w.cols < 1 || a->w.cols >= kMaxDim)
            return set_error(BQ_EARG, "%s: rows %lld / cols %lld out of range", fn, (long long)a->w.rows,
                             (long long)a->w.cols);
        if (a->w.cols % 8)
            return set_error(BQ_EARG, "%s: cols %lld not a multiple of 8", fn, (long long)a->w.cols);
        if ((rc = check_rows(fn, "dense", a->dense, a->ld_dense, a->w.rows, a->w.cols, size_of(a->dense_type))))
            return rc;
    } else {
        if (a->w.fmt != BQ_Q1_0 && a->w.fmt != BQ_Q2_0)
            return set_error(BQ_EARG, "%s: table format %d unknown", fn, (int)a->w.fmt);
        if (a->dense || a->dense_type || a->ld_dense)
            return set_error(BQ_EARG, "%s: a packed table with dense rows", fn);
        if ((rc = check_weights(fn, &a->w, a->w.fmt)))
            return rc;
    }
    if (a->tokens == 0)
        return BQ_OK;
    if (!a->ids)
        return set_error(BQ_EARG, "%s: null ids", fn);
    if (!aligned(a->ids, 8))
        return set_error(BQ_EALIGN, "%s: ids must be 8-byte aligned", fn);
    if ((rc = check_rows(fn, "out", a->out, a->ld_out, a->tokens, a->w.cols, size_of(a->type))))
        return rc;
    return launched(fn, launch_embed(*a, static_cast<hipStream_t>(s)));
}

BQ_EXPORT int bq_gated_q8(const bq_gated *a, bq_stream s)
{
    const char *fn = "bq_gated_q8";
    if (!a)
        return set_error(BQ_EARG, "%s: null arguments", fn);
    if (!known(a->type))
        return set_error(BQ_EARG, "%s: type %d unknown", fn, (int)a->type);
    if (!known_act(a->act))
        return set_error(BQ_EARG, "%s: act %d unknown", fn, (int)a->act);
    if (a->qa != 32 && a->qa != 64 && a->qa != 128)
        return set_error(BQ_EARG, "%s: qa %d not in {32, 64, 128}", fn, (int)a->qa);
    if (a->f16_scale != 0 && a->f16_scale != 1)
        return set_error(BQ_EARG, "%s: f16_scale %d is not 0 or 1", fn, (int)a->f16_scale);
    int rc = check_tokens(fn, a->tokens);
    if (rc)
        return rc;
    if (a->n < 1 || a->n >= kRowsMax || a->n % a->qa)
        return set_error(BQ_EARG, "%s: n %lld is not a multiple of qa %d in [1, 2^31)", fn, (long long)a->n, (int)a->qa);
    if (a->tokens == 0)
        return BQ_OK;
    const int size = size_of(a->type);
    if ((rc = check_rows(fn, "gate", a->gate, a->ld_gate, a->tokens, a->n, size)) ||
        (rc = check_rows(fn, "up", a->up, a->ld_up, a->tokens, a->n, size)) ||
        (a->y && (rc = check_rows(fn, "y", a->y, a->ld_y, a->tokens, a->n, size))))
        return rc;
    if (a->y && a->tokens > 1 && ((a->y == a->gate && a->ld_y != a->ld_gate) || (a->y == a->up && a->ld_y != a->ld_up)))
        return set_error(BQ_EARG, "%s: y in place of gate or up needs its leading dimension", fn);
    if (!a->q || !a->d)
        return set_error(BQ_EARG, "%s: null q or d", fn);
    if (a->tokens > 1 && (a->ld_q < a->n || a->ld_q > kLdMax || a->ld_d < a->n / a->qa || a->ld_d > kLdMax))
        return set_error(BQ_EARG, "%s: leading dimensions of q or d too small, or above 2^40", fn);
    if (!aligned(a->q, 8) || !aligned(a->d, 4) || (a->tokens > 1 && a->ld_q % 16))
        return set_error(BQ_EALIGN, "%s: q must be 8-byte aligned (ld_q a multiple of 16), d 4-byte aligned", fn);
    return launched(fn, launch_gated(*a, static_cast<hipStream_t>(s)));
}

BQ_EXPORT int bq_matmul_work_bytes(const bq_product *a, int64_t *bytes)
{
    const char *fn = "bq_matmul_work_bytes";
    if (!bytes)
        return set_error(BQ_EARG, "%s: null bytes", fn);
    const int rc = check_product(fn, a);
    if (rc)
        return rc;
    *bytes = a->a.ncols ? matmul_work(*a) : 0;
    return BQ_OK;
}

BQ_EXPORT int bq_matmul(const bq_product *a, bq_stream s)
{
    const char *fn = "bq_matmul";
    int rc = check_product(fn, a);
    if (!rc)
        rc = check_weights(fn, &a->w, a->w.fmt);
    if (rc)
        return rc;
    const int64_t tokens = a->a.ncols, rows = a->w.rows;
    if (tokens == 0)
        return BQ_OK;
    if ((rc = check_act(fn, &a->a, a->w.cols, INT_MAX)))
        return rc;
    if (tokens > 1 && (a->a.ld_q > kLdMax || a->a.ld_d > kLdMax))
        return set_error(BQ_EARG, "%s: leading dimensions of the activations above 2^40", fn);
    const int size = size_of(a->type);
    if ((rc = check_loose(fn, "y", a->y, a->ld_y, tokens, rows, size)) ||
        (a->mul && (rc = check_loose(fn, "mul", a->mul, a->ld_mul, tokens, rows, size))) ||
        (a->res && (rc = check_loose(fn, "res", a->res, a->ld_res, tokens, rows, size))) ||
        (a->bias && (rc = check_loose(fn, "bias", a->bias, rows, 1, rows, 4))))
        return rc;
    if (tokens > 1 && ((a->y == a->mul && a->ld_y != a->ld_mul) || (a->y == a->res && a->ld_y != a->ld_res)))
        return set_error(BQ_EARG, "%s: y in place of mul or res needs its leading dimension", fn);
    if ((rc = check_work(fn, a->work, a->work_bytes, matmul_work(*a))))
        return rc;
    return launched(fn, launch_matmul(*a, static_cast<hipStream_t>(s)));
}

BQ_EXPORT int bq_sample_work_bytes(const bq_draw *a, int64_t *bytes)
{
    const char *fn = "bq_sample_work_bytes";
    if (!bytes)
        return set_error(BQ_EARG, "%s: null bytes", fn);
    const int rc = check_draw(fn, a);
    if (rc)
        return rc;
    *bytes = a->rows ? sample_work(*a) : 0;
    return BQ_OK;
}

BQ_EXPORT int bq_sample(const bq_draw *a, bq_stream s)
{
    const char *fn = "bq_sample";
    int rc = check_draw(fn, a);
    if (rc)
        return rc;
    if (a->rows == 0)
        return BQ_OK;
    if ((rc = check_loose(fn, "logits", a->logits, a->ld_logits, a->rows, a->vocab, size_of(a->type))))
        return rc;
    if (!a->u || !a->token)
        return set_error(BQ_EARG, "%s: null u or token", fn);
    if (!aligned(a->u, 4) || !aligned(a->temperature, 4) || !aligned(a->top_k, 4) || !aligned(a->top_p, 4) ||
        !aligned(a->min_p, 4) || !aligned(a->token, 8) || !aligned(a->logprob, 4))
        return set_error(BQ_EALIGN, "%s: token must be 8-byte aligned, the other arrays 4-byte", fn);
    if ((rc = check_work(fn, a->work, a->work_bytes, sample_work(*a))))
        return rc;
    return launched(fn, launch_sample(*a, static_cast<hipStream_t>(s)));
}
