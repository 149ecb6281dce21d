// bq_check.h -- internal to libbq: argument checks that several entry points
// share (bq_api.cpp, bq_layer.cpp, bq_model.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/bq.h"
#include "bq_layout.h"

namespace bq {

constexpr int64_t kRowsMax = int64_t(1) << 31;
constexpr int64_t kLdMax = int64_t(1) << 40;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool known(int type) { return type == BQ_F32 || type == BQ_F16 || type == BQ_BF16; }
inline int size_of(int type) { return type == BQ_F32 ? 4 : 2; }

inline int launched(const char *fn, hipError_t e)
{
    return e == hipSuccess ? BQ_OK : set_error(BQ_EHIP, "%s: %s", fn, hipGetErrorString(e));
}

// A tensor of `rows` rows of `n` elements of `size` bytes, ld elements apart,
// each row 16-byte aligned.
inline int check_rows(const char *fn, const char *what, const void *p, int64_t ld, int64_t rows, int64_t n, int size)
{
    if (!p)
        return set_error(BQ_EARG, "%s: null %s", fn, what);
    if (rows > 1 && (ld < n || ld > kLdMax))
        return set_error(BQ_EARG, "%s: leading dimension %lld of %s below its row length %lld, or above 2^40", fn,
                         (long long)ld, what, (long long)n);
    if (!aligned(p, 16) || (rows > 1 && ld * size % 16))
        return set_error(BQ_EALIGN, "%s: %s rows must be 16-byte aligned", fn, what);
    return BQ_OK;
}

inline int check_tokens(const char *fn, int64_t tokens)
{
    if (tokens < 0 || tokens >= kRowsMax)
        return set_error(BQ_EARG, "%s: tokens %lld not in [0, 2^31)", fn, (long long)tokens);
    return BQ_OK;
}

inline int check_work(const char *fn, const void *work, int64_t have, int64_t need)
{
    if (need && !work)
        return set_error(BQ_EARG, "%s: null work", fn);
    if (have < need)
        return set_error(BQ_EARG, "%s: work holds %lld bytes, needs %lld", fn, (long long)have, (long long)need);
    if (need && !aligned(work, 16))
        return set_error(BQ_EALIGN, "%s: work must be 16-byte aligned", fn);
    return BQ_OK;
}

// A packed matrix of this format, and the activations of 1 to max_cols columns
// for a matrix of cols columns (bq_api.cpp).
int check_weights(const char *fn, const bq_weights *w, int fmt);
int check_act(const char *fn, const bq_act *a, int64_t cols, int max_cols);

}  // namespace bq
