// bq_rows.h -- internal to libbq: the rows of a request, from two neighbouring
// offsets that a device array holds.  Plain arithmetic for host and device.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define BQ_ANYWHERE __host__ __device__ __forceinline__
#else
#define BQ_ANYWHERE inline
#endif

namespace bq {

// Rows lo .. hi - 1 as far as they lie in [0, tokens), tokens < 2^31: a request
// that starts in front of the rows, or ends in front of its start, has none.
// Compared before they are subtracted: the offsets may hold anything.
struct Rows {
    int first, n;
};
BQ_ANYWHERE Rows rows_between(int lo, int hi, int64_t tokens)
{
    const int end = hi > tokens ? (int)tokens : hi;
    const bool any = lo >= 0 && lo < end;
    return Rows{any ? lo : 0, any ? end - lo : 0};
}

}  // namespace bq
