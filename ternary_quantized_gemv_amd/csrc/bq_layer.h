// bq_layer.h -- internal to libbq: argument blocks and launchers of the
// operators between the products.  The entry points in bq_layer.cpp check
// every argument first; the launchers validate nothing and return
// hipGetLastError().
#pragma once

#include "../../include/bq.h"
#include "bq_types.h"

namespace bq {

struct NormArgs {
    const void *x, *res, *w;
    void *h, *y;
    int8_t *q;
    float *d;
    int64_t ld_x, ld_res, ld_h, ld_y, ld_q, ld_d;
    int32_t n, qa;
    int32_t f16_scale;
    double eps;
};
hipError_t launch_norm(int type, const NormArgs &a, int64_t rows, hipStream_t st);

hipError_t launch_append(const bq_append &a, hipStream_t st);

// How bq_paged_attn splits its work (attn_plan), for each of its two kernels:
// tiles of `cols` rows of one key head's queries, `tiles` of them at most per
// request (0: not launched), each over `chunks` pieces of `chunk` keys that the
// join adds up.
struct AttnSplit {
    int cols;
    int tiles;
    int chunks;
    int chunk;
};
struct AttnPlan {
    AttnSplit few, many;
    int stride;  // places per row for the pieces
    int64_t work_bytes;
};
AttnPlan attn_plan(const bq_attn &a);
hipError_t launch_attn(const bq_attn &a, const AttnPlan &p, hipStream_t st);

int64_t adapters_work(const bq_adapters &a);
hipError_t launch_adapters(const bq_adapters &a, hipStream_t st);

}  // namespace bq
