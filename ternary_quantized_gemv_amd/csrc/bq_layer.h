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
    int64_t row0;  // of a launch
    int32_t n, qa;
    int32_t f16_scale;
    double eps;
};
hipError_t launch_norm(int type, NormArgs a, int64_t rows, hipStream_t st);

hipError_t launch_append(const bq_append &a, hipStream_t st);

// How bq_paged_attn splits its work (attn_plan).  The kernel for few rows
// (few.cols of one key head's queries a tile, 0: not launched) cuts the keys of
// all requests into about few.items pieces per key head on the device, where
// the lengths are known (one piece a request with few.split 0); few.grid
// workgroups per key head walk them.  The kernel for many rows (many.cols a
// tile, workgroups for many.tiles of them per key head, 0: not launched) takes
// many.chunks pieces of many.chunk keys.  The joins add the pieces up.
//
// Scratch: for the pieces of split requests, cols rows of dim sums each, then
// their (maximum, sum of weights) pairs -- 2 few.items per key head: a request
// in c >= 2 pieces has more than c / 2 times the keys of one, and all requests
// have few.items times that -- and many.tiles * many.chunks; then notes of the
// kernels to the joins.
struct AttnPlan {
    struct {
        int cols;
        int grid;
        int items;
        int split;
    } few;
    struct {
        int cols;
        int tiles;
        int chunks;
        int chunk;
    } many;
    int64_t few_stats, many_sums, many_stats, notes;  // byte offsets in the scratch (few's sums at 0)
    int64_t work_bytes;
};
AttnPlan attn_plan(const bq_attn &a);
hipError_t launch_attn(const bq_attn &a, const AttnPlan &p, hipStream_t st);

int64_t adapters_work(const bq_adapters &a);
hipError_t launch_adapters(const bq_adapters &a, hipStream_t st);

}  // namespace bq
