// bq_model.h -- internal to libbq: launchers of the operators around the
// layers.  The entry points in bq_model.cpp check every argument first; the
// launchers validate nothing and return hipGetLastError().
#pragma once

#include "../../include/bq.h"
#include "bq_types.h"

namespace bq {

hipError_t launch_embed(const bq_table &a, hipStream_t st);
hipError_t launch_gated(const bq_gated &a, hipStream_t st);

int64_t matmul_work(const bq_product &a);
hipError_t launch_matmul(const bq_product &a, hipStream_t st);

int64_t sample_work(const bq_draw &a);
hipError_t launch_sample(const bq_draw &a, hipStream_t st);

}  // namespace bq
