// kv_plan.h -- internal interface of the cache's plan.  Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace tfu {

// Pages, starts, positions and slots of a step's requests.
struct KvPlanParams {
    const int32_t *lens, *new_tokens, *free_span;
    int32_t *table, *free_pages, *lens_out, *starts, *positions, *slots, *span_out;
    int64_t table_stride;
    uint32_t N, max_pages, page, page_bits, num_pages, T;  // page: 2^page_bits
};
constexpr int kMostRequests = 8192;  // three sums and a length of each in shared memory: 128 KiB

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t stream);

// Status word: 0, or 1 when a length, the span, what was given back or a new row's page was out of range.
cudaError_t read_kv_plan_status(unsigned* out, bool clear);

}  // namespace tfu
