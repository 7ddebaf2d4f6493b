// attention_plan.h -- the document plan of the attention kernels.
#pragma once

#include "attention.h"

namespace tfu {

// Write the tile bits (TilePlan) of every row tile: rows are queries, or keys.
cudaError_t launch_plan(const AttentionParams& p, uint32_t* plan, bool rows_are_keys, uint32_t rows_per_tile,
                        cudaStream_t stream);

}  // namespace tfu
