// rotary.h -- internal interface of the rotary positions of Q and K in place.  Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "relayout.h"

namespace tfu {

constexpr uint32_t kRotaryPairs = 128;  // of a head of 256

// A [B, T, heads, D] view of P head groups, and where its rotated rows go: base addresses and byte strides.
struct RotaryTensor {
    const uint8_t* in[kMaxShards];
    uint8_t* out[kMaxShards];
    int64_t ib, it, ih, ob, ot, oh;
    uint32_t Hl;        // heads per group
    uint32_t in_place;  // what is not rotated stays where it is
};

struct RotaryParams {
    RotaryTensor x[2];         // q, k
    const int32_t* positions;  // [B][T] or null: first + t
    int32_t first;
    uint32_t B, T, D, R;
    uint32_t q_heads, heads;   // over all groups: of q, of both
    uint32_t chunk, chunks;    // heads a thread takes, and how many such sets there are
    uint32_t items;            // threads a row (kernel's units of work in one head row)
    float magnitude, sign;     // sign: -1 for the inverse
    uint64_t turn[kRotaryPairs];  // frequency as a 64-bit fraction of a turn a position
};

// width: elements of a vector (8, 4, 2, 1); below 8 with half-split pairs only
cudaError_t launch_rotary(const RotaryParams& p, bool bf16, bool half_split, uint32_t width, cudaStream_t stream);

}  // namespace tfu
