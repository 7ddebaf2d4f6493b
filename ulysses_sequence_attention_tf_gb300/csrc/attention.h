// attention.h -- internal interface of the attention over the head groups and of
// its gradient.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "relayout.h"

namespace tfu {

// A [B, tokens, heads, D] view of every head group: base addresses and byte strides.
struct GroupView {
    uint8_t* base[kMaxShards];
    int64_t b, t, h;
};

struct AttentionParams {
    GroupView q, k, v, out;
    GroupView dout, dq, dk, dv;  // backward only
    float* lse[kMaxShards];      // [B][Hl][Sq] per group, or null
    float* delta;                // backward: workspace [P][B][Hl][Sq], sum_d dO * O of each row
    const float* slopes;         // [P * Hl] or null
    const int32_t* prefix;       // [B] or null
    const int32_t* q_docs;       // [B][Sq] or null
    const int32_t* k_docs;       // [B][Sk]
    float scale, cap;            // cap 0: scores are not capped
    uint32_t P, B, Sq, Sk;
    uint32_t Hl, Hkl, shared;    // query and key heads per group, query heads per key head
    uint32_t D;
    uint32_t causal;
};

cudaError_t launch_attention(const AttentionParams& p, bool bf16, cudaStream_t stream);
// *launches: kernels launched
cudaError_t launch_attention_backward(const AttentionParams& p, bool bf16, cudaStream_t stream, int* launches);

}  // namespace tfu
