// linear.h -- internal interface of linear attention with a decay for each head.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "attention.h"
#include "relayout.h"

namespace tfu {

// One recurrence over the tokens of every sequence and head, in rising order or (reverse) in falling, with lambda =
// e^-decay[head]:
//   S <- lambda S + kv_scale k^T v,  out = out_scale q S
//   reverse:  S <- S + kv_scale k^T v,  out = out_scale q S,  S <- lambda S
// The forward pass and each gradient is one, with q, k and v standing for the tensors in brackets:
//   out: (q, k, v), kv_scale 1, out_scale scale            dq: (dout, v, k) on the transposed state, likewise
//   dk: (v, dout, q) reverse, kv_scale scale, out_scale 1, transposed     dv: (k, q, dout) reverse, likewise
// In reverse the state starts as the gradient of the final state and ends as that of the state in front.
struct LinearPass {
    GroupView q, k, v, out;    // [B, S, Hl, D] of each head group (rows: B = 1)
    const float* state;        // where S starts: [N or slots][H][D][D], or null: 0
    float* final_state;        // where it ends, or null.  May be this pass's `state`
    const float* decay;        // [H]
    const int32_t* starts;     // rows: [N + 1], first row of each sequence; null: N batch rows of S tokens
    const int32_t* slots;      // rows: [N], states of the sequences
    uint32_t num_slots;
    uint32_t P, N, S, Hl, D;   // S: tokens of a batch row, or rows of the row tensors
    uint32_t most;             // bound of the tokens of one sequence
    uint32_t reverse, transposed;  // transposed: S lies as its transpose in state (such a pass has no final_state)
    float kv_scale, out_scale;
};

struct LinearSequence {
    int64_t first;   // row
    uint32_t b, len;
    uint32_t slot;
    bool ok;
};

#ifdef __CUDACC__
// S -> e^-x S + y.  For small x as S + (e^-x - 1) S with the bracket from expm1f, so that thousands of steps near 1 do not
// add up the rounding of e^-x; above 1/2 as a product, whose rounding follows what is kept of S and not S itself.
struct Fade {
    float factor, whole;
    __device__ __forceinline__ explicit Fade(float x) : factor(x < 0.5f ? expm1f(-x) : expf(-x)), whole(x < 0.5f ? 1.f : 0.f) {}
    __device__ __forceinline__ float of(float s, float y) const { return fmaf(whole, s, fmaf(s, factor, y)); }
};

__device__ __forceinline__ LinearSequence linear_sequence(const LinearPass& p, uint32_t n, unsigned* status) {
    if (!p.starts) return {0, n, p.S, n, true};
    const int64_t from = p.starts[n], to = p.starts[n + 1], slot = p.slots[n];
    const bool ok = from >= 0 && from <= to && to <= int64_t(p.S) && to - from <= int64_t(p.most) && slot >= 0 && slot < int64_t(p.num_slots);
    if (!ok) {
        if (threadIdx.x == 0) atomicOr(status, 1u);
        return {0, 0, 0, 0, false};
    }
    return {from, 0, uint32_t(to - from), uint32_t(slot), to > from};
}
#endif

constexpr uint32_t kLinearChunk = 128;  // tokens: TMEM lanes

// The chunk kernels' launches: one pass forward, or the three of the gradients over the same batch rows at once;
// every sequence cut into `segments` of seg_chunks chunks (1: not cut).
constexpr uint32_t kLinearPasses = 3;
struct LinearChunkParams {
    GroupMaps maps[4];                    // of the tensors, boxes of 128 tokens
    LinearPass pass[kLinearPasses];
    uint32_t tensor[kLinearPasses][3];    // a pass's q, k, v among the maps
    uint32_t wide_out[kLinearPasses];     // rows of out are 32-byte aligned
    uint32_t passes, segments, seg_chunks;
    float* parts;                         // workspace [passes][N * H][segments][D][D], used where there are several segments
};
cudaError_t launch_linear_chunks(const LinearChunkParams& p, bool bf16, cudaStream_t stream, int* launches);

// token by token: single ones and short runs
cudaError_t launch_linear_steps(const LinearPass& p, bool bf16, cudaStream_t stream);

// Status words: 0, or 1 when a sequence's slot or starts were out of range and it was left out.
cudaError_t read_linear_steps_status(unsigned* out, bool clear);
cudaError_t read_linear_chunks_status(unsigned* out, unsigned* waits, bool clear);  // *waits: 1 when a bounded wait gave up

}  // namespace tfu
