// attention.h -- internal interface of the attention over the head groups and of
// its gradient.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "relayout.h"

namespace tfu {

constexpr uint32_t kAttnRows = 128;   // rows of a tile: TMEM lanes
constexpr uint32_t kAttnPair = 256;   // query rows of a forward CTA: two tiles

// A [B, tokens, heads, D] view of every head group: base addresses and byte strides.
struct GroupView {
    uint8_t* base[kMaxShards];
    int64_t b, t, h;
};

struct AttentionParams {
    GroupView q, k, v, out;
    GroupView dout, dq, dk, dv;  // backward only
    float* lse[kMaxShards];      // [B][Hl][Sq] per group, or null
    float* delta;                // backward: workspace [P][B][Hl][Sq], sum_j P dP of each row
    uint32_t* plan;              // with documents: the visible tiles (TilePlan)
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

// Tensor maps of the head groups' views: 4-D (D, heads, tokens, B), boxes of 64
// elements x 128 or 64 tokens of one head with the 128-byte swizzle.
struct GroupMaps {
    CUtensorMap m[kMaxShards];
};

// CTAs run one an SM, in rounds.  The units (row tiles of a head) of the last, partly
// filled round are cut into `parts` along the other side; a part leaves fp32 sums at
// part[slot], slot = its CTA's number behind the whole units, and a second kernel joins
// them in order.  Without documents and causal mask only: the units cost the same then.
struct Split {
    uint32_t whole, parts;  // units that are not cut, parts of each other one (1: none is cut)
    float* part;            // forward: O rows; dQ rows, then W rows; dK rows, then dV rows
    float2* stat;           // forward: a row's reference (log2) and sum; dQ: what delta lacks (x)
};
constexpr uint32_t kAttnSms = 152;   // SMs of a GB300
constexpr uint32_t kLeastPart = 8;   // tiles of the other side in a part: below, the join costs more than it gives
inline Split plan_split(const uint64_t units, const uint32_t tiles, bool even) {
    Split s{uint32_t(units), 1, nullptr, nullptr};
    const uint32_t rest = uint32_t(units % kAttnSms);
    if (!even || rest == 0) return s;
    uint32_t parts = kAttnSms / rest;
    if (parts > tiles / kLeastPart) parts = tiles / kLeastPart;
    if (parts < 2) return s;
    s.whole = uint32_t(units - rest);
    s.parts = parts;
    return s;
}

// Heads whose tiles the units interleave: one, but with the causal mask as many as have their other
// side (two tensors of `tokens` rows) in half of the L2 together.
inline uint32_t head_block(bool causal, uint64_t heads, uint64_t tokens, uint32_t D) {
    const uint64_t bytes = 4 * tokens * D, fit = bytes ? (uint64_t(64) << 20) / bytes : heads;
    return !causal || fit < 1 ? 1 : uint32_t(fit < heads ? fit : heads);
}

// Forward pass with documents: whether units go by their work, the longest first (in the gradients' kernels the
// few registers of it cost more than it gave: training without documents 2.10 -> 2.16 ms).  Only where a CTA finds its place among
// `entries` row tiles in about a microsecond, and where the other side of all heads stays in half of the L2.
inline bool rank_units(uint64_t entries, uint32_t words, uint64_t heads, uint64_t tokens, uint32_t D) {
    return entries <= 256 && entries * words <= 1024 && 4 * heads * tokens * D <= uint64_t(64) << 20;
}

struct ForwardParams {
    GroupMaps q, k, v;
    AttentionParams a;
    uint32_t q_tiles;     // of kAttnPair rows
    uint32_t head_block;  // heads that units interleave (head_block())
    bool ranked;          // units in the order of the plan's work (rank_units())
    Split split;
};

struct BackwardParams {
    GroupMaps q, k, v, dout;      // boxes of 128 tokens
    GroupMaps q_half, dout_half;  // boxes of 64
    AttentionParams a;
    uint32_t* key_plan;           // with documents: row tiles of keys (a.plan: of 128 queries)
    float* sizes;                 // fp16: largest |dO|^2 by head and q_tile, then |V|^2 by key head and k_tile
    uint32_t q_tiles, k_tiles;    // of kAttnRows rows
    uint32_t head_block, key_head_block;
    Split dq_split, dkv_split;
};

// With documents, a kernel in front of the attention writes for every row tile
// of a batch row one bit per tile of the other side, twice: [0] some pair may be
// visible, [1] every pair is.
struct TilePlan {
    uint32_t row_tiles, words;  // words of one bit set
    __host__ __device__ size_t bytes(uint32_t B) const { return size_t(B) * row_tiles * words * 2 * sizeof(uint32_t); }
};
inline TilePlan tile_plan(uint32_t rows, uint32_t rows_per_tile, uint32_t cols) {
    const uint32_t col_tiles = (cols + kAttnRows - 1) / kAttnRows;
    return {(rows + rows_per_tile - 1) / rows_per_tile, (col_tiles + 31) / 32};
}

// Encode the maps of P groups ([B, tokens, heads, D] 16-bit views, boxes of box_tokens);
// false if the driver refuses.
bool encode_group_maps(GroupMaps* maps, const GroupView& v, uint32_t P, uint32_t B, uint32_t tokens, uint32_t heads,
                       uint32_t D, uint32_t box_tokens, bool bf16);

// Join the parts of cut units: rows of kAttnPair (forward) or kAttnRows a unit.
cudaError_t launch_join_forward(const ForwardParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_join_dq(const BackwardParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_join_gradient(const AttentionParams& p, const Split& s, const GroupView& out, const float* part, float factor,
                                 uint32_t row_tiles, uint32_t rows, uint32_t heads, bool bf16, cudaStream_t stream);

// *launches: kernels launched
cudaError_t launch_attention(const ForwardParams& p, bool bf16, cudaStream_t stream, int* launches);
cudaError_t launch_attention_backward(const BackwardParams& p, bool bf16, cudaStream_t stream, int* launches);

// Status words of the attention kernels: 0, or 1 when a bounded wait gave up.
cudaError_t read_attention_status(unsigned* out, bool clear);
cudaError_t read_attention_backward_status(unsigned* out, bool clear);

}  // namespace tfu
