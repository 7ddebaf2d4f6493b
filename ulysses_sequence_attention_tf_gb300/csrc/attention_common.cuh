// attention_common.cuh -- the scores and the mask of the attention kernels.
//
//   x_ij = scale * q_i . k_j
//   y_ij = cap * tanh(x_ij / cap)              (x_ij where cap == 0)
//   z_ij = y_ij - slope_h * |pos_i - j|        pos_i = i + Sk - Sq
//   key j is visible to query i iff  j < bound_i  and the documents agree:
//     bound_i = Sk, or with a causal mask min(Sk, max(pos_i + 1, prefix_b, 0));
//     q_docs_i == k_docs_j >= 0 where there are documents.
// Masked scores are left out by selection, never by adding a large number.
#pragma once

#include "attention.h"
#include "device_common.cuh"

namespace tfu {
namespace dev {

// keys [0, bound) are inside the causal or prefix mask of query i of batch row b
__device__ __forceinline__ int key_bound(const AttentionParams& p, uint32_t b, int64_t i) {
    if (!p.causal) return int(p.Sk);
    int64_t n = i + 1 + int64_t(p.Sk) - int64_t(p.Sq);
    if (p.prefix) {
        const int64_t pre = p.prefix[b];
        n = pre > n ? pre : n;
    }
    n = n < 0 ? 0 : n;
    return int(n < int64_t(p.Sk) ? n : int64_t(p.Sk));
}

template <Fused kF>
__device__ __forceinline__ float to_float(uint16_t v) {
    float lo, hi;
    unpack2<kF>(uint32_t(v), lo, hi);
    return lo;
}
template <Fused kF>
__device__ __forceinline__ uint16_t to_half(float v) {
    return uint16_t(pack2<kF>(v, 0.f) & 0xffffu);
}

}  // namespace dev
}  // namespace tfu
