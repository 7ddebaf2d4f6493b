// attention_common.cuh -- the scores and the mask of the attention kernels.
//
//   x_ij = scale * q_i . k_j
//   y_ij = cap * tanh(x_ij / cap)              (x_ij where cap == 0)
//   z_ij = y_ij - slope_h * |pos_i - j|        pos_i = i + Sk - Sq
//   key j is visible to query i iff  j < bound_i  and the documents agree:
//     bound_i = Sk, or with a causal mask min(Sk, max(pos_i + 1, prefix_b, 0));
//     q_docs_i == k_docs_j >= 0 where there are documents.
// Masked scores are left out by selection, never by adding a large number.
// Exponentials are base 2 (ex2.approx, 2 units in the last place): z is kept times log2 e.
#pragma once

#include "attention.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace tfu {
namespace dev {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// tanh by 1 - 2 / (e^(2x) + 1): within 2^-22 of tanh x for every x.
__device__ __forceinline__ float tanh_wide(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(x * (2.0f * kLog2e)) + 1.0f));
    return fmaf(-2.0f, r, 1.0f);
}

// tanh x / x for |x| <= kTanhNear as a polynomial in y = x^2, fitted for the least
// relative error (7.3e-8): no transcendental instruction.
constexpr float kTanhNear = 0.6f;
__device__ __forceinline__ uint64_t tanh_over_x(uint64_t y) {
    auto both = [](float c) { return f2_pack(c, c); };
    uint64_t r = f2_fma(y, both(0.015475417487323284f), both(-0.05210147425532341f));
    r = f2_fma(y, r, both(0.13310173153877258f));
    r = f2_fma(y, r, both(-0.33332309126853943f));
    return f2_fma(y, r, both(0.9999999403953552f));
}

// The tiles of the other side that a row tile visits, in order: all of [0, n), or
// those with a bit in `words`.
struct TileIter {
    const uint32_t* words;
    int n, pos;
    uint32_t bits;
    __device__ TileIter(const uint32_t* w, int count) : words(w), n(count), pos(w ? -32 : 0), bits(0) {}
    __device__ __forceinline__ int next() {
        if (!words) return pos < n ? pos++ : -1;
        while (bits == 0) {
            pos += 32;
            if (pos >= n) return -1;
            bits = __ldg(words + (pos >> 5));
        }
        const int b = __ffs(bits) - 1;
        bits &= bits - 1;
        return pos + b;
    }
};

// Registers written by tcgen05.ld may be read after this (the wait, and what the
// compiler may not move above it).
__device__ __forceinline__ void tc_landed(uint32_t (&r)[32]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]));
    asm volatile("" : "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

}  // namespace dev
}  // namespace tfu
