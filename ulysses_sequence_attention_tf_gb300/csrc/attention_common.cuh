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

// tanh x / x for |x| <= kTanhNear as a polynomial in y = x^2 without a transcendental instruction, fitted
// to it for a small relative error: 9.1e-8 with the coefficients as stored, evaluated in 64 bits.
constexpr float kTanhNear = 0.6f;
constexpr float kTanh0 = 0.9999999403953552f, kTanh1 = -0.33332309126853943f, kTanh2 = 0.13310173153877258f,
                kTanh3 = -0.05210147425532341f, kTanh4 = 0.015475417487323284f;
__device__ __forceinline__ uint64_t tanh_over_x(uint64_t y) {
    auto both = [](float c) { return f2_pack(c, c); };
    uint64_t r = f2_fma(y, both(kTanh4), both(kTanh3));
    r = f2_fma(y, r, both(kTanh2));
    r = f2_fma(y, r, both(kTanh1));
    return f2_fma(y, r, both(kTanh0));
}

// The unit of a CTA, and which part of how many it takes.
struct Unit {
    uint32_t u, part, parts, slot;
    __device__ Unit(const Split& s, uint32_t cta) : u(cta), part(0), parts(1), slot(0) {
        if (cta >= s.whole) {
            slot = cta - s.whole;
            u = s.whole + slot / s.parts;
            part = slot % s.parts;
            parts = s.parts;
        }
    }
    __device__ int begin(int n) const { return int(int64_t(n) * part / parts); }
    __device__ int end(int n) const { return int(int64_t(n) * (part + 1) / parts); }
};

// Row tile and head of unit u: tile by tile over `block` heads, then the next heads.  causal: unequal
// tiles, the longest first over many heads, so that the last units to start are short.
struct TileHead {
    uint32_t tile, head;
    __device__ TileHead(uint32_t u, uint32_t tiles, uint32_t heads, uint32_t block) {
        const uint32_t first = u / (tiles * block) * block, in = u % (tiles * block), here = min(block, heads - first);
        tile = in / here;
        head = first + in % here;
    }
};

// Documents make row tiles unequal in no known order: the row tile (of all batch rows' `entries`) that
// visits the rank-th most tiles, found by every CTA for itself from the plan.  For all threads;
// scratch: 1 + entries words of shared memory, free for bulk copies afterwards.
__device__ __forceinline__ uint32_t ranked_entry(const uint32_t* plan, uint32_t entries, uint32_t words, uint32_t rank, uint32_t* scratch) {
    for (uint32_t e = threadIdx.x; e < entries; e += blockDim.x) {
        uint32_t visits = 0;
        for (uint32_t w = 0; w < words; ++w) visits += __popc(__ldg(plan + size_t(e) * 2 * words + w));
        scratch[1 + e] = visits;
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < entries; e += blockDim.x) {
        const uint32_t own = scratch[1 + e];
        uint32_t before = 0;
        for (uint32_t f = 0; f < entries; ++f) before += scratch[1 + f] > own || (scratch[1 + f] == own && f < e);
        if (before == rank) scratch[0] = e;
    }
    __syncthreads();
    const uint32_t found = scratch[0];
    fence_async_shared();
    __syncthreads();
    return found;
}

// The tiles of the other side that a row tile visits, in order: all of [from, n), or
// those with a bit in `words`.
struct TileIter {
    const uint32_t* words;
    int n, pos;
    uint32_t bits;
    __device__ TileIter(const uint32_t* w, int count, int from = 0) : words(w), n(count), pos(w ? -32 : from), bits(0) {}
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

// kN columns of this thread's TMEM lane from taddr, as floats
template <int kN>
__device__ __forceinline__ void load_row(uint32_t taddr, float (&v)[kN]) {
    uint32_t r[kN / 32][32];
#pragma unroll
    for (int x = 0; x < kN / 32; ++x) tc_ld32(taddr + x * 32, r[x]);
    tc_wait_ld();
#pragma unroll
    for (int x = 0; x < kN / 32; ++x) {
        tc_landed(r[x]);
#pragma unroll
        for (int y = 0; y < 32; ++y) v[x * 32 + y] = __uint_as_float(r[x][y]);
    }
}

// Scores beyond scale * q.k: none, the cap, or cap (if any) and bias and any scale.
enum class Score { kPlain, kCap, kAny };

// The bias of a tile is linear in the key where all of its keys lie on one side of the query:
// side = 1 (keys at or before it), -1 (behind it), 0 (both).  rows, keys: first ones of the
// tile; under a plain causal mask what lies behind a query does not count.
__device__ __forceinline__ int bias_side(int row_pos0, int rows, int key0, int keys, bool causal_only) {
    return row_pos0 >= key0 + keys - 1 || causal_only ? 1 : row_pos0 + rows - 1 <= key0 ? -1 : 0;
}

// z of one row's 128 scores, times log2 e, in place (kCap, kAny).  far: the query's position
// less the tile's first key.
template <Score kScore>
__device__ __forceinline__ void finish_scores(float (&s)[128], float scale, float cap, float slope, float far, int side) {
    auto both = [](float v) { return f2_pack(v, v); };
    const float k = slope * kLog2e;
    if (kScore == Score::kCap || cap != 0.f) {
        const float to_x = scale / cap, to_z = cap * kLog2e;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 128; i += 2) most = fmaxf(fmaxf(fabsf(s[i]), fabsf(s[i + 1])), most);
        if (__all_sync(0xffffffffu, most * fabsf(to_x) <= kTanhNear)) {
            const uint64_t x2 = both(to_x), z2 = both(to_z);
#pragma unroll
            for (int i = 0; i < 128; i += 2) {
                const uint64_t x = f2_mul(f2_pack(s[i], s[i + 1]), x2);
                f2_unpack(f2_mul(f2_mul(x, z2), tanh_over_x(f2_mul(x, x))), s[i], s[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) s[i] = to_z * tanh_wide(s[i] * to_x);
        }
        if (kScore == Score::kCap) return;
        scale = kLn2;  // s is z already
    }
    const float c = scale * kLog2e;
    if (side != 0) {  // z = c s - side k (far - i)
        const float at = side > 0 ? -k * far : k * far, by = side > 0 ? k : -k;
        const uint64_t c2 = both(c);
#pragma unroll
        for (int i = 0; i < 128; i += 2)
            f2_unpack(f2_fma(f2_pack(s[i], s[i + 1]), c2, f2_pack(fmaf(float(i), by, at), fmaf(float(i + 1), by, at))), s[i], s[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = fmaf(-k, fabsf(far - float(i)), s[i] * c);
    }
}

// Bit x: key x of a block of 32 that starts at key0 lies below the row's bound.
__device__ __forceinline__ uint32_t bound_bits(int bound, int key0) {
    const int n = bound - key0;
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// bits[g] &= keys of block g (its lane's document kd[g]) that belong to the row's document: one
// ballot a block for every document among the warp's rows, one or two as a rule.
template <int kBlocks>
__device__ __forceinline__ void keep_document(uint32_t (&bits)[kBlocks], const int32_t (&kd)[kBlocks], int32_t doc) {
    uint32_t mine[kBlocks] = {};
    for (uint32_t left = 0xffffffffu; left;) {
        const int32_t d = __shfl_sync(0xffffffffu, doc, __ffs(left) - 1);
        const bool here = doc == d;
#pragma unroll
        for (int g = 0; g < kBlocks; ++g) {
            const uint32_t same = __ballot_sync(0xffffffffu, kd[g] == d);
            if (here) mine[g] = same;
        }
        left &= ~__ballot_sync(0xffffffffu, here);
    }
#pragma unroll
    for (int g = 0; g < kBlocks; ++g) bits[g] &= mine[g];
}

constexpr float kSlack = 8.0f;  // growth of a row's maximum that its reference lets pass, in powers of two

// One arrival of a warp whose lanes are done with what they wrote to TMEM and shared memory.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    tc_fence_before();
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void bounds_of(const float (&s)[128], float& top, float& low, bool with_low) {
    float t[4], u[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        t[x] = u[x] = s[x];
#pragma unroll
        for (int y = x + 4; y < 128; y += 4) {
            t[x] = fmaxf(t[x], s[y]);
            if (with_low) u[x] = fminf(u[x], s[y]);
        }
    }
    top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    low = fminf(fminf(u[0], u[1]), fminf(u[2], u[3]));
}

// The row's reference m follows the tile's maximum z when that outgrows it (or V's scale
// changed: down); l and the kD output columns, which hold something when `started`, go along.
template <int kD>
__device__ __forceinline__ void move_reference(float most, float down, bool started, float& m, float& l, uint32_t o_row) {
    const bool grow = most > m + kSlack;  // from -inf: on any visible key
    if (!__any_sync(0xffffffffu, grow || down != 1.0f)) return;
    const float to = grow ? most : m;
    const float shrink = grow ? ex2(m - to) : 1.0f;
    l *= shrink;
    m = to;
    if (!started) return;
    const float f = shrink * down;
#pragma unroll 1
    for (int x = 0; x < kD; x += 32) {
        uint32_t r[32];
        tc_ld32(o_row + x, r);
        tc_wait_ld();
        tc_landed(r);
#pragma unroll
        for (int y = 0; y < 32; ++y) r[y] = __float_as_uint(__uint_as_float(r[y]) * f);
        tc_st32(o_row + x, r);
    }
}

// Weights 2^(argument of two scores) of a row's 128 scores: summed into l, and in 16 bits over
// the row's score columns.  The first 64 keys are announced on p_half, the others on p_half + 8.
template <Fused kF, typename Argument>
__device__ __forceinline__ void write_weights(const float (&s)[128], float& l, uint32_t s_tmem, uint32_t p_half,
                                              Argument argument) {
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        uint32_t w[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            const int e = x * 32 + 2 * y;
            float lo, hi;
            f2_unpack(argument(f2_pack(s[e], s[e + 1])), lo, hi);
            lo = ex2(lo);
            hi = ex2(hi);
            sum[y & 1] = f2_add(sum[y & 1], f2_pack(lo, hi));
            w[y] = pack2<kF>(lo, hi);
        }
        tc_st16(s_tmem + x * 16, w);
        if (x == 1 || x == 3) {
            tc_wait_st();
            warp_arrive(p_half + (x == 3 ? 8 : 0));
        }
    }
    float a0, a1;
    f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
    l += a0 + a1;
}

// One tile of keys into a row's softmax: s holds 128 scores (z = c * s, -inf where masked), m the
// reference, l the sum, s_tmem the row's score columns, o_row its output columns.
template <Fused kF, int kD>
__device__ __forceinline__ void fold_tile(float (&s)[128], float c, float down, bool started, float& m, float& l,
                                          uint32_t s_tmem, uint32_t o_row, uint32_t p_half) {
    float top, low;
    bounds_of(s, top, low, false);
    move_reference<kD>(c * top, down, started, m, l, o_row);
    const float base = m == -INFINITY ? 0.f : m;
    const uint64_t c2 = f2_pack(c, c), b2 = f2_pack(-base, -base);
    write_weights<kF>(s, l, s_tmem, p_half, [&](uint64_t v) { return f2_fma(v, c2, b2); });
}

// The same for capped scores without a mask or a bias, from the raw products: z is a polynomial
// (tanh x / x in x^2 times x, the cap folded in), so that the exponent's argument takes 4 to 7
// fused operations; the maximum of z is z of the maximum.  kRaw: the nearest scores skip the
// product x = s * scale / cap, its factor folded into the coefficients (for a factor that
// leaves them in range).  False, with nothing done, where |x| of some row of the warp is
// beyond the polynomials.
constexpr float kTanhNearest = 0.2f;  // second degree in x^2: 1.2e-7 relative
constexpr float kTanhNearest0 = 0.9999998807907104f, kTanhNearest1 = -0.3332858979701996f, kTanhNearest2 = 0.1301540732383728f;
template <Fused kF, int kD, bool kRaw>
__device__ __forceinline__ bool fold_capped_tile(float (&s)[128], float scale, float cap, float down, bool started, float& m,
                                                 float& l, uint32_t s_tmem, uint32_t o_row, uint32_t p_half) {
    const float to_x = scale / cap, to_z = cap * kLog2e;
    float top, low;
    bounds_of(s, top, low, true);
    const float far = fmaxf(fabsf(top), fabsf(low)) * to_x;
    if (!__all_sync(0xffffffffu, far <= kTanhNear)) return false;
    auto both = [](float v) { return f2_pack(v, v); };
    const float unit = kRaw ? to_x : 1.0f, a2 = to_z * unit * unit * unit * unit * unit * kTanhNearest2;
    if (__all_sync(0xffffffffu, far <= kTanhNearest && (!kRaw || (to_x >= 0x1p-16f && a2 <= kFltMax)))) {
        const float a0 = to_z * unit * kTanhNearest0, a1 = to_z * unit * unit * unit * kTanhNearest1;
        const float x = kRaw ? top : top * to_x, y = x * x;
        move_reference<kD>(x * fmaf(y, fmaf(y, a2, a1), a0), down, started, m, l, o_row);
        const uint64_t nb = both(m == -INFINITY ? 0.f : -m), b0 = both(a0), b1 = both(a1), b2 = both(a2), x2 = both(to_x);
        write_weights<kF>(s, l, s_tmem, p_half, [&](uint64_t v) {
            if (!kRaw) v = f2_mul(v, x2);
            const uint64_t y2 = f2_mul(v, v);
            return f2_fma(v, f2_fma(y2, f2_fma(y2, b2, b1), b0), nb);
        });
    } else {
        const float x = top * to_x;
        float t, unused;
        f2_unpack(tanh_over_x(both(x * x)), t, unused);
        move_reference<kD>(to_z * x * t, down, started, m, l, o_row);
        const uint64_t nb = both(m == -INFINITY ? 0.f : -m), x2 = both(to_x), z2 = both(to_z);
        write_weights<kF>(s, l, s_tmem, p_half, [&](uint64_t v) {
            v = f2_mul(v, x2);
            return f2_fma(f2_mul(v, z2), tanh_over_x(f2_mul(v, v)), nb);
        });
    }
    return true;
}

}  // namespace dev
}  // namespace tfu
