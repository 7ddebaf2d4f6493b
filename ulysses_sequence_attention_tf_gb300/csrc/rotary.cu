// rotary.cu -- rotary positions of Q and K where they lie: a part of the head, any frequencies, any positions.
//
//   x0' = m (x0 cos a - x1 sin a)     x1' = m (x0 sin a + x1 cos a)     a = position * frequency
//
// The angle is kept in turns as a 64-bit fraction: position times the frequency's fraction, modulo
// 2^64, is the angle modulo one turn, whatever the position; the fraction itself is the nearest of 64 bits (rotary_turns.h), so
// position 2^31 is 2^-34 of a turn off.  Its upper 32 bits give the sine and cosine.  So no table is read and no 64-bit
// float is computed, and the positions may come from the device.
//
// A thread takes one item of a row -- one vector of 8 elements (4 pairs) with interleaved pairs, two
// vectors half of R apart (their pairs) with half-split ones -- and a set of heads, for which the sines and cosines
// are the same.  Bound: DRAM, each row read and written once.  80 heads of 32760 tokens, D = 128, bf16: 197 us, 6.8 TB/s,
// the copy bandwidth (217 with sincospif and a division for every head); 24 heads of 12002 tokens, half of D = 64: 14 us,
// 5.2 TB/s.  With few heads a row's sines and cosines show: 4 heads of 60000 tokens 30 us, 4.1 TB/s.
#include "device_common.cuh"
#include "rotary.h"

namespace tfu {
namespace {

using namespace dev;

constexpr int kThreadsR = 256;
constexpr int kUnroll = 4;  // heads whose loads are on their way together

// W 16-bit elements as they lie in memory.
template <int W>
struct Packed {
    uint32_t w[(W + 1) / 2];
};
// Not the read-only path: in place, the same kernel writes these addresses.
template <int W>
__device__ __forceinline__ Packed<W> load(const uint8_t* p) {
    Packed<W> v;
    if constexpr (W == 8)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
                     : "l"(p)
                     : "memory");
    else if constexpr (W == 4)
        asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.w[0]), "=r"(v.w[1]) : "l"(p) : "memory");
    else if constexpr (W == 2)
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(v.w[0]) : "l"(p) : "memory");
    else
        v.w[0] = *reinterpret_cast<const volatile uint16_t*>(p);
    return v;
}
template <int W>
__device__ __forceinline__ void store(uint8_t* p, const Packed<W>& v) {
    if constexpr (W == 8)
        asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3])
                     : "memory");
    else if constexpr (W == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
    else if constexpr (W == 2)
        *reinterpret_cast<uint32_t*>(p) = v.w[0];
    else
        *reinterpret_cast<uint16_t*>(p) = uint16_t(v.w[0]);
}

// Sine and cosine of a 32-bit fraction of a turn: the nearest quarter turn taken off exactly, then the Taylor series in
// [-pi/4, pi/4] (sine to x^9, remainder 1.8e-9; cosine to x^8, 2.5e-8) with fp32's roundings, about 1.2e-7 altogether.
__device__ __forceinline__ void sine_cosine(uint32_t turn, float& s, float& c) {
    const uint32_t quarter = (turn + (1u << 29)) >> 30;
    const float x = float(int32_t(turn - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    const float near_s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float near_c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
    s = quarter & 1u ? near_c : near_s;
    c = quarter & 1u ? near_s : near_c;
    s = __uint_as_float(__float_as_uint(s) ^ ((quarter & 2u) << 30));         // sine: + + - -
    c = __uint_as_float(__float_as_uint(c) ^ (((quarter + 1) & 2u) << 30));   // cosine: + - - +
}

template <Fused kF, bool kHalfSplit, int W>
__global__ void __launch_bounds__(kThreadsR) rotary_kernel(const __grid_constant__ RotaryParams p) {
    constexpr int kPairs = kHalfSplit ? W : W / 2;
    grid_dependency_wait();
    const uint32_t rows_here = kThreadsR / p.items;
    const uint32_t local = threadIdx.x / p.items, item = threadIdx.x % p.items;
    const uint64_t row = uint64_t(blockIdx.x / p.chunks) * rows_here + local;
    if (local >= rows_here || row >= uint64_t(p.B) * p.T) return;
    const uint32_t b = uint32_t(row / p.T), t = uint32_t(row % p.T);
    const uint32_t half = p.R / 2, rotating = kHalfSplit ? half / W : (p.R + W - 1) / W;
    const bool turns = item < rotating;
    // byte offsets of the item's one or two vectors in a head row
    const uint32_t lo = (turns || !kHalfSplit ? item * W : p.R + (item - rotating) * 2 * W) * 2;
    const uint32_t hi = turns ? lo + half * 2 : lo + W * 2;
    const bool second = kHalfSplit && hi < p.D * 2;
    float c[kPairs], s[kPairs];
    uint32_t keep = 0;  // pairs of the last vector that lie behind R
    if (turns) {
        const int64_t at = p.positions ? int64_t(p.positions[row]) : int64_t(p.first) + t;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const uint32_t pair = item * kPairs + i;
            if (pair >= half) keep |= 1u << i;
            sine_cosine(uint32_t((uint64_t(at) * p.turn[pair < half ? pair : 0]) >> 32), s[i], c[i]);
            s[i] *= p.magnitude * p.sign;
            c[i] *= p.magnitude;
        }
    }
    const uint32_t first = blockIdx.x % p.chunks * p.chunk, last = min(first + p.chunk, p.heads);
#pragma unroll 1
    for (uint32_t which = 0; which < 2; ++which) {
        const RotaryTensor& y = p.x[which];
        // this tensor's heads among the thread's
        const uint32_t begin = which ? max(first, p.q_heads) - p.q_heads : first, end = which ? max(last, p.q_heads) - p.q_heads : min(last, p.q_heads);
        if (begin >= end || (!turns && y.in_place)) continue;
        uint32_t g = begin / y.Hl, h = begin - g * y.Hl;
        const int64_t in_row = int64_t(b) * y.ib + int64_t(t) * y.it, out_row = int64_t(b) * y.ob + int64_t(t) * y.ot;
        for (uint32_t x0 = begin; x0 < end; x0 += kUnroll) {
            Packed<W> a[kUnroll], z[kUnroll];
            uint8_t* dst[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                dst[u] = nullptr;
                if (x0 + u >= end) continue;
                const uint8_t* src = y.in[g] + in_row + int64_t(h) * y.ih;
                dst[u] = y.out[g] + out_row + int64_t(h) * y.oh;
                a[u] = load<W>(src + lo);
                if (second) z[u] = load<W>(src + hi);
                if (++h == y.Hl) h = 0, ++g;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (!dst[u]) continue;
                if (turns) {
                    if constexpr (kHalfSplit) {
#pragma unroll
                        for (int i = 0; i < (W + 1) / 2; ++i) {
                            float a0, a1, z0, z1;
                            unpack2<kF>(a[u].w[i], a0, a1);
                            unpack2<kF>(z[u].w[i], z0, z1);
                            const int j = W > 1 ? 2 * i + 1 : 0;
                            a[u].w[i] = pack2<kF>(a0 * c[2 * i] - z0 * s[2 * i], a1 * c[j] - z1 * s[j]);
                            z[u].w[i] = pack2<kF>(a0 * s[2 * i] + z0 * c[2 * i], a1 * s[j] + z1 * c[j]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kPairs; ++i) {
                            float x0f, x1f;
                            unpack2<kF>(a[u].w[i], x0f, x1f);
                            const uint32_t turned = pack2<kF>(x0f * c[i] - x1f * s[i], x0f * s[i] + x1f * c[i]);
                            a[u].w[i] = (keep >> i) & 1u ? a[u].w[i] : turned;
                        }
                    }
                }
                store<W>(dst[u] + lo, a[u]);
                if (second) store<W>(dst[u] + hi, z[u]);
            }
        }
    }
}

template <Fused kF>
cudaError_t launch(const RotaryParams& p, bool half_split, uint32_t width, uint32_t grid, cudaStream_t stream) {
    if (!half_split) return launch_overlapped(rotary_kernel<kF, false, 8>, grid, kThreadsR, 0, stream, p);
    switch (width) {
        case 8: return launch_overlapped(rotary_kernel<kF, true, 8>, grid, kThreadsR, 0, stream, p);
        case 4: return launch_overlapped(rotary_kernel<kF, true, 4>, grid, kThreadsR, 0, stream, p);
        case 2: return launch_overlapped(rotary_kernel<kF, true, 2>, grid, kThreadsR, 0, stream, p);
        default: return launch_overlapped(rotary_kernel<kF, true, 1>, grid, kThreadsR, 0, stream, p);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, bool bf16, bool half_split, uint32_t width, cudaStream_t stream) {
    const uint32_t rows_here = kThreadsR / p.items;
    const uint64_t blocks = (uint64_t(p.B) * p.T + rows_here - 1) / rows_here;
    const uint32_t grid = uint32_t(blocks * p.chunks);
    return bf16 ? launch<Fused::kBF16>(p, half_split, width, grid, stream) : launch<Fused::kFP16>(p, half_split, width, grid, stream);
}

}  // namespace tfu
