// kv_append.cu -- appending rows of K and V to the paged 8-bit cache, with the
// RMSNorm and the rotation on the way, and the queries of the same tokens beside them.
//
// For each (page, head) that gets new rows x (fp32, after the norm and rotation):
//   e = the least exponent with max |x| <= 448 * 2^e (finite values only, e >= -100)
//   s = 2^e, or max(s_old, 2^e) when the page already holds tokens of the sequence
//   code = e4m3(x / s), one rounding; older codes become e4m3(code * s_old / s) when s grew
// Scales are powers of two, so that a division by one is exact, the 3-bit mantissa
// loses nothing against a scale of max/448, and rescaling older codes rounds only
// those that fall below e4m3's normal range.
//
// A unit is one page of one sequence; unit u of a call belongs to the sequence n
// with first(n) <= u < first(n + 1), first(n) = starts[n] / page + 2n, which leaves
// room for every page that t = starts[n + 1] - starts[n] rows can touch
// (at most (t - 1) / page + 2), so that the grid needs no length from the device.
// A CTA takes a unit and every slices-th head of K, of V and of Q; D / 16 lanes hold a row.
//
// Bound by latency and instructions: 4680 rows of 40 heads (D = 128, bf16, norm and rotation, pages of 64) take
// 67 us, 3.6 TB/s of 243 MB, with issue slots busy 49 % of the cycles, 16 warps an SM and long_scoreboard as the first
// stall: a CTA's every head loads its rows' rotation and the norm's weights again.  A lane's 16 values cost
// about 240 instructions a row.  Summing the squares plainly took 85 us to 79, room in registers for
// two passes 79 to 68.  Pages of 128 (four passes at D = 128, 84 bytes spilled): 77 us.
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "kv_cache.h"

namespace tfu {

__device__ unsigned g_kv_append_status;

namespace {

using namespace dev;

constexpr int kLeastExponent = -100;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 2^e for the least e >= kLeastExponent with most <= 448 * 2^e; most is finite and >= 0.
__device__ __forceinline__ float scale_of(float most) {
    const uint32_t bits = __float_as_uint(most);
    int e = int(bits >> 23) - 126;                 // most = m * 2^e, m in [0.5, 1) (below 2^-126: e = -126, clamped)
    e -= (bits & 0x7fffffu) <= 0x600000u ? 9 : 8;  // 448 = 0.875 * 2^9; m <= 0.875
    return __uint_as_float(uint32_t((e < kLeastExponent ? kLeastExponent : e) + 127) << 23);
}

// A lane's 16 values of a row: elements [8l, 8l + 8) and kD / 2 further on, so that both kinds of
// pairs lie within a lane.  raw[i]: values 2i, 2i + 1 of x.
template <int kD>
struct Lane {
    static constexpr int kLanes = kD / 16;  // of a row
    __device__ static __forceinline__ void load(uint32_t (&raw)[8], const uint8_t* row, bool in) {
        const uint32_t l = threadIdx.x % kLanes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 w = in ? *reinterpret_cast<const uint4*>(row + h * kD + l * 16) : make_uint4(0, 0, 0, 0);
            raw[4 * h] = w.x, raw[4 * h + 1] = w.y, raw[4 * h + 2] = w.z, raw[4 * h + 3] = w.w;
        }
    }
};

// The lane's values, normalised (kNorm: w holds the weights) and rotated; table: the row's
// (cos, sin) entries.
template <Fused kF, int kD>
__device__ __forceinline__ void norm_rotate(float (&x)[16], const uint32_t (&raw)[8], bool norm, const float (&w)[16], float eps,
                                            const float* table, Rope rope) {
    constexpr int kLanes = Lane<kD>::kLanes;
    const uint32_t l = threadIdx.x % kLanes;
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack2<kF>(raw[i], x[2 * i], x[2 * i + 1]);
    if (norm) {
        uint64_t x2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x2[i] = f2_pack(x[2 * i], x[2 * i + 1]);
        // 8 squares a half, then the halves and kLanes lanes: within 6 * 2^-24 of the sum where it is finite
        uint64_t s2 = f2_mul(x2[0], x2[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = f2_fma(x2[i], x2[i], s2);
        float ms, other;
        f2_unpack(s2, ms, other);
        ms = __fadd_rn(ms, other);
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) ms = __fadd_rn(ms, __shfl_xor_sync(0xffffffffu, ms, m));
        ms = __fmul_rn(ms, 1.0f / kD);
        // A sum that is not finite: again from 2^-72 x, for the whole warp (it holds several rows, and
        // shuffles over all of its lanes).  A mean beyond fp32 is infinite, and its row 0.
        if (!__all_sync(0xffffffffu, ms <= kFltMax)) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) t = fmaf(x[i] * 0x1p-72f, x[i] * 0x1p-72f, t);
#pragma unroll
            for (int m = 1; m < kLanes; m <<= 1) t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, m));
            if (!(ms <= kFltMax)) ms = t * (1.0f / kD) * 0x1p72f * 0x1p72f;
        }
        const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(ms, eps)));
        const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
        for (int i = 0; i < 8; ++i) f2_unpack(f2_mul(f2_mul(x2[i], inv2), f2_pack(w[2 * i], w[2 * i + 1])), x[2 * i], x[2 * i + 1]);
    }
    if (rope == Rope::kInterleaved) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {  // entries of pairs (8h + 2i, + 1) and (8h + 2i + 2, + 3)
                const float4 cs = ld_table(table + h * (kD / 2) + l * 8 + 2 * i);
                float* v = x + 8 * h + 2 * i;
                float a = v[0], b = v[1];
                v[0] = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
                v[1] = __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
                a = v[2];
                b = v[3];
                v[2] = __fsub_rn(__fmul_rn(a, cs.z), __fmul_rn(b, cs.w));
                v[3] = __fadd_rn(__fmul_rn(a, cs.w), __fmul_rn(b, cs.z));
            }
    } else if (rope == Rope::kHalfSplit) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 cs = ld_table(table + l * 16 + 2 * i);
            float a = x[i], b = x[i + 8];
            x[i] = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
            x[i + 8] = __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
            a = x[i + 1];
            b = x[i + 9];
            x[i + 1] = __fsub_rn(__fmul_rn(a, cs.z), __fmul_rn(b, cs.w));
            x[i + 9] = __fadd_rn(__fmul_rn(a, cs.w), __fmul_rn(b, cs.z));
        }
    }
}

// kIters: passes of kThreads / (D / 16) rows that a page takes.  Registers: two passes in 128 of them
// without spills took 68 us for 4680 rows of 40 heads in pages of 64, in 80 with spills 79.
template <Fused kF, int kD, int kIters, int kThreads>
__global__ void __launch_bounds__(kThreads, kIters == 1 ? 1024 / kThreads : 2) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
    constexpr int kLanes = Lane<kD>::kLanes, kRows = kThreads / kLanes;
    __shared__ float most_of[2][kThreads / 32];
    grid_dependency_wait();
    const KvCache& c = p.c;
    const uint32_t unit = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    const uint32_t shift = 31 - __clz(c.page);  // pages are powers of two
    // the last sequence whose first unit is not behind this one.  Starts that do not ascend within [0, T] may
    // have units that nothing visits: the first CTA looks at all of them
    uint32_t before = 0;
    for (uint32_t n0 = 0; n0 < c.N; n0 += kThreads) {
        const uint32_t n = n0 + threadIdx.x;
        if (blockIdx.x == 0 && n < c.N) {
            const int s0 = c.starts[n], s1 = c.starts[n + 1];
            if (s0 < 0 || s1 < s0 || s1 > int64_t(p.T)) atomicOr(&g_kv_append_status, 1u);
        }
        before += __syncthreads_count(n < c.N && int64_t(c.starts[n] >> shift) + 2 * int64_t(n) <= int64_t(unit));
    }
    if (before == 0) return;  // rows in front of starts[0] belong to no sequence
    const uint32_t n = before - 1;
    const int64_t s0 = c.starts[n], s1 = c.starts[n + 1], len = c.lens[n];
    const int64_t new_rows = s1 - s0;
    if (s0 < 0 || new_rows < 0 || s1 > int64_t(p.T) || len < new_rows || len > int64_t(c.max_pages) << shift ||
        (p.rope != Rope::kNone && len > int64_t(p.table_rows))) {
        if (threadIdx.x == 0) atomicOr(&g_kv_append_status, 1u);
        return;
    }
    const int64_t first = len - new_rows;
    const int64_t at = (first >> shift) + (int64_t(unit) - ((s0 >> shift) + 2 * int64_t(n)));  // page of the sequence
    const int64_t lo = max(first, at << shift), hi = min(len, (at + 1) << shift);
    if (lo >= hi) return;
    const uint32_t rows = uint32_t(hi - lo), off = uint32_t(lo - (at << shift));
    const int64_t row0 = s0 + (lo - first);
    const uint32_t lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
    const int64_t id = c.table[int64_t(n) * c.table_stride + at];
    const bool bad = id < 0 || id >= int64_t(c.pages);
    if (bad && threadIdx.x == 0) atomicOr(&g_kv_append_status, 1u);

    // heads of K, of V, of Q: this CTA takes every slices-th; the next one's rows are on their way
    // while one is computed
    struct Head {
        uint32_t kind, head;  // 0: K, 1: V, 2: Q
        const uint8_t* src;
        int64_t step;
    };
    const uint32_t heads = 2 * c.Hkv + (p.q.base[0] ? p.P * p.Hl : 0);
    auto head_of = [&](uint32_t y) {
        Head d;
        d.kind = y < c.Hkv ? 0 : y < 2 * c.Hkv ? 1 : 2;
        d.head = y - d.kind * c.Hkv;
        const RowView& v = d.kind == 2 ? p.q : p.src[d.kind];
        const uint32_t per_group = d.kind == 2 ? p.Hl : p.Hkl;
        d.step = v.t;
        d.src = v.base[d.head / per_group] + int64_t(d.head % per_group) * v.h + row0 * v.t;
        return d;
    };
    auto load = [&](uint32_t (&raw)[kIters][8], const Head& d, bool any) {
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            const uint32_t r = it * kRows + slot;
            Lane<kD>::load(raw[it], d.src + int64_t(r) * d.step, any && r < rows);
        }
    };
    uint32_t raw[kIters][8];
    Head now = head_of(slice);
    load(raw, now, slice < heads);
    uint32_t turn = 0;
    for (uint32_t y = slice; y < heads; y += p.slices, turn ^= 1u) {
        const bool plain = now.kind == 1;
        const uint8_t* weight = plain ? nullptr : static_cast<const uint8_t*>(p.weight[now.kind == 2 ? 1 : 0]);
        const Rope rope = plain ? Rope::kNone : p.rope;
        float w[16];
        {
            uint32_t packed[8];
            Lane<kD>::load(packed, weight, weight != nullptr);
#pragma unroll
            for (int i = 0; i < 8; ++i) unpack2<kF>(packed[i], w[2 * i], w[2 * i + 1]);
        }
        float* scale_at = c.scales[plain ? 1 : 0] + (bad ? 0 : id * c.Hkv + now.head);
        const float old = now.kind < 2 && off && !bad ? *scale_at : 0.f;
        float f[kIters][16];
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            const uint32_t r = it * kRows + slot;
            norm_rotate<kF, kD>(f[it], raw[it], weight != nullptr, w, p.eps, p.table + (r < rows ? lo + r : lo) * kD, rope);
        }
        const Head done = now;
        now = head_of(y + p.slices < heads ? y + p.slices : y);
        load(raw, now, y + p.slices < heads);
        if (done.kind == 2) {
            const uint32_t g = done.head / p.Hl, h = done.head % p.Hl;
            uint8_t* dst = p.q_out.base[g] + int64_t(h) * p.q_out.h + row0 * p.q_out.t + lane * 16;
#pragma unroll
            for (int it = 0; it < kIters; ++it) {
                const uint32_t r = it * kRows + slot;
                if (r >= rows) continue;
                const float* e = f[it];
#pragma unroll
                for (int x = 0; x < 2; ++x, e += 8)
                    *reinterpret_cast<uint4*>(dst + int64_t(r) * p.q_out.t + x * kD) =
                        make_uint4(pack2<kF>(e[0], e[1]), pack2<kF>(e[2], e[3]), pack2<kF>(e[4], e[5]), pack2<kF>(e[6], e[7]));
            }
            continue;
        }
        if (bad) continue;  // the same for the whole CTA
        float most = 0.f;
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            if (it * kRows + slot >= rows) continue;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(f[it][i]));  // passes over NaN
        }
        if (!(most <= kFltMax)) {  // infinities do not count
            most = 0.f;
#pragma unroll
            for (int it = 0; it < kIters; ++it)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = fabsf(f[it][i]);
                    if (it * kRows + slot < rows && a <= kFltMax) most = fmaxf(most, a);
                }
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
        if (threadIdx.x % 32 == 0) most_of[turn][threadIdx.x / 32] = most;
        __syncthreads();  // also: every thread has read the old scale, and the other turn's maxima
#pragma unroll
        for (int x = 0; x < kThreads / 32; ++x) most = fmaxf(most, most_of[turn][x]);
        const float scale = fmaxf(old, scale_of(most));
        const float inv = 1.0f / scale;  // exact
        uint8_t* codes = c.codes[done.kind] + ((id * c.Hkv + done.head) << shift) * kD;
        if (off && old < scale) {  // the page's older tokens move to the larger scale
            const float ratio = old * inv;
            for (uint32_t i = threadIdx.x; i < off * kD / 8; i += kThreads) {
                uint2 u = reinterpret_cast<const uint2*>(codes)[i];
                uint32_t* parts[2] = {&u.x, &u.y};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 a = from_e4m3x2(uint16_t(*parts[h])), b = from_e4m3x2(uint16_t(*parts[h] >> 16));
                    *parts[h] = uint32_t(e4m3x2(a.x * ratio, a.y * ratio)) | uint32_t(e4m3x2(b.x * ratio, b.y * ratio)) << 16;
                }
                reinterpret_cast<uint2*>(codes)[i] = u;
            }
        }
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            const uint32_t r = it * kRows + slot;
            if (r >= rows) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t u[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float* e = f[it] + 8 * h + 4 * z;
                    u[z] = uint32_t(e4m3x2(e[0] * inv, e[1] * inv)) | uint32_t(e4m3x2(e[2] * inv, e[3] * inv)) << 16;
                }
                *reinterpret_cast<uint2*>(codes + int64_t(off + r) * kD + h * (kD / 2) + lane * 8) = make_uint2(u[0], u[1]);
            }
        }
        if (threadIdx.x == 0) *scale_at = scale;
    }
}

// CTAs of a call: enough for kAppendCtas, so that a CTA takes several heads and has the next
// one's rows on their way; a head each where there are few units.
constexpr uint32_t kAppendCtas = 1824;

template <Fused kF, int kD, int kIters, int kThreads>
cudaError_t launch(KvAppendParams p, cudaStream_t stream) {
    const uint32_t heads = 2 * p.c.Hkv + (p.q.base[0] ? p.P * p.Hl : 0), want = (kAppendCtas + p.units - 1) / p.units;
    p.slices = want < heads ? want : heads;
    return launch_overlapped(kv_append_kernel<kF, kD, kIters, kThreads>, p.units * p.slices, kThreads, 0, stream, p);
}

// As many threads as a page's rows have lanes, up to 256.
template <Fused kF, int kD>
cudaError_t launch_typed(const KvAppendParams& p, cudaStream_t stream) {
    constexpr int kLeast = 16 * Lane<kD>::kLanes;  // a page of 16: 64 threads at D = 64, 128 at D = 128
    switch (p.c.page) {
        case 16: return launch<kF, kD, 1, kLeast>(p, stream);
        case 32: return launch<kF, kD, 1, 2 * kLeast>(p, stream);
        case 64: return launch<kF, kD, kLeast / 64, 256>(p, stream);
        default: return launch<kF, kD, kLeast / 32, 256>(p, stream);  // 128
    }
}

template <Fused kF>
cudaError_t launch_sized(const KvAppendParams& p, cudaStream_t stream) {
    return p.c.D == 64 ? launch_typed<kF, 64>(p, stream) : launch_typed<kF, 128>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_sized<Fused::kBF16>(p, stream) : launch_sized<Fused::kFP16>(p, stream);
}

cudaError_t read_kv_append_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv_append_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_kv_append_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
