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
// One CTA per unit and head of K, of V and of Q; D / 8 lanes hold a row.
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "kv_cache.h"

namespace tfu {

__device__ unsigned g_kv_append_status;

namespace {

using namespace dev;

constexpr int kAppendThreads = 256;
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

// The lane's 8 values of a row, normalised (weight not null) and rotated.
template <Fused kF, int kLanes>
__device__ __forceinline__ void norm_rotate(float (&x)[8], const uint32_t (&raw)[4], const uint32_t* weight, float eps,
                                            const float* table, Rope rope) {
    const uint32_t lane = threadIdx.x % kLanes;
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<kF>(raw[i], x[2 * i], x[2 * i + 1]);
    if (weight) {
        uint64_t x2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x2[i] = f2_pack(x[2 * i], x[2 * i + 1]);
        const float ms = row_mean_sq<kLanes, 4, true>(x2, nullptr);
        const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(ms, eps)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2<kF>(__ldg(weight + lane * 4 + i), a, b);
            x[2 * i] = __fmul_rn(__fmul_rn(x[2 * i], inv), a);
            x[2 * i + 1] = __fmul_rn(__fmul_rn(x[2 * i + 1], inv), b);
        }
    }
    if (rope == Rope::kInterleaved) {
        const float* t = table + lane * 8;  // entries 4 * lane ..: (cos, sin) of pairs (2i, 2i + 1)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float4 cs = ld_table(t + 2 * i);
            float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
            a = x[2 * i + 2];
            b = x[2 * i + 3];
            x[2 * i + 2] = __fsub_rn(__fmul_rn(a, cs.z), __fmul_rn(b, cs.w));
            x[2 * i + 3] = __fadd_rn(__fmul_rn(a, cs.w), __fmul_rn(b, cs.z));
        }
    } else if (rope == Rope::kHalfSplit) {
        const bool upper = lane >= kLanes / 2;
        const float* t = table + (lane % (kLanes / 2)) * 16;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 cs = ld_table(t + 2 * i);
            const float y0 = __shfl_xor_sync(0xffffffffu, x[i], kLanes / 2);
            const float y1 = __shfl_xor_sync(0xffffffffu, x[i + 1], kLanes / 2);
            x[i] = upper ? __fadd_rn(__fmul_rn(y0, cs.y), __fmul_rn(x[i], cs.x))
                         : __fsub_rn(__fmul_rn(x[i], cs.x), __fmul_rn(y0, cs.y));
            x[i + 1] = upper ? __fadd_rn(__fmul_rn(y1, cs.w), __fmul_rn(x[i + 1], cs.z))
                             : __fsub_rn(__fmul_rn(x[i + 1], cs.z), __fmul_rn(y1, cs.w));
        }
    }
}

// kIters: passes of kAppendThreads / (D / 8) rows that a page takes.
template <Fused kF, int kD, int kIters>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
    constexpr int kLanes = kD / 8, kRows = kAppendThreads / kLanes;
    __shared__ float most_of[kAppendThreads / 32];
    grid_dependency_wait();
    const KvCache& c = p.c;
    const uint32_t unit = blockIdx.x;
    // the last sequence whose first unit is not behind this one
    uint32_t before = 0;
    for (uint32_t n0 = 0; n0 < c.N; n0 += kAppendThreads) {
        const uint32_t n = n0 + threadIdx.x;
        before += __syncthreads_count(n < c.N && int64_t(c.starts[n]) / c.page + 2 * int64_t(n) <= int64_t(unit));
    }
    if (before == 0) return;  // rows in front of starts[0] belong to no sequence
    const uint32_t n = before - 1;
    const int64_t s0 = c.starts[n], s1 = c.starts[n + 1], len = c.lens[n];
    const int64_t new_rows = s1 - s0;
    if (s0 < 0 || new_rows < 0 || s1 > int64_t(p.T) || len < new_rows || len > int64_t(c.max_pages) * c.page ||
        (p.rope != Rope::kNone && len > int64_t(p.table_rows))) {
        if (threadIdx.x == 0) atomicOr(&g_kv_append_status, 1u);
        return;
    }
    const int64_t first = len - new_rows;
    const int64_t at = first / c.page + (int64_t(unit) - (s0 / c.page + 2 * int64_t(n)));  // page of the sequence
    const int64_t lo = max(first, at * c.page), hi = min(len, (at + 1) * c.page);
    if (lo >= hi) return;
    const uint32_t rows = uint32_t(hi - lo), off = uint32_t(lo - at * c.page);
    const int64_t row0 = s0 + (lo - first);
    const uint32_t lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;

    uint32_t y = blockIdx.y;
    const bool is_q = y >= 2 * c.Hkv;
    const uint32_t x = is_q ? 0 : y / c.Hkv;  // 0: K, 1: V
    const uint32_t head = is_q ? y - 2 * c.Hkv : y % c.Hkv;
    const uint32_t per_group = is_q ? p.Hl : p.Hkl;
    const RowView& v = is_q ? p.q : p.src[x];
    const uint8_t* src = v.base[head / per_group] + int64_t(head % per_group) * v.h + row0 * v.t + lane * 16;
    const bool plain = !is_q && x == 1;
    const uint32_t* weight = plain ? nullptr : static_cast<const uint32_t*>(p.weight[is_q ? 1 : 0]);
    const Rope rope = plain ? Rope::kNone : p.rope;

    if (is_q) {
        uint8_t* dst = p.q_out.base[head / per_group] + int64_t(head % per_group) * p.q_out.h + row0 * p.q_out.t + lane * 16;
#pragma unroll 1
        for (uint32_t r0 = 0; r0 < rows; r0 += kRows) {
            const uint32_t r = r0 + slot;
            const bool in = r < rows;
            uint32_t raw[4] = {0, 0, 0, 0};
            if (in) {
                const uint4 w = *reinterpret_cast<const uint4*>(src + int64_t(r) * v.t);
                raw[0] = w.x, raw[1] = w.y, raw[2] = w.z, raw[3] = w.w;
            }
            float f[8];
            norm_rotate<kF, kLanes>(f, raw, weight, p.eps, p.table + (in ? lo + r : lo) * kD, rope);
            if (in)
                *reinterpret_cast<uint4*>(dst + int64_t(r) * p.q_out.t) = make_uint4(
                    pack2<kF>(f[0], f[1]), pack2<kF>(f[2], f[3]), pack2<kF>(f[4], f[5]), pack2<kF>(f[6], f[7]));
        }
        return;
    }

    const int64_t id = c.table[int64_t(n) * c.table_stride + at];
    if (id < 0 || id >= int64_t(c.pages)) {
        if (threadIdx.x == 0) atomicOr(&g_kv_append_status, 1u);
        return;
    }
    uint8_t* codes = c.codes[x] + (id * c.Hkv + head) * int64_t(c.page) * kD;
    float* scale_at = c.scales[x] + id * c.Hkv + head;
    const float old = off ? *scale_at : 0.f;

    float f[kIters][8];
    float most = 0.f;
    uint32_t raw[kIters][4];
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
        const uint32_t r = it * kRows + slot;
        const uint4 w = r < rows ? *reinterpret_cast<const uint4*>(src + int64_t(r) * v.t) : make_uint4(0, 0, 0, 0);
        raw[it][0] = w.x, raw[it][1] = w.y, raw[it][2] = w.z, raw[it][3] = w.w;
    }
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
        const uint32_t r = it * kRows + slot;
        norm_rotate<kF, kLanes>(f[it], raw[it], weight, p.eps, p.table + (r < rows ? lo + r : lo) * kD, rope);
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = fabsf(f[it][i]);
                most = a <= kFltMax ? fmaxf(most, a) : most;
            }
        }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, w));
    if (threadIdx.x % 32 == 0) most_of[threadIdx.x / 32] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) most = fmaxf(most, most_of[w]);
    const float fresh = scale_of(most);
    const float scale = fmaxf(old, fresh);
    const float inv = 1.0f / scale;  // exact
    if (off && old < scale) {  // the page's older tokens move to the larger scale
        const float ratio = old * inv;
        for (uint32_t i = threadIdx.x; i < off * kD / 8; i += kAppendThreads) {
            uint2 w = reinterpret_cast<const uint2*>(codes)[i];
            uint32_t* parts[2] = {&w.x, &w.y};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 a = from_e4m3x2(uint16_t(*parts[h])), b = from_e4m3x2(uint16_t(*parts[h] >> 16));
                *parts[h] = uint32_t(e4m3x2(a.x * ratio, a.y * ratio)) | uint32_t(e4m3x2(b.x * ratio, b.y * ratio)) << 16;
            }
            reinterpret_cast<uint2*>(codes)[i] = w;
        }
    }
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
        const uint32_t r = it * kRows + slot;
        if (r >= rows) continue;
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = uint32_t(e4m3x2(f[it][4 * h] * inv, f[it][4 * h + 1] * inv)) |
                   uint32_t(e4m3x2(f[it][4 * h + 2] * inv, f[it][4 * h + 3] * inv)) << 16;
        *reinterpret_cast<uint2*>(codes + int64_t(off + r) * kD + lane * 8) = make_uint2(w[0], w[1]);
    }
    if (threadIdx.x == 0) *scale_at = scale;  // every thread read the old one before the barrier above
}

template <Fused kF, int kD, int kIters>
cudaError_t launch(const KvAppendParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.units, 2 * p.c.Hkv + (p.q.base[0] ? p.P * p.Hl : 0));
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<kF, kD, kIters>, p);
}

template <Fused kF>
cudaError_t launch_typed(const KvAppendParams& p, cudaStream_t stream) {
    if (p.c.D == 64)
        return p.c.page <= 32 ? launch<kF, 64, 1>(p, stream) : p.c.page == 64 ? launch<kF, 64, 2>(p, stream)
                                                                              : launch<kF, 64, 4>(p, stream);
    switch (p.c.page) {
        case 16: return launch<kF, 128, 1>(p, stream);
        case 32: return launch<kF, 128, 2>(p, stream);
        case 64: return launch<kF, 128, 4>(p, stream);
        default: return launch<kF, 128, 8>(p, stream);
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_typed<Fused::kBF16>(p, stream) : launch_typed<Fused::kFP16>(p, stream);
}

cudaError_t read_kv_append_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv_append_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_kv_append_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
