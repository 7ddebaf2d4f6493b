// kv_attend.cu -- attention of each sequence's newest tokens over the paged 8-bit cache.
//
// The scores and the softmax are those of attention_forward.cu with K = code * scale
// and V = code * scale of the page's head; key j of a sequence is in page j / page_size of
// its table row.
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "kv_cache.h"

namespace tfu {

__device__ unsigned g_kv_attend_status;

namespace {

using namespace dev;

constexpr int kRowThreads = 128;
constexpr int kKeys = 16;  // keys of a block: a page is a whole number of blocks

__device__ __forceinline__ float from_e4m3(uint8_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
    return __half2float(__ushort_as_half(uint16_t(h)));
}

template <Fused kF>
__device__ __forceinline__ float to_float(uint16_t v) {
    float lo, hi;
    unpack2<kF>(uint32_t(v), lo, hi);
    return lo;
}

// A row is a (token, query head) pair of one sequence and key head; kLanes = D / 32 lanes share it.
template <Fused kF, int kD>
__global__ void __launch_bounds__(kRowThreads) kv_attend_kernel(const __grid_constant__ KvAttendParams p) {
    constexpr int kLanes = kD / 32, kRows = kRowThreads / kLanes;
    __shared__ float ks[kKeys][kD], vs[kKeys][kD];
    const KvCache& c = p.c;
    const uint32_t part = threadIdx.x % kLanes;
    const uint32_t kh = blockIdx.y, n = blockIdx.z;
    const int64_t s0 = c.starts[n], s1 = c.starts[n + 1], len = c.lens[n];
    const int64_t tokens = s1 - s0;
    if (s0 < 0 || tokens < 0 || s1 > int64_t(p.T) || len < tokens || len > int64_t(p.max_len) || tokens > int64_t(p.max_tokens)) {
        if (threadIdx.x == 0) atomicOr(&g_kv_attend_status, 1u);
        return;
    }
    const int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes;
    if (int64_t(blockIdx.x) * kRows >= tokens * p.shared) return;
    const bool valid = r < tokens * p.shared;
    const int64_t token = valid ? r / p.shared : 0;
    const uint32_t head = kh * p.shared + uint32_t(valid ? r % p.shared : 0);  // over all groups
    const uint32_t g = head / p.Hl, h = head % p.Hl;
    float q[32], o[32];
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.q.base[g] + (s0 + token) * p.q.t + h * p.q.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) {
        q[d] = valid ? to_float<kF>(qp[part * 32 + d]) : 0.f;
        o[d] = 0.f;
    }
    const int64_t pos = len - tokens + token;
    const int64_t bound = !valid ? 0 : p.causal ? pos + 1 : len;
    const float slope = p.slopes ? p.slopes[head] : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int64_t j0 = 0; j0 < len; j0 += kKeys) {
        if (!__syncthreads_or(j0 < bound)) break;
        const int64_t id = c.table[n * c.table_stride + j0 / c.page];
        const bool bad = id < 0 || id >= int64_t(c.pages);
        if (bad) {
            if (threadIdx.x == 0) atomicOr(&g_kv_attend_status, 1u);
            continue;
        }
        const int64_t at = (id * c.Hkv + kh) * int64_t(c.page) + j0 % c.page;
        const float sk = c.scales[0][id * c.Hkv + kh], sv = c.scales[1][id * c.Hkv + kh];
        for (int x = threadIdx.x; x < kKeys * kD; x += kRowThreads) {
            const int j = x / kD, d = x % kD;
            const bool in = j0 + j < len;
            ks[j][d] = in ? from_e4m3(c.codes[0][(at + j) * kD + d]) * sk : 0.f;
            vs[j][d] = in ? from_e4m3(c.codes[1][(at + j) * kD + d]) * sv : 0.f;
        }
        __syncthreads();
        float z[kKeys], top = m;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            float s = 0.f;
#pragma unroll
            for (int d = 0; d < 32; ++d) s = fmaf(q[d], ks[j][part * 32 + d], s);
#pragma unroll
            for (int w = 1; w < kLanes; w <<= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
            s *= p.scale;
            if (p.cap != 0.f) s = p.cap * tanhf(s / p.cap);
            s -= slope * fabsf(float(pos - (j0 + j)));
            z[j] = j0 + j < bound ? s : -INFINITY;
            top = fmaxf(top, z[j]);
        }
        const float base = top == -INFINITY ? 0.f : top;
        const float shrink = expf(m - base);
        l *= shrink;
#pragma unroll
        for (int d = 0; d < 32; ++d) o[d] *= shrink;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            if (z[j] == -INFINITY) continue;
            const float e = expf(z[j] - base);
            l += e;
#pragma unroll
            for (int d = 0; d < 32; ++d) o[d] = fmaf(e, vs[j][part * 32 + d], o[d]);
        }
        m = top;
    }
    if (!valid) return;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    uint16_t* op = reinterpret_cast<uint16_t*>(p.out.base[g] + (s0 + token) * p.out.t + h * p.out.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) op[part * 32 + d] = uint16_t(pack2<kF>(o[d] * inv, 0.f) & 0xffffu);
    if (p.lse[g] && part == 0) p.lse[g][int64_t(h) * p.T + s0 + token] = m + logf(l);
}

template <Fused kF, int kD>
cudaError_t launch(const KvAttendParams& p, cudaStream_t stream) {
    constexpr uint32_t kRows = kRowThreads / (kD / 32);
    kv_attend_kernel<kF, kD><<<dim3((p.max_tokens * p.shared + kRows - 1) / kRows, p.c.Hkv, p.c.N), kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendParams& p, bool bf16, cudaStream_t stream) {
    if (p.c.D == 64) return bf16 ? launch<Fused::kBF16, 64>(p, stream) : launch<Fused::kFP16, 64>(p, stream);
    return bf16 ? launch<Fused::kBF16, 128>(p, stream) : launch<Fused::kFP16, 128>(p, stream);
}

cudaError_t read_kv_attend_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv_attend_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_kv_attend_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
