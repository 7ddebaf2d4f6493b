// attention_forward.cu -- attention over the head groups, forward.
//
// One pass over the keys with the running maximum m and sum l of each row's
// softmax (Milakov & Gimelshein, "Online normalizer calculation for softmax",
// 2018): for each block of keys, m' = max(m, max z), l = l e^(m - m') + sum e^(z - m'),
// o = o e^(m - m') + sum e^(z - m') v.  Everything in fp32; the output is rounded once.
#include "attention_common.cuh"

namespace tfu {

namespace {

using namespace dev;

constexpr int kRowThreads = 128;
constexpr int kKeys = 32;  // keys of a block

// kLanes = D / 32 lanes share a query row, 32 dims each.
template <Fused kF, int kD>
__global__ void __launch_bounds__(kRowThreads) attention_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kLanes = kD / 32, kRows = kRowThreads / kLanes;
    __shared__ float ks[kKeys][kD], vs[kKeys][kD];
    __shared__ int32_t kdoc[kKeys];
    const uint32_t part = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const uint32_t h = blockIdx.y % p.Hl, b = blockIdx.y / p.Hl % p.B, g = blockIdx.y / p.Hl / p.B;
    const uint32_t kh = h / p.shared;
    const int64_t i = int64_t(blockIdx.x) * kRows + row;
    const bool valid = i < int64_t(p.Sq);
    float q[32], o[32];
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.q.base[g] + b * p.q.b + (valid ? i : 0) * p.q.t + h * p.q.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) {
        q[d] = valid ? to_float<kF>(qp[part * 32 + d]) : 0.f;
        o[d] = 0.f;
    }
    const int bound = valid ? key_bound(p, b, i) : 0;
    const int32_t doc = valid && p.q_docs ? p.q_docs[int64_t(b) * p.Sq + i] : -1;
    const float slope = p.slopes ? p.slopes[g * p.Hl + h] : 0.f;
    const int64_t pos = i + int64_t(p.Sk) - int64_t(p.Sq);
    float m = -INFINITY, l = 0.f;
    const uint8_t* kb = p.k.base[g] + b * p.k.b + kh * p.k.h;
    const uint8_t* vb = p.v.base[g] + b * p.v.b + kh * p.v.h;
    for (int j0 = 0; j0 < int(p.Sk); j0 += kKeys) {
        if (!__syncthreads_or(j0 < bound)) break;
        for (int x = threadIdx.x; x < kKeys * kD; x += kRowThreads) {
            const int j = x / kD, d = x % kD;
            const bool in = j0 + j < int(p.Sk);
            ks[j][d] = in ? to_float<kF>(reinterpret_cast<const uint16_t*>(kb + int64_t(j0 + j) * p.k.t)[d]) : 0.f;
            vs[j][d] = in ? to_float<kF>(reinterpret_cast<const uint16_t*>(vb + int64_t(j0 + j) * p.v.t)[d]) : 0.f;
        }
        if (p.k_docs && threadIdx.x < kKeys)
            kdoc[threadIdx.x] = j0 + int(threadIdx.x) < int(p.Sk) ? p.k_docs[int64_t(b) * p.Sk + j0 + threadIdx.x] : -1;
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
            const bool see = j0 + j < bound && (!p.k_docs || (doc >= 0 && kdoc[j] == doc));
            z[j] = see ? s : -INFINITY;
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
        __syncthreads();
    }
    if (!valid) return;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    uint16_t* op = reinterpret_cast<uint16_t*>(p.out.base[g] + b * p.out.b + i * p.out.t + h * p.out.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) op[part * 32 + d] = to_half<kF>(o[d] * inv);
    if (p.lse[g] && part == 0) p.lse[g][(int64_t(b) * p.Hl + h) * p.Sq + i] = m + logf(l);
}

template <Fused kF, int kD>
cudaError_t launch(const AttentionParams& p, cudaStream_t stream) {
    constexpr uint32_t kRows = kRowThreads / (kD / 32);
    attention_kernel<kF, kD><<<dim3((p.Sq + kRows - 1) / kRows, p.B * p.P * p.Hl), kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const AttentionParams& p, bool bf16, cudaStream_t stream) {
    if (p.D == 64) return bf16 ? launch<Fused::kBF16, 64>(p, stream) : launch<Fused::kFP16, 64>(p, stream);
    return bf16 ? launch<Fused::kBF16, 128>(p, stream) : launch<Fused::kFP16, 128>(p, stream);
}

}  // namespace tfu
