// attention_backward.cu -- the gradient of the attention over the head groups.
//
// With the weights P_ij = e^(z_ij - lse_i) recomputed from Q, K and the saved
// log-sum-exp, and delta_i = sum_d dO_id O_id:
//   dV_j = sum_i P_ij dO_i
//   dx_ij = P_ij (dO_i . V_j - delta_i) (1 - tanh^2(x_ij / cap))    (the last factor where scores are capped)
//   dQ_i = scale * sum_j dx_ij K_j        dK_j = scale * sum_i dx_ij Q_i
// dQ is summed by the rows that own it in one kernel, dK and dV by the keys that
// own them in another (over all query heads that share the key head): no atomics,
// so the same inputs give the same bits.
#include "attention_common.cuh"

namespace tfu {

namespace {

using namespace dev;

constexpr int kRowThreads = 128;
constexpr int kOther = 16;  // rows of the other side in a block

// delta_i = sum_d dO_id O_id: a warp per row.
template <Fused kF>
__global__ void __launch_bounds__(256) delta_kernel(const __grid_constant__ AttentionParams p) {
    const uint64_t rows = uint64_t(p.P) * p.B * p.Hl * p.Sq;
    const uint64_t r = uint64_t(blockIdx.x) * 8 + threadIdx.x / 32;
    const uint32_t lane = threadIdx.x % 32;
    if (r >= rows) return;
    const uint32_t i = r % p.Sq, h = r / p.Sq % p.Hl, b = r / p.Sq / p.Hl % p.B, g = r / p.Sq / p.Hl / p.B;
    const uint16_t* o = reinterpret_cast<const uint16_t*>(p.out.base[g] + b * p.out.b + int64_t(i) * p.out.t + h * p.out.h);
    const uint16_t* d = reinterpret_cast<const uint16_t*>(p.dout.base[g] + b * p.dout.b + int64_t(i) * p.dout.t + h * p.dout.h);
    float s = 0.f;
    for (uint32_t x = lane; x < p.D; x += 32) s = fmaf(to_float<kF>(o[x]), to_float<kF>(d[x]), s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (lane == 0) p.delta[r] = s;
}

// x -> weight P and the slope of the cap; both 0 where the pair is masked.
__device__ __forceinline__ void weight_of(const AttentionParams& p, float dot, float slope, int64_t far, float lse, bool see,
                                          float& w, float& bend) {
    float s = dot * p.scale;
    bend = 1.f;
    if (p.cap != 0.f) {
        const float t = tanhf(s / p.cap);
        s = p.cap * t;
        bend = 1.f - t * t;
    }
    s -= slope * fabsf(float(far));
    w = see ? expf(s - lse) : 0.f;
}

template <Fused kF, int kD>
__global__ void __launch_bounds__(kRowThreads) dq_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kLanes = kD / 32, kRows = kRowThreads / kLanes;
    __shared__ float ks[kOther][kD], vs[kOther][kD];
    __shared__ int32_t kdoc[kOther];
    const uint32_t part = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const uint32_t h = blockIdx.y % p.Hl, b = blockIdx.y / p.Hl % p.B, g = blockIdx.y / p.Hl / p.B;
    const uint32_t kh = h / p.shared;
    const int64_t i = int64_t(blockIdx.x) * kRows + row;
    const bool valid = i < int64_t(p.Sq);
    float q[32], dy[32], acc[32];
    const int64_t at = valid ? i : 0;
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.q.base[g] + b * p.q.b + at * p.q.t + h * p.q.h);
    const uint16_t* dp = reinterpret_cast<const uint16_t*>(p.dout.base[g] + b * p.dout.b + at * p.dout.t + h * p.dout.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) {
        q[d] = valid ? to_float<kF>(qp[part * 32 + d]) : 0.f;
        dy[d] = valid ? to_float<kF>(dp[part * 32 + d]) : 0.f;
        acc[d] = 0.f;
    }
    const int bound = valid ? key_bound(p, b, i) : 0;
    const int32_t doc = valid && p.q_docs ? p.q_docs[int64_t(b) * p.Sq + i] : -1;
    const float slope = p.slopes ? p.slopes[g * p.Hl + h] : 0.f;
    const int64_t pos = i + int64_t(p.Sk) - int64_t(p.Sq);
    const int64_t stat = (int64_t(b) * p.Hl + h) * p.Sq + at;
    const float lse = p.lse[g][stat];
    const float delta = p.delta[int64_t(g) * p.B * p.Hl * p.Sq + stat];
    const uint8_t* kb = p.k.base[g] + b * p.k.b + kh * p.k.h;
    const uint8_t* vb = p.v.base[g] + b * p.v.b + kh * p.v.h;
    for (int j0 = 0; j0 < int(p.Sk); j0 += kOther) {
        if (!__syncthreads_or(j0 < bound)) break;
        for (int x = threadIdx.x; x < kOther * kD; x += kRowThreads) {
            const int j = x / kD, d = x % kD;
            const bool in = j0 + j < int(p.Sk);
            ks[j][d] = in ? to_float<kF>(reinterpret_cast<const uint16_t*>(kb + int64_t(j0 + j) * p.k.t)[d]) : 0.f;
            vs[j][d] = in ? to_float<kF>(reinterpret_cast<const uint16_t*>(vb + int64_t(j0 + j) * p.v.t)[d]) : 0.f;
        }
        if (p.k_docs && threadIdx.x < kOther)
            kdoc[threadIdx.x] = j0 + int(threadIdx.x) < int(p.Sk) ? p.k_docs[int64_t(b) * p.Sk + j0 + threadIdx.x] : -1;
        __syncthreads();
#pragma unroll 4
        for (int j = 0; j < kOther; ++j) {
            float s = 0.f, t = 0.f;
#pragma unroll
            for (int d = 0; d < 32; ++d) {
                s = fmaf(q[d], ks[j][part * 32 + d], s);
                t = fmaf(dy[d], vs[j][part * 32 + d], t);
            }
#pragma unroll
            for (int w = 1; w < kLanes; w <<= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, w);
                t += __shfl_xor_sync(0xffffffffu, t, w);
            }
            const bool see = j0 + j < bound && (!p.k_docs || (doc >= 0 && kdoc[j] == doc));
            if (!see) continue;
            float w, bend;
            weight_of(p, s, slope, pos - (j0 + j), lse, see, w, bend);
            const float dx = w * (t - delta) * bend * p.scale;
#pragma unroll
            for (int d = 0; d < 32; ++d) acc[d] = fmaf(dx, ks[j][part * 32 + d], acc[d]);
        }
        __syncthreads();
    }
    if (!valid) return;
    uint16_t* op = reinterpret_cast<uint16_t*>(p.dq.base[g] + b * p.dq.b + i * p.dq.t + h * p.dq.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) op[part * 32 + d] = to_half<kF>(acc[d]);
}

template <Fused kF, int kD>
__global__ void __launch_bounds__(kRowThreads) dkv_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kLanes = kD / 32, kRows = kRowThreads / kLanes;
    __shared__ float qs[kOther][kD], ds[kOther][kD];
    __shared__ float lses[kOther], deltas[kOther];
    __shared__ int32_t qdoc[kOther];
    __shared__ int bounds[kOther];
    const uint32_t part = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const uint32_t kh = blockIdx.y % p.Hkl, b = blockIdx.y / p.Hkl % p.B, g = blockIdx.y / p.Hkl / p.B;
    const int64_t j = int64_t(blockIdx.x) * kRows + row;
    const bool valid = j < int64_t(p.Sk);
    float k[32], v[32], dk[32], dv[32];
    const int64_t at = valid ? j : 0;
    const uint16_t* kp = reinterpret_cast<const uint16_t*>(p.k.base[g] + b * p.k.b + at * p.k.t + kh * p.k.h);
    const uint16_t* vp = reinterpret_cast<const uint16_t*>(p.v.base[g] + b * p.v.b + at * p.v.t + kh * p.v.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) {
        k[d] = valid ? to_float<kF>(kp[part * 32 + d]) : 0.f;
        v[d] = valid ? to_float<kF>(vp[part * 32 + d]) : 0.f;
        dk[d] = dv[d] = 0.f;
    }
    const int32_t doc = valid && p.k_docs ? p.k_docs[int64_t(b) * p.Sk + j] : -1;
    const int64_t ahead = int64_t(p.Sk) - int64_t(p.Sq);
    for (uint32_t h = kh * p.shared; h < (kh + 1) * p.shared; ++h) {
        const float slope = p.slopes ? p.slopes[g * p.Hl + h] : 0.f;
        const uint8_t* qb = p.q.base[g] + b * p.q.b + h * p.q.h;
        const uint8_t* db = p.dout.base[g] + b * p.dout.b + h * p.dout.h;
        const int64_t stat = (int64_t(b) * p.Hl + h) * p.Sq;
        for (int64_t i0 = 0; i0 < int64_t(p.Sq); i0 += kOther) {
            __syncthreads();
            for (int x = threadIdx.x; x < kOther * kD; x += kRowThreads) {
                const int i = x / kD, d = x % kD;
                const bool in = i0 + i < int64_t(p.Sq);
                qs[i][d] = in ? to_float<kF>(reinterpret_cast<const uint16_t*>(qb + (i0 + i) * p.q.t)[d]) : 0.f;
                ds[i][d] = in ? to_float<kF>(reinterpret_cast<const uint16_t*>(db + (i0 + i) * p.dout.t)[d]) : 0.f;
            }
            if (threadIdx.x < kOther) {
                const int64_t i = i0 + threadIdx.x;
                const bool in = i < int64_t(p.Sq);
                lses[threadIdx.x] = in ? p.lse[g][stat + i] : 0.f;
                deltas[threadIdx.x] = in ? p.delta[int64_t(g) * p.B * p.Hl * p.Sq + stat + i] : 0.f;
                qdoc[threadIdx.x] = in && p.q_docs ? p.q_docs[int64_t(b) * p.Sq + i] : -1;
                bounds[threadIdx.x] = in ? key_bound(p, b, i) : 0;
            }
            __syncthreads();
#pragma unroll 4
            for (int i = 0; i < kOther; ++i) {
                float s = 0.f, t = 0.f;
#pragma unroll
                for (int d = 0; d < 32; ++d) {
                    s = fmaf(k[d], qs[i][part * 32 + d], s);
                    t = fmaf(v[d], ds[i][part * 32 + d], t);
                }
#pragma unroll
                for (int w = 1; w < kLanes; w <<= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, w);
                    t += __shfl_xor_sync(0xffffffffu, t, w);
                }
                const bool see = valid && j < bounds[i] && (!p.k_docs || (doc >= 0 && qdoc[i] == doc));
                if (!see) continue;
                float w, bend;
                weight_of(p, s, slope, i0 + i + ahead - j, lses[i], see, w, bend);
                const float dx = w * (t - deltas[i]) * bend * p.scale;
#pragma unroll
                for (int d = 0; d < 32; ++d) {
                    dv[d] = fmaf(w, ds[i][part * 32 + d], dv[d]);
                    dk[d] = fmaf(dx, qs[i][part * 32 + d], dk[d]);
                }
            }
        }
    }
    if (!valid) return;
    uint16_t* ok = reinterpret_cast<uint16_t*>(p.dk.base[g] + b * p.dk.b + j * p.dk.t + kh * p.dk.h);
    uint16_t* ov = reinterpret_cast<uint16_t*>(p.dv.base[g] + b * p.dv.b + j * p.dv.t + kh * p.dv.h);
#pragma unroll
    for (int d = 0; d < 32; ++d) {
        ok[part * 32 + d] = to_half<kF>(dk[d]);
        ov[part * 32 + d] = to_half<kF>(dv[d]);
    }
}

template <Fused kF, int kD>
cudaError_t launch(const AttentionParams& p, cudaStream_t stream, int* launches) {
    constexpr uint32_t kRows = kRowThreads / (kD / 32);
    const uint64_t rows = uint64_t(p.P) * p.B * p.Hl * p.Sq;
    if (rows > 0) {
        delta_kernel<kF><<<unsigned((rows + 7) / 8), 256, 0, stream>>>(p);
        dq_kernel<kF, kD><<<dim3((p.Sq + kRows - 1) / kRows, p.P * p.B * p.Hl), kRowThreads, 0, stream>>>(p);
        *launches += 2;
    }
    if (p.Sk > 0) {
        dkv_kernel<kF, kD><<<dim3((p.Sk + kRows - 1) / kRows, p.P * p.B * p.Hkl), kRowThreads, 0, stream>>>(p);
        *launches += 1;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_backward(const AttentionParams& p, bool bf16, cudaStream_t stream, int* launches) {
    *launches = 0;
    if (p.D == 64)
        return bf16 ? launch<Fused::kBF16, 64>(p, stream, launches) : launch<Fused::kFP16, 64>(p, stream, launches);
    return bf16 ? launch<Fused::kBF16, 128>(p, stream, launches) : launch<Fused::kFP16, 128>(p, stream, launches);
}

}  // namespace tfu
