// linear_steps.cu -- linear attention token by token: single tokens of generation, and short runs.
//
//   forward: S <- lambda S + k^T v,  out = out_scale q S      reverse: the same with S <- lambda S behind the output
//
// A CTA of 256 threads takes columns of one head's state, all rows of them: a thread four columns of
// every R-th row, in registers for all tokens, so a state is read and written once a call.  lambda S as Fade takes it.
// Rows that the threads of a column hold are summed by shuffles and through shared memory.
// Bound: DRAM, 8 D^2 bytes of state a head and call.  One token of 64 sequences, 32 heads, D = 128: 44 us, 6.0 TB/s (0.89 of
// the copy bandwidth); of one sequence, 8 heads, D = 64: 4.4 us of the GPU, 6 a call.  With few heads a CTA takes 32 columns, so that
// more of them share a state.
#include "device_common.cuh"
#include "linear.h"

namespace tfu {

__device__ unsigned g_linear_steps_status;

namespace {

using namespace dev;

constexpr int kThreadsL = 256, kWarpsL = kThreadsL / 32;

template <Fused kF, int kD, int kLanes>
__global__ void __launch_bounds__(kThreadsL) linear_steps_kernel(const __grid_constant__ LinearPass p) {
    constexpr int kCols = 4 * kLanes, kBlocks = kD / kCols, kGroups = kThreadsL / kLanes, kRows = kD / kGroups;
    __shared__ float rows[2][2][kD];  // by parity of the token: q, k
    __shared__ float cols[2][kCols];  // v
    __shared__ float4 sums[2][kWarpsL][kLanes];
    grid_dependency_wait();
    const uint32_t heads = p.P * p.Hl, block = blockIdx.x % kBlocks, head = blockIdx.x / kBlocks % heads, n = blockIdx.x / kBlocks / heads;
    const uint32_t g = head / p.Hl, h = head % p.Hl, warp = threadIdx.x / 32;
    const uint32_t lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, col = block * kCols + lane * 4;
    const LinearSequence seq = linear_sequence(p, n, &g_linear_steps_status);
    if (p.starts && !seq.ok) return;

    const int64_t at = (int64_t(seq.slot) * heads + head) * (kD * kD);
    float4 s[kRows];
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
        const uint32_t i = group + x * kGroups;
        if (!p.state)
            s[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        else if (p.transposed)
            s[x] = make_float4(p.state[at + col * kD + i], p.state[at + (col + 1) * kD + i], p.state[at + (col + 2) * kD + i],
                               p.state[at + (col + 3) * kD + i]);
        else
            s[x] = *reinterpret_cast<const float4*>(p.state + at + i * kD + col);
    }
    const Fade fade(p.decay[head]);

    // a token's rows: threads 0.. take 8 elements of q, the next of k, the next the CTA's columns of v
    constexpr int kVecs = kD / 8, kVecsV = kCols / 8;
    const uint32_t part = threadIdx.x / kVecs, vec = threadIdx.x % kVecs;
    const bool loads = part < 2 || (part == 2 && vec < kVecsV);
    const GroupView& from = part == 0 ? p.q : part == 1 ? p.k : p.v;
    const uint8_t* src = loads ? from.base[g] + int64_t(seq.b) * from.b + int64_t(h) * from.h + (part == 2 ? block * kCols * 2 : 0) + vec * 16 : nullptr;
    auto row = [&](uint32_t x) { return seq.first + (p.reverse ? seq.len - 1 - x : x); };
    auto fetch = [&](uint32_t x) {
        if (!loads) return;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + row(x) * from.t));
        float* dst = (part < 2 ? rows[x & 1][part] : cols[x & 1]) + vec * 8;
        unpack2<kF>(w.x, dst[0], dst[1]);
        unpack2<kF>(w.y, dst[2], dst[3]);
        unpack2<kF>(w.z, dst[4], dst[5]);
        unpack2<kF>(w.w, dst[6], dst[7]);
    };
    if (seq.len > 0) fetch(0);
    __syncthreads();
    for (uint32_t x = 0; x < seq.len; ++x) {
        const uint32_t now = x & 1;
        const float4 v = *reinterpret_cast<const float4*>(&cols[now][lane * 4]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
            const float q = rows[now][0][group + y * kGroups], k = rows[now][1][group + y * kGroups] * p.kv_scale;
            float4& z = s[y];
            if (!p.reverse) z = make_float4(fade.of(z.x, k * v.x), fade.of(z.y, k * v.y), fade.of(z.z, k * v.z), fade.of(z.w, k * v.w));
            else z = make_float4(fmaf(k, v.x, z.x), fmaf(k, v.y, z.y), fmaf(k, v.z, z.z), fmaf(k, v.w, z.w));
            o.x = fmaf(q, z.x, o.x);
            o.y = fmaf(q, z.y, o.y);
            o.z = fmaf(q, z.z, o.z);
            o.w = fmaf(q, z.w, o.w);
            if (p.reverse) z = make_float4(fade.of(z.x, 0.f), fade.of(z.y, 0.f), fade.of(z.z, 0.f), fade.of(z.w, 0.f));
        }
#pragma unroll
        for (int d = kLanes; d < 32; d *= 2) {
            o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
        }
        if (threadIdx.x % 32 < kLanes) sums[now][warp][lane] = o;
        if (x + 1 < seq.len) fetch(x + 1);
        __syncthreads();
        if (threadIdx.x < kCols / 2) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < kWarpsL; ++w) {
                const float2 y = reinterpret_cast<const float2*>(sums[now][w])[threadIdx.x];
                a += y.x;
                b += y.y;
            }
            uint8_t* dst = p.out.base[g] + int64_t(seq.b) * p.out.b + row(x) * p.out.t + int64_t(h) * p.out.h + block * kCols * 2;
            reinterpret_cast<uint32_t*>(dst)[threadIdx.x] = pack2<kF>(a * p.out_scale, b * p.out_scale);
        }
    }
    if (!p.final_state) return;
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
        const uint32_t i = group + x * kGroups;
        *reinterpret_cast<float4*>(p.final_state + at + i * kD + col) = s[x];
    }
}

template <Fused kF, int kD, int kLanes>
cudaError_t launch(const LinearPass& p, cudaStream_t stream) {
    return launch_overlapped(linear_steps_kernel<kF, kD, kLanes>, p.N * p.P * p.Hl * (kD / (4 * kLanes)), kThreadsL, 0, stream, p);
}

// Few heads: the state's columns over several CTAs.
template <Fused kF, int kD>
cudaError_t launch_split(const LinearPass& p, cudaStream_t stream) {
    return uint64_t(p.N) * p.P * p.Hl < 2 * kAttnSms ? launch<kF, kD, 8>(p, stream) : launch<kF, kD, kD / 4>(p, stream);
}

}  // namespace

cudaError_t launch_linear_steps(const LinearPass& p, bool bf16, cudaStream_t stream) {
    if (p.D == 64) return bf16 ? launch_split<Fused::kBF16, 64>(p, stream) : launch_split<Fused::kFP16, 64>(p, stream);
    return bf16 ? launch_split<Fused::kBF16, 128>(p, stream) : launch_split<Fused::kFP16, 128>(p, stream);
}

cudaError_t read_linear_steps_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_linear_steps_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_linear_steps_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
