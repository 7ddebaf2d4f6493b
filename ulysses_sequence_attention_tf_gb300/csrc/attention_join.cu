// attention_join.cu -- joins the parts of attention units that were cut along the other side
// (Split in attention.h): a warp a row, parts in order, so that the result is always the same.
#include "attention_common.cuh"

namespace tfu {

namespace {

using namespace dev;

constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 32;

// kPer values of a lane's row as 16-bit values
template <Fused kF, int kPer>
__device__ __forceinline__ void store_lane(uint8_t* row, uint32_t lane, const float (&v)[kPer]) {
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(row + lane * 8) = make_uint2(pack2<kF>(v[0], v[1]), pack2<kF>(v[2], v[3]));
    else
        *reinterpret_cast<uint32_t*>(row + lane * 4) = pack2<kF>(v[0], v[1]);
}
template <int kPer>
__device__ __forceinline__ void load_lane(float (&v)[kPer], const float* row, uint32_t lane) {
    if constexpr (kPer == 4)
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(row + lane * 4);
    else
        *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(row + lane * 2);
}

// O of every part relative to its own reference: o = sum o_c 2^(m_c - m) / sum l_c 2^(m_c - m).
template <Fused kF, int kD>
__global__ void __launch_bounds__(kJoinThreads) join_forward_kernel(const __grid_constant__ ForwardParams fp) {
    constexpr int kPer = kD / 32;
    grid_dependency_wait();
    const AttentionParams& p = fp.a;
    const uint32_t lane = threadIdx.x % 32, at = blockIdx.x * kJoinRows + threadIdx.x / 32;
    const uint32_t cut = at / kAttnPair, r = at % kAttnPair;
    uint32_t u = fp.split.whole + cut;
    const uint32_t i = u % fp.q_tiles * kAttnPair + r;
    u /= fp.q_tiles;
    const uint32_t h = u % p.Hl, b = u / p.Hl % p.B, g = u / p.Hl / p.B;
    if (i >= p.Sq) return;
    const int64_t row0 = int64_t(cut) * fp.split.parts * kAttnPair + r;
    float top = -INFINITY;
    for (uint32_t c = 0; c < fp.split.parts; ++c) top = fmaxf(top, fp.split.stat[row0 + int64_t(c) * kAttnPair].x);
    float l = 0.f, o[kPer] = {};
    for (uint32_t c = 0; c < fp.split.parts; ++c) {
        const int64_t row = row0 + int64_t(c) * kAttnPair;
        const float2 st = fp.split.stat[row];
        float v[kPer];
        load_lane(v, fp.split.part + row * kD, lane);
        const float f = st.x == -INFINITY ? 0.f * st.y : ex2(st.x - top);  // a part without weight, or with NaN
        l = fmaf(f, st.y, l);
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] = fmaf(f, v[x], o[x]);
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] *= inv;
    store_lane<kF>(p.out.base[g] + int64_t(b) * p.out.b + int64_t(i) * p.out.t + int64_t(h) * p.out.h, lane, o);
    if (lane == 0 && p.lse[g])
        p.lse[g][(int64_t(b) * p.Hl + h) * p.Sq + i] = (top == -INFINITY ? 0.f : top * kLn2) + logf(l);
}

// dQ = scale * (sum of the parts' sums - e * sum of their W), e the sum of what they lack of delta.
template <Fused kF, int kD>
__global__ void __launch_bounds__(kJoinThreads) join_dq_kernel(const __grid_constant__ AttentionParams p, const Split s, uint32_t row_tiles,
                                                               int64_t rows_in_parts) {
    constexpr int kPer = kD / 32;
    grid_dependency_wait();
    const uint32_t lane = threadIdx.x % 32, at = blockIdx.x * kJoinRows + threadIdx.x / 32;
    const uint32_t cut = at / kAttnRows, r = at % kAttnRows;
    uint32_t u = s.whole + cut;
    const uint32_t i = u % row_tiles * kAttnRows + r;
    u /= row_tiles;
    const uint32_t h = u % p.Hl, b = u / p.Hl % p.B, g = u / p.Hl / p.B;
    if (i >= p.Sq) return;
    float o[kPer] = {}, w[kPer] = {}, e = 0.f;
    for (uint32_t c = 0; c < s.parts; ++c) {
        const int64_t row = (int64_t(cut) * s.parts + c) * kAttnRows + r;
        float v[kPer];
        e += s.stat[row].x;
        load_lane(v, s.part + row * kD, lane);
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] += v[x];
        load_lane(v, s.part + (rows_in_parts + row) * kD, lane);
#pragma unroll
        for (int x = 0; x < kPer; ++x) w[x] += v[x];
    }
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = fmaf(-e, w[x], o[x]) * p.scale;
    store_lane<kF>(p.dq.base[g] + int64_t(b) * p.dq.b + int64_t(i) * p.dq.t + int64_t(h) * p.dq.h, lane, o);
    if (lane == 0) p.delta[(int64_t(u) * p.Sq) + i] += e;
}

// dK, dV: the sum of the parts times `factor`.
template <Fused kF, int kD>
__global__ void __launch_bounds__(kJoinThreads) join_gradient_kernel(const __grid_constant__ GroupView out, const float* part,
                                                                     const Split s, float factor, uint32_t row_tiles, uint32_t rows,
                                                                     uint32_t heads, uint32_t B) {
    constexpr int kPer = kD / 32;
    grid_dependency_wait();
    const uint32_t lane = threadIdx.x % 32, at = blockIdx.x * kJoinRows + threadIdx.x / 32;
    const uint32_t cut = at / kAttnRows, r = at % kAttnRows;
    uint32_t u = s.whole + cut;
    const uint32_t i = u % row_tiles * kAttnRows + r;
    u /= row_tiles;
    const uint32_t h = u % heads, b = u / heads % B, g = u / heads / B;
    if (i >= rows) return;
    float o[kPer] = {};
    for (uint32_t c = 0; c < s.parts; ++c) {
        float v[kPer];
        load_lane(v, part + ((int64_t(cut) * s.parts + c) * kAttnRows + r) * kD, lane);
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] += v[x];
    }
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] *= factor;
    store_lane<kF>(out.base[g] + int64_t(b) * out.b + int64_t(i) * out.t + int64_t(h) * out.h, lane, o);
}

template <Fused kF, int kD>
cudaError_t forward(const ForwardParams& p, cudaStream_t stream) {
    const uint32_t cut = p.q_tiles * p.a.P * p.a.B * p.a.Hl - p.split.whole;
    return launch_overlapped(join_forward_kernel<kF, kD>, cut * kAttnPair / kJoinRows, kJoinThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_join_forward(const ForwardParams& p, bool bf16, cudaStream_t stream) {
    if (p.a.D == 64) return bf16 ? forward<Fused::kBF16, 64>(p, stream) : forward<Fused::kFP16, 64>(p, stream);
    return bf16 ? forward<Fused::kBF16, 128>(p, stream) : forward<Fused::kFP16, 128>(p, stream);
}

cudaError_t launch_join_dq(const BackwardParams& p, bool bf16, cudaStream_t stream) {
    const AttentionParams& a = p.a;
    const uint32_t cut = p.q_tiles * a.P * a.B * a.Hl - p.dq_split.whole, grid = cut * kAttnRows / kJoinRows;
    auto kernel = a.D == 64 ? (bf16 ? join_dq_kernel<Fused::kBF16, 64> : join_dq_kernel<Fused::kFP16, 64>)
                            : (bf16 ? join_dq_kernel<Fused::kBF16, 128> : join_dq_kernel<Fused::kFP16, 128>);
    return launch_overlapped(kernel, grid, kJoinThreads, 0, stream, a, p.dq_split, p.q_tiles, int64_t(cut) * p.dq_split.parts * kAttnRows);
}

cudaError_t launch_join_gradient(const AttentionParams& p, const Split& s, const GroupView& out, const float* part, float factor,
                                 uint32_t row_tiles, uint32_t rows, uint32_t heads, bool bf16, cudaStream_t stream) {
    const uint32_t cut = row_tiles * p.P * p.B * heads - s.whole, grid = cut * kAttnRows / kJoinRows;
    auto kernel = p.D == 64 ? (bf16 ? join_gradient_kernel<Fused::kBF16, 64> : join_gradient_kernel<Fused::kFP16, 64>)
                            : (bf16 ? join_gradient_kernel<Fused::kBF16, 128> : join_gradient_kernel<Fused::kFP16, 128>);
    return launch_overlapped(kernel, grid, kJoinThreads, 0, stream, out, part, s, factor, row_tiles, rows, heads, p.B);
}

}  // namespace tfu
