// attention_plan.cu -- which tiles of queries and keys can see one another when
// there are documents, and the tensor maps of the head groups.
//
// A tile pair may be visible when the ranges of the two tiles' document numbers
// (padding left out) meet and the causal bound reaches the keys; it is wholly
// visible when both tiles hold one and the same document and no padding, and the
// bound of every row covers it.  Numbers need not be ordered: the ranges only
// decide what is skipped and where the element mask can be left out.
#include "attention_common.cuh"
#include "attention_plan.h"

namespace tfu {

namespace {

using namespace dev;

constexpr int kPlanThreads = 256;

struct DocRange {
    int lo, hi;   // of the numbers >= 0; lo > hi: none
    bool hole;    // padding, or a place behind the end
};

// The range of kN numbers of each lane (-1: padding, INT32_MIN: none).
template <int kN>
__device__ __forceinline__ DocRange warp_range(const int32_t (&v)[kN]) {
    DocRange r{INT32_MAX, -1, false};
    bool hole = false;
#pragma unroll
    for (int x = 0; x < kN; ++x) {
        if (v[x] >= 0) {
            r.lo = min(r.lo, v[x]);
            r.hi = max(r.hi, v[x]);
        } else {
            hole |= v[x] != INT32_MIN;
        }
    }
    r.lo = __reduce_min_sync(0xffffffffu, r.lo);
    r.hi = __reduce_max_sync(0xffffffffu, r.hi);
    r.hole = __any_sync(0xffffffffu, hole);
    return r;
}

// One CTA per row tile and batch row.  kRowsAreKeys: the row tiles are keys (of 128
// rows), the column tiles queries.
template <bool kRowsAreKeys>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ AttentionParams p, uint32_t* plan,
                                                             uint32_t rows_per_tile, uint32_t row_tiles, uint32_t words) {
    constexpr int kWarps = kPlanThreads / 32, kAhead = 4;  // a warp takes kAhead neighbours at a time
    static_assert(kWarps * kAhead == 32, "the CTA covers a word at a time");
    __shared__ DocRange row[kWarps];
    __shared__ uint32_t bits[2];
    grid_dependency_wait();
    const uint32_t rt = blockIdx.x % row_tiles, b = blockIdx.x / row_tiles, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rows = int(kRowsAreKeys ? p.Sk : p.Sq), cols = int(kRowsAreKeys ? p.Sq : p.Sk);
    const int32_t* row_docs = (kRowsAreKeys ? p.k_docs : p.q_docs) + int64_t(b) * rows;
    const int32_t* col_docs = (kRowsAreKeys ? p.q_docs : p.k_docs) + int64_t(b) * cols;
    const int r0 = int(rt * rows_per_tile), r1 = min(rows, r0 + int(rows_per_tile));
    // the row tile's numbers, 32 a warp, and the first word's column tiles at the same time
    int32_t own[1], v[kAhead][4];
    const int mine = r0 + int(threadIdx.x);
    own[0] = mine < r1 ? max(row_docs[mine], -1) : INT32_MIN;
    auto load = [&](uint32_t w) {
        const int t0 = int(w) * 32 + int(warp) * kAhead;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int at = (t0 + k) * int(kAttnRows) + x * 32 + int(lane);
                v[k][x] = at < cols ? max(col_docs[at], -1) : -1;
            }
    };
    load(0);
    const DocRange part = warp_range(own);
    if (lane == 0) row[warp] = part;
    __syncthreads();
    DocRange rr = row[0];
#pragma unroll
    for (int x = 1; x < kWarps; ++x) {
        rr.lo = min(rr.lo, row[x].lo);
        rr.hi = max(rr.hi, row[x].hi);
        rr.hole |= row[x].hole;
    }
    uint32_t* out = plan + size_t(blockIdx.x) * 2 * words;
    for (uint32_t w = 0; w < words; ++w) {
        __syncthreads();
        if (threadIdx.x < 2) bits[threadIdx.x] = 0;
        __syncthreads();
        const int t0 = int(w) * 32 + int(warp) * kAhead;
        DocRange c[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) c[k] = warp_range(v[k]);
        if (w + 1 < words) load(w + 1);
        uint32_t some = 0, all = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c0 = (t0 + k) * int(kAttnRows), c1 = min(cols, c0 + int(kAttnRows));
            if (c0 >= cols) break;
            // the last query of the pair reaches furthest, its first one least
            const int far = key_bound(p, b, (kRowsAreKeys ? c1 : r1) - 1), near = key_bound(p, b, kRowsAreKeys ? c0 : r0);
            const int k0 = kRowsAreKeys ? r0 : c0, k1 = kRowsAreKeys ? r0 + int(kAttnRows) : c0 + int(kAttnRows);
            const bool meet = rr.lo <= c[k].hi && c[k].lo <= rr.hi && rr.hi >= 0 && c[k].hi >= 0 && k0 < far;
            const bool whole = meet && rr.lo == rr.hi && c[k].lo == c[k].hi && !rr.hole && !c[k].hole && k1 <= near;
            some |= uint32_t(meet) << ((t0 + k) % 32);
            all |= uint32_t(whole) << ((t0 + k) % 32);
        }
        if (lane == 0 && some) {
            atomicOr(&bits[0], some);
            atomicOr(&bits[1], all);
        }
        __syncthreads();
        if (threadIdx.x < 2) out[threadIdx.x * words + w] = bits[threadIdx.x];
    }
}

}  // namespace

cudaError_t launch_plan(const AttentionParams& p, uint32_t* plan, bool rows_are_keys, uint32_t rows_per_tile,
                        cudaStream_t stream) {
    const TilePlan t = tile_plan(rows_are_keys ? p.Sk : p.Sq, rows_per_tile, rows_are_keys ? p.Sq : p.Sk);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(t.row_tiles * p.B);  // below 2^31 units
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return rows_are_keys ? cudaLaunchKernelEx(&cfg, plan_kernel<true>, p, plan, rows_per_tile, t.row_tiles, t.words)
                         : cudaLaunchKernelEx(&cfg, plan_kernel<false>, p, plan, rows_per_tile, t.row_tiles, t.words);
}

}  // namespace tfu
