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

__device__ __forceinline__ DocRange warp_range(const int32_t* docs, int first, int count, int end) {
    DocRange r{INT32_MAX, -1, false};
    bool hole = false;
    for (int i = threadIdx.x % 32; i < count; i += 32) {
        const int d = first + i < end ? docs[first + i] : -1;
        if (d >= 0) {
            r.lo = min(r.lo, d);
            r.hi = max(r.hi, d);
        } else {
            hole = true;
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
    __shared__ DocRange row;
    __shared__ uint32_t bits[2];
    grid_dependency_wait();
    const uint32_t rt = blockIdx.x % row_tiles, b = blockIdx.x / row_tiles, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rows = int(kRowsAreKeys ? p.Sk : p.Sq), cols = int(kRowsAreKeys ? p.Sq : p.Sk);
    const int32_t* row_docs = (kRowsAreKeys ? p.k_docs : p.q_docs) + int64_t(b) * rows;
    const int32_t* col_docs = (kRowsAreKeys ? p.q_docs : p.k_docs) + int64_t(b) * cols;
    const int r0 = int(rt * rows_per_tile), r1 = min(rows, r0 + int(rows_per_tile));
    if (warp == 0) {
        const DocRange r = warp_range(row_docs, r0, r1 - r0, rows);
        if (lane == 0) row = r;
    }
    __syncthreads();
    const DocRange rr = row;
    uint32_t* out = plan + size_t(blockIdx.x) * 2 * words;
    constexpr int kWarps = kPlanThreads / 32, kAhead = 4;  // a warp takes kAhead neighbours at a time
    static_assert(kWarps * kAhead == 32, "the CTA covers a word at a time");
    for (uint32_t w = 0; w < words; ++w) {
        __syncthreads();
        if (threadIdx.x < 2) bits[threadIdx.x] = 0;
        __syncthreads();
        int lo[kAhead], hi[kAhead];
        bool hole[kAhead];
        const int t0 = int(w) * 32 + int(warp) * kAhead;
        int32_t v[kAhead][4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int at = (t0 + k) * int(kAttnRows) + x * 32 + int(lane);
                v[k][x] = at < cols ? col_docs[at] : -1;
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            lo[k] = INT32_MAX;
            hi[k] = -1;
            bool h = false;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                h |= v[k][x] < 0;
                if (v[k][x] >= 0) {
                    lo[k] = min(lo[k], v[k][x]);
                    hi[k] = max(hi[k], v[k][x]);
                }
            }
            lo[k] = __reduce_min_sync(0xffffffffu, lo[k]);
            hi[k] = __reduce_max_sync(0xffffffffu, hi[k]);
            hole[k] = __any_sync(0xffffffffu, h);
        }
        uint32_t some = 0, all = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c0 = (t0 + k) * int(kAttnRows), c1 = min(cols, c0 + int(kAttnRows));
            if (c0 >= cols) break;
            // the last query of the pair reaches furthest, its first one least
            const int far = key_bound(p, b, (kRowsAreKeys ? c1 : r1) - 1), near = key_bound(p, b, kRowsAreKeys ? c0 : r0);
            const int k0 = kRowsAreKeys ? r0 : c0, k1 = kRowsAreKeys ? r0 + int(kAttnRows) : c0 + int(kAttnRows);
            const bool meet = rr.lo <= hi[k] && lo[k] <= rr.hi && rr.hi >= 0 && hi[k] >= 0 && k0 < far;
            const bool whole = meet && rr.lo == rr.hi && lo[k] == hi[k] && !rr.hole && !hole[k] && k1 <= near;
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
