// kv_common.cuh -- what the kernels of the attention over the paged cache share.
#pragma once

#include "attention_common.cuh"
#include "kv_cache.h"

namespace tfu {
namespace dev {

// What a CTA needs of its sequence; ok = false: nothing to do (flagged if out of range).
struct Sequence {
    int64_t s0;
    int tokens, len, chunks;
    bool ok;
};
__device__ __forceinline__ Sequence sequence_of(const KvAttendParams& p, uint32_t n, unsigned* status) {
    const KvCache& c = p.c;
    const int64_t s0 = c.starts[n], s1 = c.starts[n + 1], len = c.lens[n], tokens = s1 - s0;
    Sequence s{s0, int(tokens), int(len), 0, false};
    if (s0 < 0 || tokens < 0 || s1 > int64_t(p.T) || len < tokens || len > int64_t(p.max_len) || tokens > int64_t(p.max_tokens)) {
        if (threadIdx.x == 0) atomicOr(status, 1u);
        return s;
    }
    s.ok = tokens > 0;
    s.chunks = int((uint32_t(len) + p.chunk - 1) / p.chunk);
    return s;
}

__device__ __forceinline__ uint32_t to_f16x2(uint32_t e4m3_pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(e4m3_pair)));
    return h;
}

// The power of two that puts a row's largest magnitude into [2^14, 2^15): Q times it is
// exact in fp16 but for values 2^28 below the largest.  1 for a row of zeros or one that is not finite.
__device__ __forceinline__ float f16_factor(float most) {
    const int e = 14 - (int(__float_as_uint(most) >> 23) - 127);
    return most == 0.f || !(most <= kFltMax) ? 1.0f : __uint_as_float(uint32_t(min(e, 100) + 127) << 23);
}

// 16 bytes into shared memory as they come; zeros if not `there` (then nothing is read).
__device__ __forceinline__ void copy_async16(uint32_t smem, const void* global, bool there = true) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(global), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
}  // namespace dev
}  // namespace tfu
