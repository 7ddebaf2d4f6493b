// tcgen05.cuh -- the pieces of the 5th-generation tensor core kernels (sm_103a):
// mbarriers with bounded waits, TMA loads, TMEM, tcgen05.mma and its descriptors.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace tfu {
namespace dev {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// One lane of the (converged) warp.  In a branch on this the compiler knows that a single
// thread runs and keeps descriptors and addresses in uniform registers; with a test of the
// lane number instead, four 128 x 128 x 128 products took 4493 cycles beside busy warps, not 2055.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// kCS: acquire at cluster scope (arrivals and copies of the other CTA of a pair).
template <bool kCS = false>
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (kCS) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    }
    return ok != 0;
}
__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// generic-proxy writes to shared memory become visible to TMA and the tensor cores
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

constexpr long long kWaitCycles = 4000000000LL;  // ~2 s at 2 GHz

// Wait for the phase of `bar` with parity `parity`; false if the abort flag is
// raised or the budget runs out (then records bit 0 of *status and raises the flag,
// and also the flag at shared::cluster address `peer_flag` of the other CTA of a
// pair when it is not 0).
template <bool kCS = false>
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                             long long budget = kWaitCycles, uint32_t peer_flag = 0) {
    if (mbar_try_wait<kCS>(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait<kCS>(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > budget) {
                atomicOr(status, 1u);
                *abort_flag = 1;
                if (peer_flag) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_flag), "r"(1u) : "memory");
                return false;
            }
        }
    }
}

// The same without the abort flag (draining after an abort): bounded only.
template <bool kCS = false>
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait<kCS>(bar, parity)) {
        if (clock64() - t0 > kWaitCycles) return;
    }
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_load_2d(uint32_t smem_dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// ---------------------------------------------------------------- TMEM
__device__ __forceinline__ void tmem_alloc(uint32_t smem_result, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_result), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive 32-bit columns of this thread's TMEM lane (warp-collective: the
// warp is reconverged first).
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// one column, and four of them (waited for)
__device__ __forceinline__ void tc_st1(uint32_t taddr, uint32_t r) {
    __syncwarp();
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}
__device__ __forceinline__ void tc_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- MMA
// Instruction descriptor of tcgen05.mma kind::f16: D fp32 (bits 4-5 = 1), A and B
// bf16 (bits 7-9, 10-12 = 1) or fp16 (0), A K-major (bit 15 = 0), B K-major (bit
// 16 = 0) or MN-major (1), N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t f16_idesc(bool bf16, uint32_t m, uint32_t n, bool b_mn_major) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) | ((n >> 3) << 17) |
           ((m >> 4) << 24);
}

constexpr uint32_t kSwizzleRow = 128;  // bytes of a row in the 128-byte swizzle

// Shared-memory matrix descriptor of an operand tile whose rows are 128 bytes with
// the 128-byte swizzle, 8-row groups 1024 bytes apart: start address >> 4 (bits
// 0-13), leading byte offset >> 4 at bits 16-29, stride byte offset (1024 >> 4) at
// bits 32-45, descriptor version 1 at bits 46-47, base offset 0 (tiles are aligned
// to the swizzle pattern), swizzle mode 2 (128-byte) at bits 61-63.
//  K-major (rows = M or N, 64 16-bit K elements a row): the leading offset is
//    unused; a K step of 16 elements advances the start by 32 bytes.
//  MN-major (rows = K, 64 M or N elements a row): the leading offset is the
//    distance of the next 64 M or N elements; a K step of 16 rows advances the
//    start by 2048 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t smem_addr, uint32_t leading_bytes = 16) {
    constexpr uint64_t kMode = 2;
    return uint64_t((smem_addr & 0x3FFFFu) >> 4) | (uint64_t(leading_bytes >> 4) << 16) |
           (uint64_t((8 * kSwizzleRow) >> 4) << 32) | (uint64_t(1) << 46) | (kMode << 61);
}

// D[tmem] (+)= A[smem] * B[smem]^T, one K = 16 step
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The descriptor of sw128_desc in halves: everything but the low word is the same for every
// tile, and an offset inside a tile is an addition to the low word.  One thread issues all
// products of a CTA while its other warps keep the schedulers busy, so what it
// computes between two of them counts.
constexpr uint32_t kDescHigh = ((8 * kSwizzleRow) >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr, uint32_t leading_bytes = 16) {
    return ((smem_addr & 0x3FFFFu) >> 4) | (leading_bytes >> 4) << 16;
}
template <bool kAccumulate>
__device__ __forceinline__ void tc_mma_low(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_low), "r"(b_low), "r"(idesc), "n"(kDescHigh), "n"(kAccumulate ? 1 : 0)
        : "memory");
}
// A in TMEM: lane = row, a 32-bit column holds two K elements.
__device__ __forceinline__ void tc_mma_ts_low(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_low), "r"(idesc), "n"(kDescHigh), "r"(accumulate)
        : "memory");
}
// D = A B^T over kD elements of K: both operands K-major, 64 elements a half, halves
// kHalfA and kHalfB bytes apart.
template <int kD, uint32_t kHalfA, uint32_t kHalfB>
__device__ __forceinline__ void tc_product(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc) {
    tc_mma_low<false>(d_tmem, a_low, b_low, idesc);
#pragma unroll
    for (uint32_t kk = 1; kk < kD / 16; ++kk)
        tc_mma_low<true>(d_tmem, a_low + ((kk / 4 * kHalfA + kk % 4 * 32) >> 4), b_low + ((kk / 4 * kHalfB + kk % 4 * 32) >> 4),
                         idesc);
}
// D (+)= A B with A from TMEM (kK elements of K, 32-bit columns of two), B MN-major.
template <int kK>
__device__ __forceinline__ void tc_product_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc,
                                              uint32_t accumulate) {
    tc_mma_ts_low(d_tmem, a_tmem, b_low, idesc, accumulate);
#pragma unroll
    for (uint32_t kk = 1; kk < kK / 16; ++kk) tc_mma_ts_low(d_tmem, a_tmem + kk * 8, b_low + kk * (2048 >> 4), idesc, 1u);
}

// Arrive once on `bar` when every tcgen05 operation this thread issued so far completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

}  // namespace dev
}  // namespace tfu
