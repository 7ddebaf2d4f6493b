// attention_backward.cu -- the gradient of the attention over the head groups, on the
// 5th-generation tensor cores.
//
// With the weights P_ij = e^(z_ij - lse_i) recomputed from Q, K and the saved
// log-sum-exp, and delta_i = sum_j P_ij dP_ij:
//   dP_ij = dO_i . V_j                          dV_j = sum_i P_ij dO_i
//   dx_ij = P_ij (dP_ij - delta_i) bend_ij      bend = 1 - tanh^2(x / cap) where scores are capped, else 1
//   dQ_i  = scale * sum_j dx_ij K_j             dK_j = scale * sum_i dx_ij Q_i
//
// Two kernels: dq_kernel owns query rows and sums over the keys, dkv_kernel owns
// key rows and sums over the queries of every head that shares the key head.  S and
// dP are computed in both, which spares the read-modify-write of dQ in memory: no
// atomics, so the same inputs give the same bits.
//
// delta_i = sum_d dO_id O_id, but O is given rounded (by up to 2^-8 in bf16), and what that leaves out, e_i,
// counts times P_ij against dx.  Modelled in 64 bits with bf16 roundings, one row in a hundred was off by 2.4 % with a
// distance bias of 0.63, by 31 % with 2, and by 14 % where keys and values have means as large as their
// spread, instead of 0.3 to 0.5 %; rows of three keys by 2 %.  dq_kernel therefore takes d0 = dO . O
// only as a first value, sums what is missing,
//   e_i = sum_j P_ij (dP_ij - d0_i) = delta_i - d0_i      (sum_j P_ij = 1), and
//   dQ_i = scale * (sum_j P_ij (dP_ij - d0_i) bend_ij K_j - e_i * sum_j P_ij bend_ij K_j):
// one product more, whose roundings count only times e_i.  It hands d0 + e to dkv_kernel.
// Eight products are executed where five would do.
//
// fp16: dx of a long row is about |dO| |V| / Sk and would fall into the subnormals, so it is kept times a power of
// two: |dx| <= P |dO_i| 2 max_j |V_j|, of which sizes_kernel finds the parts in front, and lift puts that
// bound below 2^15.  dq_kernel takes a factor for each row, dkv_kernel, which sums over them, one for its key head.
// P is kept times 2^8 for the same reason.
//
// P and dx are rounded to the I/O type as operands (one MMA takes A and B of one type; a second operand
// for the rest would cost a product more for each): with bf16 that adds about 0.0017 of the norm to
// gradients whose own rounding is as large.
//
// Bound: the products, and the rows' threads beside them that wait for TMEM.  8192 tokens, 5 heads, D = 128, bf16:
//  * dQ 245 us, the matrix pipe busy 62 % of the cycles.  The rows' P, P K and S of the next tile wait for one
//    another: without the product P K 215 us, with two buffers for S besides (no room at D = 128 with W) 190.
//  * dK and dV 273 us and 54 %: TMEM holds dK, dV and two pairs of S and dP of 64 queries, whose products take
//    391 cycles where 256 would be ideal; 128 queries a step do not fit.  fp16 290: the factor costs registers.
// D = 64 with bias, 24 causal heads of 6001 tokens: 267 and 369 us, pipe busy 37 and 26 %, issue slots 51 and 53 %: the
// rows' threads.  Spills: dkv_kernel 40 to 184 bytes, 3 % of its instructions at D = 128, 8 % with bias; the capped
// dq_kernel 64 to 92, 1 %.  Earlier forms (16380 tokens, 5 heads, before P K): 8 row warps 2.88 ms, 16 2.72; rings
// of their own for K and V in dQ 2.46; units cut along the other side 2.09; with P K 2.42.
#include "attention_common.cuh"
#include "attention_order.h"
#include "attention_plan.h"

namespace tfu {

__device__ unsigned g_attention_backward_status;

namespace {

using namespace dev;

constexpr int kThreadsB = 640;  // 16 warps for the rows, 4 for the rest

// compile-time switches of the inner loops
template <bool kV>
struct Bool {
    static constexpr bool value = kV;
};
constexpr uint32_t kHalfTile = kAttnRows * kSwizzleRow;  // 128 rows of 64 elements: 16 KiB

__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return bounded_wait(bar, parity, abort_flag, &g_attention_backward_status);
}

// What of a pair is seen (bits 0 and 1): NaN in padding must not reach a product as a factor of a weight 0.
__device__ __forceinline__ uint64_t keep_pair(uint64_t v, uint32_t see) {
    float a, b;
    f2_unpack(v, a, b);
    return f2_pack(see & 1u ? a : 0.f, see & 2u ? b : 0.f);
}

// Arguments of the weights of a row's scores, for pairs of them: log2 e z - lse2, where `add`
// holds -lse2 and what the bias gives; and (capped) the slope 1 - tanh^2 of each.
template <bool kCap>
struct ToWeight {
    uint64_t c2, x2, z2;  // log2 e scale; scale / cap, log2 e cap
    bool near;            // |x| of every score of the warp is within the polynomial
    template <int kN>
    __device__ __forceinline__ ToWeight(const AttentionParams& p, const float (&s)[kN]) {
        const float c = p.scale * kLog2e, to_x = kCap ? p.scale / p.cap : 0.f, to_z = p.cap * kLog2e;
        c2 = f2_pack(c, c);
        x2 = f2_pack(to_x, to_x);
        z2 = f2_pack(to_z, to_z);
        near = true;
        if constexpr (kCap) {
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < kN; ++i) most = fmaxf(fabsf(s[i]), most);
            near = __all_sync(0xffffffffu, most * fabsf(to_x) <= kTanhNear);
        }
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t s, uint64_t add, uint64_t& bend) const {
        if constexpr (!kCap) return f2_fma(s, c2, add);
        uint64_t t = f2_mul(s, x2);
        if (near) {
            t = f2_mul(t, tanh_over_x(f2_mul(t, t)));
        } else {
            float a, b;
            f2_unpack(t, a, b);
            t = f2_pack(tanh_wide(a), tanh_wide(b));
        }
        const uint64_t one = f2_pack(1.f, 1.f);
        bend = f2_sub(one, f2_mul(t, t));
        return f2_fma(t, z2, add);
    }
};

// 16-bit pairs of kN values over TMEM columns from taddr
template <Fused kF, int kN>
__device__ __forceinline__ void store_row16(uint32_t taddr, const float (&v)[kN]) {
#pragma unroll
    for (int x = 0; x < kN / 32; ++x) {
        uint32_t w[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) w[y] = pack2<kF>(v[x * 32 + 2 * y], v[x * 32 + 2 * y + 1]);
        tc_st16(taddr + x * 16, w);
    }
}

// kCols accumulator columns times `factor` to a row of 16-bit values
template <Fused kF, int kCols>
__device__ __forceinline__ void write_row(uint32_t taddr, bool any, bool valid, float factor, uint8_t* dst) {
#pragma unroll 1
    for (int x = 0; x < kCols; x += 32) {
        uint32_t r[32];
        if (any) {
            tc_ld32(taddr + x, r);
            tc_wait_ld();
            tc_landed(r);
        } else {
#pragma unroll
            for (int y = 0; y < 32; ++y) r[y] = 0;
        }
#pragma unroll
        for (int y = 0; y < 32; y += 8) {
            uint4 w;
            uint32_t* o = &w.x;
#pragma unroll
            for (int z = 0; z < 4; ++z)
                o[z] = pack2<kF>(__uint_as_float(r[y + 2 * z]) * factor, __uint_as_float(r[y + 2 * z + 1]) * factor);
            if (valid) *reinterpret_cast<uint4*>(dst + (x + y) * 2) = w;
        }
    }
}

// 32 columns of dQ: factor * (back * sums - e * weights)
template <Fused kF>
__device__ __forceinline__ void write_dq(uint32_t sums, uint32_t weights, bool any, bool valid, float back, float e, float factor,
                                         uint8_t* dst) {
    float a[32] = {}, w[32] = {};
    if (any) {
        load_row<32>(sums, a);
        load_row<32>(weights, w);
    }
#pragma unroll
    for (int x = 0; x < 32; x += 8) {
        uint32_t o[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
            o[z] = pack2<kF>(fmaf(-e, w[x + 2 * z], a[x + 2 * z] * back) * factor,
                             fmaf(-e, w[x + 2 * z + 1], a[x + 2 * z + 1] * back) * factor);
        if (valid) *reinterpret_cast<uint4*>(dst + x * 2) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// accumulator columns times `factor` in fp32, for a part of a unit
template <int kCols>
__device__ __forceinline__ void write_sums(uint32_t taddr, float factor, float* dst) {
#pragma unroll 1
    for (int x = 0; x < kCols; x += 32) {
        uint32_t r[32];
        tc_ld32(taddr + x, r);
        tc_wait_ld();
        tc_landed(r);
#pragma unroll
        for (int y = 0; y < 32; ++y) r[y] = __float_as_uint(__uint_as_float(r[y]) * factor);
#pragma unroll
        for (int y = 0; y < 32; y += 4) *reinterpret_cast<uint4*>(dst + x + y) = make_uint4(r[y], r[y + 1], r[y + 2], r[y + 3]);
    }
}

// sum_d a_d b_d of two 16-bit rows; squares: sum_d a_d^2
template <Fused kF, int kD>
__device__ __forceinline__ float row_dot(const uint8_t* a, const uint8_t* b, float& squares) {
    float s = 0.f, t = 0.f;
#pragma unroll 4
    for (int x = 0; x < kD / 8; ++x) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(a) + x), v = __ldg(reinterpret_cast<const uint4*>(b) + x);
        const uint32_t* uw = &u.x;
        const uint32_t* vw = &v.x;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            float a0, a1, b0, b1;
            unpack2<kF>(uw[y], a0, a1);
            unpack2<kF>(vw[y], b0, b1);
            s = fmaf(a0, b0, s);
            s = fmaf(a1, b1, s);
            t = fmaf(a0, a0, t);
            t = fmaf(a1, a1, t);
        }
    }
    squares = t;
    return s;
}

// ---------------------------------------------------------------- fp16: sizes
// The largest |dO_i|^2 of every query row tile of a head, then the largest |V_j|^2 of every key
// tile of a key head; padding left out.  A CTA a tile, D / 8 lanes a row.
constexpr int kSizeThreads = 256;
template <int kD>
__global__ void __launch_bounds__(kSizeThreads) sizes_kernel(const __grid_constant__ BackwardParams bp) {
    constexpr uint32_t kLanes = kD / 8, kPass = kSizeThreads / kLanes;
    const AttentionParams& p = bp.a;
    __shared__ float most_of[kSizeThreads / 32];
    grid_dependency_wait();
    const uint32_t q_units = bp.q_tiles * p.P * p.B * p.Hl;
    const bool keys = blockIdx.x >= q_units;
    const uint32_t tiles = keys ? bp.k_tiles : bp.q_tiles, heads = keys ? p.Hkl : p.Hl, tokens = keys ? p.Sk : p.Sq;
    uint32_t u = keys ? blockIdx.x - q_units : blockIdx.x;
    const uint32_t row0 = u % tiles * kAttnRows;
    u /= tiles;
    const uint32_t h = u % heads, b = u / heads % p.B, g = u / heads / p.B;
    const GroupView& view = keys ? p.v : p.dout;
    const int32_t* docs = keys ? p.k_docs : p.q_docs;
    const uint8_t* base = view.base[g] + int64_t(b) * view.b + int64_t(h) * view.h + threadIdx.x % kLanes * 16;
    float most = 0.f;
#pragma unroll
    for (uint32_t x = 0; x < kAttnRows / kPass; ++x) {
        const uint32_t i = row0 + x * kPass + threadIdx.x / kLanes;
        float t = 0.f;
        if (i < tokens && !(docs && docs[int64_t(b) * tokens + i] < 0)) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(base + int64_t(i) * view.t));
            const uint32_t* v = &w.x;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                float a0, a1;
                unpack2<Fused::kFP16>(v[y], a0, a1);
                t = fmaf(a0, a0, t);
                t = fmaf(a1, a1, t);
            }
        }
#pragma unroll
        for (uint32_t m = 1; m < kLanes; m <<= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
        most = fmaxf(most, t);  // passes over NaN
    }
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    if (threadIdx.x % 32 == 0) most_of[threadIdx.x / 32] = most;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most_of[threadIdx.x % (kSizeThreads / 32)])));
    if (threadIdx.x == 0) bp.sizes[blockIdx.x] = most;
}

// The largest of n sizes, for a whole warp.
__device__ __forceinline__ float largest_of(const float* sizes, uint32_t n) {
    float most = 0.f;
    for (uint32_t x = threadIdx.x % 32; x < n; x += 32) most = fmaxf(most, __ldg(sizes + x));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
}

// 2^k with 2^k |dO| |V| in [2^13, 2^14), from the squares of the two; 1 where that is 0 or not finite.
__device__ __forceinline__ float lift(float out_squares, float value_squares) {
    const float t = sqrtf(out_squares) * sqrtf(value_squares);
    const int e = int(__float_as_uint(t) >> 23) - 127;
    return t > 0.f && t <= kFltMax ? __uint_as_float(uint32_t(13 - e + 127) << 23) : 1.0f;
}

// fp16: what the exponent of P is raised by, and the factor that takes it back
template <Fused kF>
struct Raised {
    static constexpr float kUp = kF == Fused::kFP16 ? 8.0f : 0.0f, kDown = kF == Fused::kFP16 ? 0x1p-8f : 1.0f;
};

// ---------------------------------------------------------------- dQ
// One CTA: 128 query rows of one head, tiles of 128 keys.
//  * warp 16, one lane: TMA.  Q and dO once, K and V through a ring K0 V0 K1 V1 ...
//  * warp 17, one lane: W += P(j) K, S(j+1) = Q K^T; dQ += dx(j) K, dP(j+1) = dO V^T, the first two
//    when P is there, the others when dx is (dq_order; P, dx from TMEM, K read MN-major for them).
//  * warps 0-15: a thread per row and quarter of the tile's keys; P (times bend) in 16 bits goes over
//    the scores it came from, dx over the dP.
// TMEM: S, dP (128 columns each), dQ, W (D columns each).
// K is held from S to dQ, about two tiles, V only for dP: three stages and two fill the shared
// memory at D = 128 (with four shared ones the load of K waited for the dQ product before it).
template <int kD>
struct DqShape {
    static constexpr uint32_t kTile = kHalfTile * (kD / 64);
    static constexpr uint32_t kKeyStages = kD == 128 ? 3 : 4, kValueStages = kD == 128 ? 2 : 4;
    static constexpr uint32_t kStages = kKeyStages + kValueStages;
    static constexpr size_t kSmem = (2 + kStages) * size_t(kTile) + 512 + 1024;  // + barriers, alignment
};

template <Fused kF, int kD, bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreadsB, 1) dq_kernel(const __grid_constant__ BackwardParams bp) {
    using S = DqShape<kD>;
    constexpr float kUp = Raised<kF>::kUp, kDown = Raised<kF>::kDown;
    constexpr uint32_t kTile = S::kTile;
    constexpr uint32_t kStages = S::kStages;
    const AttentionParams& p = bp.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (2 + kStages) * size_t(kTile));
    const uint32_t q_smem = smem_u32(smem), do_smem = q_smem + kTile, ring = q_smem + 2 * kTile;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, q_full = empty0 + 8 * kStages;
    const uint32_t s_full = q_full + 8, dp_full = s_full + 8, p_full = dp_full + 8, dx_full = p_full + 8;
    const uint32_t sums_full = dx_full + 8, done = sums_full + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 7);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // stage of tile n of K, of V, and the phase of its barriers
    auto key_stage = [](uint32_t n) { return n % S::kKeyStages; };
    auto value_stage = [](uint32_t n) { return S::kKeyStages + n % S::kValueStages; };
    auto key_phase = [](uint32_t n) { return (n / S::kKeyStages) & 1u; };
    auto value_phase = [](uint32_t n) { return (n / S::kValueStages) & 1u; };

    const Unit unit(bp.dq_split, blockIdx.x);
    const TileHead th(unit.u, bp.q_tiles, p.P * p.B * p.Hl, bp.head_block);
    const uint32_t qt = p.causal ? bp.q_tiles - 1 - th.tile : th.tile;
    const uint32_t h = th.head % p.Hl, b = th.head / p.Hl % p.B, g = th.head / p.Hl / p.B;
    const int row0 = int(qt * kAttnRows);
    const float* value_sizes = bp.sizes + size_t(bp.q_tiles) * p.P * p.B * p.Hl + size_t(th.head / p.shared) * bp.k_tiles;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, 16);  // a warp each
        mbar_init(dx_full, 16);
        mbar_init(sums_full, 16);
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 17) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    const uint32_t tmem = *tmem_slot;
    const uint32_t dp_tmem = tmem + kAttnRows, dq_tmem = tmem + 2 * kAttnRows, w_tmem = dq_tmem + kD;

    const int last = min(row0 + int(kAttnRows), int(p.Sq)) - 1;
    const int reach = (key_bound(p, b, last) + int(kAttnRows) - 1) / int(kAttnRows);
    const int first_tile = unit.begin(reach), n_tiles = unit.end(reach);
    const uint32_t words = (((p.Sk + kAttnRows - 1) / kAttnRows) + 31) / 32;
    const uint32_t* plan = p.plan ? p.plan + (size_t(b) * bp.q_tiles + qt) * 2 * words : nullptr;
    int visits = n_tiles - first_tile;
    if (plan) {
        visits = 0;
        for (uint32_t w = 0; w < words; ++w) visits += __popc(__ldg(plan + w));
    }

    if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");  // 640 * 96 at launch >= 512 * 104 + 128 * 56
    if (warp == 16 && elect_one()) {
        const CUtensorMap* maps[2] = {&bp.k.m[g], &bp.v.m[g]};
        const int kh = int(h / p.shared);
        uint32_t n = 0, loaded[2] = {0, 0};
        bool ok = true;
        if (visits > 0) {
            mbar_expect_tx(q_full, 2 * kTile);
            for (int x = 0; x < kD / 64; ++x) {
                tma_load_4d(q_smem + x * kHalfTile, &bp.q.m[g], x * 64, int(h), row0, int(b), q_full);
                tma_load_4d(do_smem + x * kHalfTile, &bp.dout.m[g], x * 64, int(h), row0, int(b), q_full);
            }
        }
        TileIter it(plan, n_tiles, first_tile);
        for (int j = it.next(); ok && j >= 0; j = it.next(), ++n) {
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t s = kv ? value_stage(n) : key_stage(n), phase_of = kv ? value_phase(n) : key_phase(n);
                const bool again = n >= (kv ? S::kValueStages : S::kKeyStages);
                if (again && !wait_for(empty0 + 8 * s, phase_of ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                mbar_expect_tx(full0 + 8 * s, kTile);
                for (int x = 0; x < kD / 64; ++x)
                    tma_load_4d(ring + s * kTile + x * kHalfTile, maps[kv], x * 64, kh, j * int(kAttnRows), int(b), full0 + 8 * s);
                loaded[kv] = n + 1;
            }
        }
        if (visits > 0) drain_phase(q_full, 0);
        for (uint32_t k = loaded[0] > S::kKeyStages ? loaded[0] - S::kKeyStages : 0; k < loaded[0]; ++k)
            drain_phase(full0 + 8 * key_stage(k), key_phase(k));
        for (uint32_t k = loaded[1] > S::kValueStages ? loaded[1] - S::kValueStages : 0; k < loaded[1]; ++k)
            drain_phase(full0 + 8 * value_stage(k), value_phase(k));
    } else if (warp == 17 && elect_one()) {
        constexpr uint32_t kIdescS = f16_idesc(kF == Fused::kBF16, kAttnRows, kAttnRows, false);
        constexpr uint32_t kIdescQ = f16_idesc(kF == Fused::kBF16, kAttnRows, kD, true);
        struct Pipe {
            decltype(key_stage) k_stage;
            decltype(value_stage) v_stage;
            decltype(key_phase) k_phase;
            decltype(value_phase) v_phase;
            uint32_t full0, empty0, s_full, dp_full, p_full, dx_full, tmem, dp_tmem, dq_tmem, w_tmem, q_low, do_low, kv_low, k_low;
            volatile int* abort_flag;
            __device__ __forceinline__ static uint32_t offset(uint32_t s) { return s * (kTile >> 4); }
            __device__ __forceinline__ bool scores(int i) {
                if (!wait_for(full0 + 8 * k_stage(i), k_phase(i), abort_flag)) return false;
                tc_fence_after();
                tc_product<kD, kHalfTile, kHalfTile>(tmem, q_low, kv_low + offset(k_stage(i)), kIdescS);
                tc_commit(s_full);
                return true;
            }
            __device__ __forceinline__ bool gradients(int i) {
                if (!wait_for(full0 + 8 * v_stage(i), v_phase(i), abort_flag)) return false;
                tc_fence_after();
                tc_product<kD, kHalfTile, kHalfTile>(dp_tmem, do_low, kv_low + offset(v_stage(i)), kIdescS);
                tc_commit(dp_full);
                tc_commit(empty0 + 8 * v_stage(i));
                return true;
            }
            __device__ __forceinline__ bool wait(DqBarrier b, uint32_t parity) {
                if (!wait_for(b == DqBarrier::kWeightsWritten ? p_full : dx_full, parity, abort_flag)) return false;
                tc_fence_after();
                return true;
            }
            // sum += a K, a in TMEM: the quarters of the keys lie 32 columns apart
            __device__ __forceinline__ void add(uint32_t sum, uint32_t a, int i) {
#pragma unroll
                for (uint32_t x = 0; x < 4; ++x)
                    tc_product_ts<32>(sum, a + 32 * x, k_low + offset(k_stage(i)) + (32 * x * kSwizzleRow >> 4), kIdescQ, i != 0 || x != 0);
            }
            __device__ __forceinline__ void weights(int i) { add(w_tmem, tmem, i); }
            __device__ __forceinline__ void update(int i) {
                add(dq_tmem, dp_tmem, i);
                tc_commit(empty0 + 8 * k_stage(i));
            }
        } pipe{key_stage, value_stage, key_phase, value_phase, full0, empty0, s_full, dp_full, p_full, dx_full, tmem, dp_tmem, dq_tmem, w_tmem,
               desc_low(q_smem), desc_low(do_smem), desc_low(ring), desc_low(ring, kHalfTile), abort_flag};
        if (visits > 0 && wait_for(q_full, 0, abort_flag)) dq_order(visits, pipe);
        tc_commit(done);
        drain_phase(done, 0);
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const uint32_t part = warp / 4, quarter = warp % 4, r = quarter * 32 + lane;  // part: 32 keys of the tile
        const int i = row0 + int(r);
        const bool valid = i < int(p.Sq);
        const uint32_t lane_base = (quarter * 32u) << 16;
        int bound = valid ? key_bound(p, b, i) : 0;
        int32_t doc = -1;
        if (plan) {
            doc = valid ? p.q_docs[int64_t(b) * p.Sq + i] : -1;
            if (doc < 0) bound = 0;
        }
        const float slope = kBias && p.slopes ? p.slopes[g * p.Hl + h] : 0.f;
        const int64_t stat = (int64_t(b) * p.Hl + h) * p.Sq + (valid ? i : 0);
        float* delta_at = p.delta + int64_t(g) * p.B * p.Hl * p.Sq + stat;
        const float lse = valid ? p.lse[g][stat] : 0.f;
        const float less = kUp - (lse == -INFINITY ? 0.f : lse * kLog2e), slope2 = slope * kLog2e;
        const int64_t at = valid ? i : 0;
        float delta = 0.f, squares = 0.f;  // d0, |dO|^2
        if (visits > 0 && valid) {
            delta = row_dot<kF, kD>(p.dout.base[g] + b * p.dout.b + at * p.dout.t + h * p.dout.h,
                                    p.out.base[g] + b * p.out.b + at * p.out.t + h * p.out.h, squares);
            if (p.plan && doc < 0) delta = 0.f;  // padding: its output gradient may be anything
        }
        // dx is kept times up, from P times 2^kUp
        const float up = kF == Fused::kFP16 && visits > 0 ? lift(squares, largest_of(value_sizes, bp.k_tiles)) : 1.0f, down = up * kDown;
        // A wait that gives up raises the abort flag: the loop then runs on over what there is, and
        // nothing is written at its end.
        TileIter it(plan, n_tiles, first_tile);
        uint64_t missing = 0;  // e times up, in pairs
        int n = 0;
        for (int j = it.next(); j >= 0; j = it.next(), ++n) {
            const uint32_t s_row = tmem + part * 32 + lane_base, dp_row = dp_tmem + part * 32 + lane_base;
            wait_for(s_full, n & 1u, abort_flag);
            tc_fence_after();
            const int j0 = j * int(kAttnRows) + int(part) * 32;
            float s[32];
            uint64_t bend[kCap ? 16 : 1];
            load_row<32>(s_row, s);
            const int pos = i + int(p.Sk) - int(p.Sq), pos0 = row0 + int(p.Sk) - int(p.Sq);
            const int side = kBias ? bias_side(pos0, int(kAttnRows), j0, 32, p.causal && !p.prefix) : 1;
            const float at = kBias && side != 0 ? less - float(side) * slope2 * float(pos - j0) : less;
            const float by = float(side) * slope2;
            const uint64_t at2 = f2_pack(at, at);
            const ToWeight<kCap> weight(p, s);
            auto weights = [&](auto linear) {
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    uint64_t add = at2;
                    if constexpr (kBias && decltype(linear)::value)
                        add = f2_pack(fmaf(float(x), by, at), fmaf(float(x + 1), by, at));
                    else if constexpr (kBias)
                        add = f2_pack(fmaf(-slope2, fabsf(float(pos - j0 - x)), less), fmaf(-slope2, fabsf(float(pos - j0 - x - 1)), less));
                    f2_unpack(weight(f2_pack(s[x], s[x + 1]), add, bend[kCap ? x / 2 : 0]), s[x], s[x + 1]);
                    s[x] = ex2(s[x]);
                    s[x + 1] = ex2(s[x + 1]);
                }
            };
            if (!kBias || side != 0)
                weights(Bool<true>{});
            else
                weights(Bool<false>{});
            const bool whole = __all_sync(0xffffffffu, plan ? (__ldg(plan + words + (j >> 5)) >> (j & 31)) & 1u : j0 + 32 <= bound);
            uint32_t bits[1] = {0xffffffffu};
            if (!whole) {
                bits[0] = bound_bits(bound, j0);
                if (plan) {
                    const int key = j0 + int(lane);
                    const int32_t kd[1] = {key < int(p.Sk) ? __ldg(p.k_docs + int64_t(b) * p.Sk + key) : -1};
                    keep_document(bits, kd, doc);
                    // padding's K rows may hold anything: clear them for the product with dx
                    if (quarter == 0 && kd[0] < 0) {
                        uint4* k = reinterpret_cast<uint4*>(smem + (2 + key_stage(n)) * size_t(kTile) +
                                                            (part * 32 + lane) * kSwizzleRow);
                        for (int x = 0; x < kD / 64; ++x)
                            for (int y = 0; y < 8; ++y) k[x * (kHalfTile / 16) + y] = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();
                }
#pragma unroll
                for (int x = 0; x < 32; ++x) s[x] = (bits[0] >> x) & 1u ? s[x] : 0.f;
                if constexpr (kCap) {
#pragma unroll
                    for (int x = 0; x < 32; x += 2) bend[x / 2] = keep_pair(bend[x / 2], bits[0] >> x);
                }
            }
            if constexpr (kCap) {
                float w[32];
#pragma unroll
                for (int x = 0; x < 32; x += 2) f2_unpack(f2_mul(f2_pack(s[x], s[x + 1]), bend[x / 2]), w[x], w[x + 1]);
                store_row16<kF, 32>(s_row, w);
            } else {
                store_row16<kF, 32>(s_row, s);
            }
            tc_wait_st();
            warp_arrive(p_full);
            wait_for(dp_full, n & 1u, abort_flag);
            tc_fence_after();
            float d[32];
            load_row<32>(dp_row, d);
            if (!whole) {
#pragma unroll
                for (int x = 0; x < 32; ++x) d[x] = (bits[0] >> x) & 1u ? d[x] : 0.f;
            }
            const float off = kF == Fused::kFP16 ? -delta * down : -delta;
            const uint64_t nd = f2_pack(off, off), down2 = f2_pack(down, down);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
                const uint64_t d2 = f2_pack(d[x], d[x + 1]);
                uint64_t dx = f2_mul(f2_pack(s[x], s[x + 1]), kF == Fused::kFP16 ? f2_fma(d2, down2, nd) : f2_add(d2, nd));
                missing = f2_add(missing, dx);
                if constexpr (kCap) dx = f2_mul(dx, bend[x / 2]);
                f2_unpack(dx, d[x], d[x + 1]);
            }
            store_row16<kF, 32>(dp_row, d);
            tc_wait_st();
            warp_arrive(dx_full);
        }
        // e of the row's four parts meets in columns of S, which no product reads any more
        bool ok = wait_for(done, 0, abort_flag);
        tc_fence_after();
        float part_sum[4] = {0.f, 0.f, 0.f, 0.f};
        if (visits > 0) {
            float lo, hi;
            f2_unpack(missing, lo, hi);
            tc_st1(tmem + lane_base + part, __float_as_uint(lo + hi));
            tc_wait_st();
            warp_arrive(sums_full);
            ok = wait_for(sums_full, 0, abort_flag) && ok;
            tc_fence_after();
            uint32_t bits[4];
            tc_ld4(tmem + lane_base, bits);
#pragma unroll
            for (int x = 0; x < 4; ++x) part_sum[x] = __uint_as_float(bits[x]);
        }
        if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
            const float back = 1.0f / up;  // exact
            const float e = ((part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3])) * back;
            const int64_t row = int64_t(unit.slot) * kAttnRows + r;  // of a part's sums
            if (part == 0 && unit.parts > 1) bp.dq_split.stat[row] = make_float2(e, 0.f);
            if (part == 0 && valid && unit.part == 0) *delta_at = unit.parts > 1 ? delta : delta + e;
            if (part < kD / 32) {
                const uint32_t from = lane_base + part * 32;
                if (unit.parts > 1) {
                    float* dst = bp.dq_split.part + row * kD + part * 32;
                    write_sums<32>(dq_tmem + from, back, dst);
                    write_sums<32>(w_tmem + from, kDown, dst + int64_t(gridDim.x - bp.dq_split.whole) * kAttnRows * kD);
                } else {
                    write_dq<kF>(dq_tmem + from, w_tmem + from, visits > 0, valid, back, e * kDown, p.scale,
                                 p.dq.base[g] + b * p.dq.b + at * p.dq.t + h * p.dq.h + part * 64);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- dK and dV
// One CTA: 128 key rows of one key head, blocks of 64 queries of every query head that
// shares it.  Scores are taken transposed, keys on the TMEM lanes, so that P and dx
// are operands as they stand:
//  * warp 16, one lane: TMA.  K and V once, Q and dO blocks through a ring.
//  * warp 17, one lane: S(n+1) = K Q^T and dP(n+1) = V dO^T into the other pair of
//    buffers, then dV += P(n) dO, dK += dx(n) Q (P, dx from TMEM, dO, Q MN-major).
//  * warps 18 and 19: the queries' log-sum-exp, delta, bounds and documents into shared memory.
//  * warps 0-3 and 8-11 take the even blocks, warps 4-7 and 12-15 the odd ones: a thread per
//    key row and half of the block's queries.
// P goes over S, dx over dP, both in 16 bits.
// TMEM: S0 dP0 S1 dP1 (64 columns each), dK, dV (D columns each).
constexpr uint32_t kQueries = 64;
constexpr int kStatSlots = 4;

// What a block's columns need of their queries.
struct QueryStats {
    float less[kQueries];   // -lse2 (fp16: + 8) and the query's part of the bias
    float delta[kQueries];  // -delta (fp16: times what dx is kept times, and 2^-8)
    int bound[kQueries], doc[kQueries];
};

template <int kD>
struct DkvShape {
    static constexpr uint32_t kTile = kHalfTile * (kD / 64);
    static constexpr uint32_t kBlock = kTile / 2;         // 64 queries
    static constexpr uint32_t kHalfBlock = kHalfTile / 2;
    static constexpr int kStages = 4;                     // of a block's Q and dO
    static constexpr size_t kSmem = 2 * kTile + size_t(kStages) * 2 * kBlock + kStatSlots * sizeof(QueryStats) + 512 + 1024;
};

// The blocks of a key tile, in order: query heads outer; all `per_head` blocks from the query
// tile `first` on, or two (one, at the end) for each tile with a bit in `words`.
struct BlockIter {
    TileIter it;
    const uint32_t* words;
    int q_tiles, first, Sq, tile, part, per_head, m;
    uint32_t head, left;
    // without words: `count` blocks from block `from` of the whole order on
    __device__ BlockIter(const uint32_t* w, int first_tile, int tiles, int sq, uint32_t per, uint32_t from, uint32_t count)
        : it(w, tiles), words(w), q_tiles(tiles), first(first_tile), Sq(sq), tile(-1), part(1), per_head(int(per)),
          m(per ? int(from % per) - 1 : -1), head(per ? from / per : 0), left(count) {}
    // first query of the next block, or -1
    __device__ __forceinline__ int next() {
        if (left == 0) return -1;
        --left;
        if (!words) {
            if (++m >= per_head) {
                m = 0;
                ++head;
            }
            return first * int(kAttnRows) + m * int(kQueries);
        }
        if (part == 0 && tile * int(kAttnRows) + int(kQueries) < Sq) {
            part = 1;
            return tile * int(kAttnRows) + int(kQueries);
        }
        while ((tile = it.next()) < 0) {  // there is one more block: in the next head
            ++head;
            it = TileIter(words, q_tiles);
        }
        part = 0;
        return tile * int(kAttnRows);
    }
};

// Blocks that one query head gives.
__device__ __forceinline__ uint32_t blocks_of(const uint32_t* words, int first, int q_tiles, int Sq) {
    const bool odd = Sq > 0 && (Sq - 1) % int(kAttnRows) < int(kQueries);  // the last tile has one block
    if (!words) return first < q_tiles ? 2 * uint32_t(q_tiles - first) - odd : 0;
    uint32_t n = 0;
    for (int w = 0; w * 32 < q_tiles; ++w) n += 2 * __popc(__ldg(words + w));
    return n - (odd && (__ldg(words + (q_tiles - 1) / 32) >> ((q_tiles - 1) % 32) & 1u));
}

template <Fused kF, int kD, bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreadsB, 1) dkv_kernel(const __grid_constant__ BackwardParams bp) {
    using S = DkvShape<kD>;
    constexpr uint32_t kTile = S::kTile, kBlock = S::kBlock, kHalfBlock = S::kHalfBlock;
    constexpr int kStages = S::kStages;
    constexpr float kUp = Raised<kF>::kUp, kDown = Raised<kF>::kDown;
    const AttentionParams& p = bp.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    QueryStats* stats = reinterpret_cast<QueryStats*>(smem + 2 * size_t(kTile) + kStages * 2 * size_t(kBlock));
    uint64_t* bars = reinterpret_cast<uint64_t*>(stats + kStatSlots);
    const uint32_t k_smem = smem_u32(smem), v_smem = k_smem + kTile, ring = k_smem + 2 * kTile;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, kv_full = empty0 + 8 * kStages;
    const uint32_t s_full0 = kv_full + 8, dx_full0 = s_full0 + 16, stat_full0 = dx_full0 + 16;
    const uint32_t stat_free0 = stat_full0 + 8 * kStatSlots, done = stat_free0 + 8 * kStatSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 6 + 2 * kStatSlots);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    const Unit unit(bp.dkv_split, blockIdx.x);
    const TileHead th(unit.u, bp.k_tiles, p.P * p.B * p.Hkl, bp.key_head_block);
    const uint32_t kt = th.tile;  // causal: the first keys are seen by most queries
    const uint32_t kh = th.head % p.Hkl, b = th.head / p.Hkl % p.B, g = th.head / p.Hkl / p.B;
    const int row0 = int(kt * kAttnRows);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(kv_full, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full0 + 8 * t, 1);
            mbar_init(dx_full0 + 8 * t, 8);  // a warp each
        }
        for (int t = 0; t < kStatSlots; ++t) {
            mbar_init(stat_full0 + 8 * t, 1);
            mbar_init(stat_free0 + 8 * t, 8);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 17) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    const uint32_t tmem = *tmem_slot;
    const uint32_t dk_tmem = tmem + 256, dv_tmem = dk_tmem + kD;

    const int ahead = int(p.Sk) - int(p.Sq);
    const int q_tiles = int((p.Sq + kAttnRows - 1) / kAttnRows);
    int first = 0;  // the first query tile in reach of the keys
    if (p.causal && !(p.prefix && row0 < p.prefix[b])) first = min(q_tiles, max(0, row0 - ahead) / int(kAttnRows));
    const uint32_t words = (uint32_t(q_tiles) + 31) / 32;
    const uint32_t* plan = p.plan ? p.plan + (size_t(b) * bp.k_tiles + kt) * 2 * words : nullptr;
    const uint32_t per_head = blocks_of(plan, first, q_tiles, int(p.Sq));
    const uint32_t first_block = uint32_t(unit.begin(int(p.shared * per_head)));
    const uint32_t blocks = uint32_t(unit.end(int(p.shared * per_head))) - first_block;
    // dx is kept times up, from P times 2^kUp: one factor for all queries of the key head
    float up = 1.0f;
    if (kF == Fused::kFP16 && blocks > 0)
        up = lift(largest_of(bp.sizes + size_t(th.head) * p.shared * q_tiles, p.shared * q_tiles),
                  largest_of(bp.sizes + size_t(q_tiles) * p.P * p.B * p.Hl + size_t(th.head) * bp.k_tiles, bp.k_tiles));
    const float down = up * kDown;
    BlockIter it(plan, first, q_tiles, int(p.Sq), per_head, first_block, blocks);

    if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");  // 640 * 96 at launch >= 512 * 104 + 128 * 56
    if (warp == 16 && elect_one()) {
        uint32_t n = 0;
        bool ok = true;
        int i0 = it.next();
        if (i0 >= 0) {
            mbar_expect_tx(kv_full, 2 * kTile);
            for (int x = 0; x < kD / 64; ++x) {
                tma_load_4d(k_smem + x * kHalfTile, &bp.k.m[g], x * 64, int(kh), row0, int(b), kv_full);
                tma_load_4d(v_smem + x * kHalfTile, &bp.v.m[g], x * 64, int(kh), row0, int(b), kv_full);
            }
        }
        const bool any = i0 >= 0;
        for (; ok && i0 >= 0; i0 = it.next()) {
            const int h = int(kh * p.shared + it.head);
            const uint32_t s = n % kStages, use = n / kStages;
            ++n;
            if (use > 0 && !wait_for(empty0 + 8 * s, (use - 1) & 1u, abort_flag)) {
                ok = false;
                --n;
                break;
            }
            mbar_expect_tx(full0 + 8 * s, 2 * kBlock);
            for (int qd = 0; qd < 2; ++qd)
                for (int x = 0; x < kD / 64; ++x)
                    tma_load_4d(ring + (2 * s + qd) * kBlock + x * kHalfBlock, qd == 0 ? &bp.q_half.m[g] : &bp.dout_half.m[g], x * 64,
                                h, i0, int(b), full0 + 8 * s);
        }
        if (any) drain_phase(kv_full, 0);
        for (uint32_t k = n > uint32_t(kStages) ? n - kStages : 0; k < n; ++k)
            drain_phase(full0 + 8 * (k % kStages), (k / kStages) & 1u);
    } else if (warp == 17 && elect_one()) {
        constexpr uint32_t kIdescS = f16_idesc(kF == Fused::kBF16, kAttnRows, kQueries, false);
        constexpr uint32_t kIdescD = f16_idesc(kF == Fused::kBF16, kAttnRows, kD, true);
        const uint32_t k_low = desc_low(k_smem), v_low = desc_low(v_smem), n_low = desc_low(ring),
                       t_low = desc_low(ring, kHalfBlock);
        auto transposed = [&](uint32_t n) {  // S and dP of block n
            const uint32_t s = n % kStages;
            if (!wait_for(full0 + 8 * s, (n / kStages) & 1u, abort_flag)) return false;
            tc_fence_after();
            const uint32_t d = tmem + (n & 1) * 2 * kQueries, q = n_low + s * (2 * kBlock >> 4);
            tc_product<kD, kHalfTile, kHalfBlock>(d, k_low, q, kIdescS);
            tc_product<kD, kHalfTile, kHalfBlock>(d + kQueries, v_low, q + (kBlock >> 4), kIdescS);
            tc_commit(s_full0 + 8 * (n & 1));
            return true;
        };
        bool ok = blocks == 0 || (wait_for(kv_full, 0, abort_flag) && transposed(0));
        for (uint32_t n = 0; ok && n < blocks; ++n) {
            if (n + 1 < blocks && !(ok = transposed(n + 1))) break;
            if (!(ok = wait_for(dx_full0 + 8 * (n & 1), (n >> 1) & 1u, abort_flag))) break;
            tc_fence_after();
            const uint32_t a = tmem + (n & 1) * 2 * kQueries, q = t_low + n % kStages * (2 * kBlock >> 4);
#pragma unroll
            for (uint32_t x = 0; x < 2; ++x)  // dV += P dO; the halves of the queries lie 32 columns apart
                tc_product_ts<32>(dv_tmem, a + 32 * x, q + (kBlock >> 4) + (32 * x * kSwizzleRow >> 4), kIdescD, n | x);
#pragma unroll
            for (uint32_t x = 0; x < 2; ++x)  // dK += dx Q
                tc_product_ts<32>(dk_tmem, a + kQueries + 32 * x, q + (32 * x * kSwizzleRow >> 4), kIdescD, n | x);
            tc_commit(empty0 + 8 * (n % kStages));
        }
        tc_commit(done);
        drain_phase(done, 0);
    } else if (warp >= 18) {
        uint32_t n = 0;
        for (int i0 = it.next(); i0 >= 0; i0 = it.next(), ++n) {
            if ((n & 1u) != (warp & 1u)) continue;
            // two queries a lane; what is read is on its way before the slot is free
            const int64_t stat = (int64_t(b) * p.Hl + kh * p.shared + it.head) * p.Sq;
            const float slope2 = kBias && p.slopes ? p.slopes[g * p.Hl + kh * p.shared + it.head] * kLog2e : 0.f;
            const int side = kBias ? bias_side(i0 + ahead, int(kQueries), row0, int(kAttnRows), p.causal && !p.prefix) : 0;
            float less[2], delta[2];
            int bound[2], doc[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = i0 + int(lane) + 32 * x;
                less[x] = -INFINITY;  // no such query: weight 0
                delta[x] = 0.f;
                bound[x] = 0;
                doc[x] = -1;
                if (i < int(p.Sq)) {
                    const float lse = p.lse[g][stat + i];
                    delta[x] = -down * p.delta[int64_t(g) * p.B * p.Hl * p.Sq + stat + i];
                    bound[x] = key_bound(p, b, i);
                    if (plan) {
                        doc[x] = p.q_docs[int64_t(b) * p.Sq + i];
                        if (doc[x] < 0) {
                            bound[x] = 0;
                            delta[x] = 0.f;
                        }
                    }
                    if (lse != -INFINITY) less[x] = kUp - lse * kLog2e - float(side * (int(lane) + 32 * x)) * slope2;
                }
            }
            if (n >= uint32_t(kStatSlots)) {  // block n - kStatSlots has been computed
                const bool ok = wait_for(stat_free0 + 8 * (n % kStatSlots), (n / kStatSlots - 1) & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) break;
            }
            QueryStats& st = stats[n % kStatSlots];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int at = int(lane) + 32 * x;
                st.less[at] = less[x];
                st.delta[at] = delta[x];
                st.bound[at] = bound[x];
                st.doc[at] = doc[x];
            }
            warp_arrive(stat_full0 + 8 * (n % kStatSlots));
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const uint32_t t = warp / 4 % 2, half = warp / 8, quarter = warp % 4, r = quarter * 32 + lane;
        const int j = row0 + int(r);
        const bool valid = j < int(p.Sk);
        const uint32_t lane_base = (quarter * 32u) << 16;
        const int32_t doc = plan && valid ? p.k_docs[int64_t(b) * p.Sk + j] : -1;
        const uint32_t s_row = tmem + t * 2 * kQueries + 32 * half + lane_base, dp_row = s_row + kQueries;
        uint32_t n = 0;
        for (int i0 = it.next(); i0 >= 0; i0 = it.next(), ++n) {
            if ((n & 1u) != t) continue;
            const uint32_t slot = n % kStatSlots;
            wait_for(stat_full0 + 8 * slot, (n / kStatSlots) & 1u, abort_flag);  // (see dq_kernel for a wait that gives up)
            wait_for(s_full0 + 8 * t, (n >> 1) & 1u, abort_flag);
            tc_fence_after();
            const QueryStats& st = stats[slot];
            const float slope2 = kBias && p.slopes ? p.slopes[g * p.Hl + kh * p.shared + it.head] * kLog2e : 0.f;
            const int side = kBias ? bias_side(i0 + ahead, int(kQueries), row0, int(kAttnRows), p.causal && !p.prefix) : 0;
            // the query's part of the bias counts from the block's first one
            const float far = float(i0 + int(32 * half) + ahead - j), own = -float(side) * slope2 * float(i0 + ahead - j);
            const uint64_t own2 = f2_pack(own, own), down2 = f2_pack(down, down);
            float s[32], d[32];
            load_row<32>(s_row, s);
            const ToWeight<kCap> weight(p, s);
            const int qt = i0 / int(kAttnRows);
            const bool whole = plan ? (__ldg(plan + words + (qt >> 5)) >> (qt & 31)) & 1u  // the same for every thread
                                    : i0 + int(kQueries) <= int(p.Sq) && row0 + int(kAttnRows) <= st.bound[0];
            uint32_t bits = 0xffffffffu;
            if (!whole) {
#pragma unroll
                for (int x = 0; x < 32; x += 4) {
                    const int4 bound = *reinterpret_cast<const int4*>(st.bound + 32 * half + x),
                               doc4 = *reinterpret_cast<const int4*>(st.doc + 32 * half + x);
                    const int* bo = &bound.x;
                    const int* dc = &doc4.x;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        if (j >= bo[y] || (plan && dc[y] != doc)) bits &= ~(1u << (x + y));
                }
                // padding's Q and dO rows may hold anything: clear them for the products with dx and P
                if (plan && half == 0 && r < kQueries && st.doc[r] < 0) {
                    for (int qd = 0; qd < 2; ++qd) {
                        uint4* row = reinterpret_cast<uint4*>(smem + 2 * size_t(kTile) +
                                                              (2 * (n % kStages) + qd) * size_t(kBlock) + r * kSwizzleRow);
                        for (int x = 0; x < kD / 64; ++x)
                            for (int y = 0; y < 8; ++y) row[x * (kHalfBlock / 16) + y] = make_uint4(0, 0, 0, 0);
                    }
                }
                if (plan) fence_async_shared();
            }
            load_row<32>(dp_row, d);
            auto gradients = [&](auto masked, auto linear) {
#pragma unroll
                for (int x = 0; x < 32; x += 4) {
                    const float4 less = *reinterpret_cast<const float4*>(st.less + 32 * half + x),
                                 nd = *reinterpret_cast<const float4*>(st.delta + 32 * half + x);
#pragma unroll
                    for (int y = 0; y < 4; y += 2) {
                        const int e = x + y;
                        const float l0 = y ? less.z : less.x, l1 = y ? less.w : less.y;
                        uint64_t add = f2_pack(l0, l1), bend = 0;
                        if constexpr (kBias && decltype(linear)::value)
                            add = f2_add(add, own2);
                        else if constexpr (kBias)
                            add = f2_pack(fmaf(-slope2, fabsf(far + float(e)), l0), fmaf(-slope2, fabsf(far + float(e + 1)), l1));
                        f2_unpack(weight(f2_pack(s[e], s[e + 1]), add, bend), s[e], s[e + 1]);
                        s[e] = ex2(s[e]);
                        s[e + 1] = ex2(s[e + 1]);
                        if constexpr (decltype(masked)::value) {
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const bool see = (bits >> (e + z)) & 1u;
                                s[e + z] = see ? s[e + z] : 0.f;
                                d[e + z] = see ? d[e + z] : 0.f;
                            }
                            if constexpr (kCap) bend = keep_pair(bend, bits >> e);
                        }
                        const uint64_t off = y ? f2_pack(nd.z, nd.w) : f2_pack(nd.x, nd.y), d2 = f2_pack(d[e], d[e + 1]);
                        uint64_t dx = f2_mul(f2_pack(s[e], s[e + 1]), kF == Fused::kFP16 ? f2_fma(d2, down2, off) : f2_add(d2, off));
                        if constexpr (kCap) dx = f2_mul(dx, bend);
                        f2_unpack(dx, d[e], d[e + 1]);
                    }
                }
            };
            if (whole && (!kBias || side != 0))
                gradients(Bool<false>{}, Bool<true>{});
            else if (!kBias || side != 0)
                gradients(Bool<true>{}, Bool<true>{});
            else
                gradients(Bool<true>{}, Bool<false>{});
            store_row16<kF, 32>(s_row, s);
            store_row16<kF, 32>(dp_row, d);
            tc_wait_st();
            warp_arrive(dx_full0 + 8 * t);
            if (lane == 0) mbar_arrive(stat_free0 + 8 * slot);
        }
        // n counts every block, of both halves of the warps
        const bool ok = wait_for(done, 0, abort_flag);
        if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
            tc_fence_after();
            const int64_t at = valid ? j : 0;
            constexpr int kCols = kD / 2;  // of each half of the warps
            const uint32_t from = (t == 0 ? dv_tmem : dk_tmem) + lane_base + half * kCols;
            if (unit.parts > 1) {
                const int64_t cut = int64_t(bp.k_tiles) * p.P * p.B * p.Hkl - bp.dkv_split.whole;  // units in parts
                const int64_t row = (t == 0 ? cut * unit.parts + unit.slot : int64_t(unit.slot)) * kAttnRows + r;
                write_sums<kCols>(from, t == 0 ? 1.0f : 1.0f / up, bp.dkv_split.part + row * kD + half * kCols);
            } else if (t == 0) {
                write_row<kF, kCols>(from, n > 0, valid, kDown, p.dv.base[g] + b * p.dv.b + at * p.dv.t + kh * p.dv.h + half * kCols * 2);
            } else {
                write_row<kF, kCols>(from, n > 0, valid, p.scale / up,
                                     p.dk.base[g] + b * p.dk.b + at * p.dk.t + kh * p.dk.h + half * kCols * 2);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <Fused kF, int kD, bool kCap, bool kBias>
cudaError_t launch(const BackwardParams& p, cudaStream_t stream, int* launches) {
    cudaError_t e;
    BackwardParams q = p;
    if (kF == Fused::kFP16 && p.a.Sq > 0 && p.a.Sk > 0) {
        const uint32_t tiles = p.q_tiles * p.a.P * p.a.B * p.a.Hl + p.k_tiles * p.a.P * p.a.B * p.a.Hkl;
        if ((e = launch_overlapped(sizes_kernel<kD>, tiles, kSizeThreads, 0, stream, p)) != cudaSuccess) return e;
        *launches += 1;
    }
    if (p.a.Sq > 0) {
        if (p.a.plan) {
            if ((e = launch_plan(p.a, p.a.plan, false, kAttnRows, stream)) != cudaSuccess) return e;
            *launches += 1;
        }
        auto kernel = dq_kernel<kF, kD, kCap, kBias>;
        constexpr size_t smem = DqShape<kD>::kSmem;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem))) != cudaSuccess) return e;
        const uint32_t units = p.q_tiles * p.a.P * p.a.B * p.a.Hl;
        const Split& cut = p.dq_split;
        e = launch_overlapped(kernel, cut.whole + (units - cut.whole) * cut.parts, kThreadsB, smem, stream, p);
        if (e != cudaSuccess) return e;
        *launches += 1;
        if (cut.parts > 1) {
            e = launch_join_dq(p, kF == Fused::kBF16, stream);
            if (e != cudaSuccess) return e;
            *launches += 1;
        }
    }
    if (p.a.Sk > 0) {
        if (p.a.plan) {
            q.a.plan = p.key_plan;
            if ((e = launch_plan(q.a, q.a.plan, true, kAttnRows, stream)) != cudaSuccess) return e;
            *launches += 1;
        }
        auto kernel = dkv_kernel<kF, kD, kCap, kBias>;
        constexpr size_t smem = DkvShape<kD>::kSmem;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem))) != cudaSuccess) return e;
        const uint32_t units = p.k_tiles * p.a.P * p.a.B * p.a.Hkl;
        const Split& cut = p.dkv_split;
        e = launch_overlapped(kernel, cut.whole + (units - cut.whole) * cut.parts, kThreadsB, smem, stream, q);
        if (e != cudaSuccess) return e;
        *launches += 1;
        if (cut.parts > 1) {
            const float* dv_part = cut.part + int64_t(units - cut.whole) * cut.parts * kAttnRows * kD;
            constexpr float kDown = Raised<kF>::kDown;
            e = launch_join_gradient(p.a, cut, p.a.dk, cut.part, p.a.scale, p.k_tiles, p.a.Sk, p.a.Hkl, kF == Fused::kBF16, stream);
            if (e == cudaSuccess)
                e = launch_join_gradient(p.a, cut, p.a.dv, dv_part, kDown, p.k_tiles, p.a.Sk, p.a.Hkl, kF == Fused::kBF16, stream);
            if (e != cudaSuccess) return e;
            *launches += 2;
        }
    }
    return cudaSuccess;
}

template <Fused kF, int kD>
cudaError_t launch_scored(const BackwardParams& p, cudaStream_t stream, int* launches) {
    if (p.a.cap != 0.f)
        return p.a.slopes ? launch<kF, kD, true, true>(p, stream, launches) : launch<kF, kD, true, false>(p, stream, launches);
    return p.a.slopes ? launch<kF, kD, false, true>(p, stream, launches) : launch<kF, kD, false, false>(p, stream, launches);
}

}  // namespace

cudaError_t launch_attention_backward(const BackwardParams& p, bool bf16, cudaStream_t stream, int* launches) {
    *launches = 0;
    if (p.a.D == 64)
        return bf16 ? launch_scored<Fused::kBF16, 64>(p, stream, launches) : launch_scored<Fused::kFP16, 64>(p, stream, launches);
    return bf16 ? launch_scored<Fused::kBF16, 128>(p, stream, launches) : launch_scored<Fused::kFP16, 128>(p, stream, launches);
}

cudaError_t read_attention_backward_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_backward_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attention_backward_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
