// attention_forward.cu -- attention over the head groups, forward, on the
// 5th-generation tensor cores.
//
// One pass over the keys with the running reference m and sum l of each row's
// softmax (Milakov & Gimelshein, "Online normalizer calculation for softmax",
// 2018), z in units of log2: o = sum 2^(z - m) v, l = sum 2^(z - m).  m follows the
// row's maximum only when that outgrows it by more than 2^8: what is scaled by
// 2^(m_old - m) then is rare, the weights stay below 2^8 and all sums are fp32.
//
// A CTA of 384 threads takes two tiles of 128 queries of one head and walks the
// tiles of 128 keys that some query can see:
//  * warp 8, one lane: TMA producer.  Q once, then K and V tiles through a ring of
//    stages in the order K0 V0 K1 V1 ...
//  * warp 9, one lane: issues S_t = Q_t K^T (both operands from shared memory) and
//    O_t += P_t V (P_t from TMEM, V read MN-major) for t = 0, 1.  The matrix pipe
//    completes in order, so S_t of the next keys may overwrite P_t behind the
//    product that reads it, and a finished S_t says that O_t stands still.
//  * warps 0-3 and 4-7: one thread a query row of tile 0 or 1.  Reads the row's 128
//    scores from TMEM, masks, takes maximum, weights and sum, writes the 16-bit
//    weights back over the scores, and at the end divides and stores the row.
// While one tile's softmax runs, the matrix pipe works on the other tile.
// Registers move from the last warpgroup (two idle warps among it) to the rows' threads.
// TMEM: S0 S1 (128 columns each, P on top of S), O0 O1 (D columns each).
//
// Bound: the products, 4 D flops a pair of tokens, and beside them the rows' threads.  32760 tokens, 5
// heads, D = 128, bf16, capped scores: 2.14 to 2.23 ms, 1230 to 1280 TFLOP/s; 8192 tokens uncapped: the matrix pipe is busy
// 67 % of the cycles, the exponentials' pipe 34 %; capped: 53 and 27 %.  A pair of tiles keeps the pipe fed through the
// softmax of either; one elected thread issues a 128 x 128 x 128 product in 518 cycles of 512.  D = 64 halves
// the products, not the scores: 24 heads of 6001 tokens with causal mask and bias take 196 us,
// the pipe busy 26 %, issue slots 48 %.  Every instance spills 56 to 80 bytes: local loads and stores
// are 1.1 to 1.4 % of its instructions.
#include "attention_common.cuh"
#include "attention_plan.h"

namespace tfu {

__device__ unsigned g_attention_status;

namespace {

using namespace dev;

constexpr int kThreadsA = 384;
constexpr uint32_t kHalfTile = kAttnRows * kSwizzleRow;  // 128 rows of 64 elements: 16 KiB

template <int kD>
struct Shape {
    static constexpr uint32_t kTile = kHalfTile * (kD / 64);
    static constexpr int kStages = kD == 128 ? 5 : 8;
    static constexpr size_t kSmem = 2 * kTile + size_t(kStages) * kTile + 512 + 1024;  // tiles, barriers, alignment
};

template <Fused kF, int kD, Score kScore>
__global__ void __launch_bounds__(kThreadsA, 1) attention_kernel(const __grid_constant__ ForwardParams fp) {
    using S = Shape<kD>;
    constexpr uint32_t kTile = S::kTile;
    constexpr int kStages = S::kStages;
    const AttentionParams& p = fp.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (2 + kStages) * size_t(kTile));
    const uint32_t q_smem = smem_u32(smem), ring = q_smem + 2 * kTile;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, q_full = empty0 + 8 * kStages;
    const uint32_t s_full0 = q_full + 8, p_half0 = s_full0 + 16, o_full = p_half0 + 32;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    const Unit unit(fp.split, blockIdx.x);
    const TileHead th(unit.u, fp.q_tiles, p.P * p.B * p.Hl, fp.head_block);
    uint32_t qt = p.causal ? fp.q_tiles - 1 - th.tile : th.tile;  // the rows that see most first
    uint32_t h = th.head % p.Hl, b = th.head / p.Hl % p.B, g = th.head / p.Hl / p.B;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(q_full, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full0 + 8 * t, 1);
            mbar_init(p_half0 + 16 * t, 4);  // a warp each
            mbar_init(p_half0 + 16 * t + 8, 4);
        }
        mbar_init(o_full, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    const uint32_t tmem = *tmem_slot;
    const uint32_t o_tmem = tmem + 2 * kAttnRows;

    const uint32_t words = (((p.Sk + kAttnRows - 1) / kAttnRows) + 31) / 32;
    if (fp.ranked) {
        const uint32_t heads = p.P * p.Hl, head = unit.u % heads;
        const uint32_t e = ranked_entry(p.plan, p.B * fp.q_tiles, words, unit.u / heads, reinterpret_cast<uint32_t*>(smem));
        qt = e % fp.q_tiles, b = e / fp.q_tiles, h = head % p.Hl, g = head / p.Hl;
    }
    const int row0 = int(qt * kAttnPair);
    const int tiles = row0 + int(kAttnRows) < int(p.Sq) ? 2 : 1;

    // the keys in reach of the last row, in tiles; with documents the plan picks among them
    const int last = min(row0 + int(kAttnPair), int(p.Sq)) - 1;
    const int reach = (key_bound(p, b, last) + int(kAttnRows) - 1) / int(kAttnRows);
    const int n_tiles = unit.end(reach);
    const uint32_t* plan = p.plan ? p.plan + (size_t(b) * fp.q_tiles + qt) * 2 * words : nullptr;
    TileIter it(plan, n_tiles, unit.begin(reach));

    // 384 * 168 registers at launch = 256 * 216 + 128 * 72
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8 && elect_one()) {
        // ---------------- TMA producer
        const CUtensorMap* maps[2] = {&fp.k.m[g], &fp.v.m[g]};
        const int kh = int(h / p.shared);
        uint32_t n = 0;  // tiles loaded into the ring
        bool ok = true;
        int j = it.next();
        if (j >= 0) {
            mbar_expect_tx(q_full, uint32_t(tiles) * kTile);
            for (int t = 0; t < tiles; ++t)
                for (int x = 0; x < kD / 64; ++x)
                    tma_load_4d(q_smem + t * kTile + x * kHalfTile, &fp.q.m[g], x * 64, int(h), row0 + t * int(kAttnRows),
                                int(b), q_full);
        }
        for (; ok && j >= 0; j = it.next()) {
            for (int kv = 0; kv < 2; ++kv, ++n) {
                const uint32_t s = n % kStages, use = n / kStages;
                if (use > 0 && !bounded_wait(empty0 + 8 * s, (use - 1) & 1u, abort_flag, &g_attention_status)) {
                    ok = false;
                    break;
                }
                mbar_expect_tx(full0 + 8 * s, kTile);
                for (int x = 0; x < kD / 64; ++x)
                    tma_load_4d(ring + s * kTile + x * kHalfTile, maps[kv], x * 64, kh, j * int(kAttnRows), int(b),
                                full0 + 8 * s);
            }
        }
        // every load has landed before the CTA exits
        if (n > 0) drain_phase(q_full, 0);
        for (uint32_t k = n > uint32_t(kStages) ? n - kStages : 0; k < n; ++k)
            drain_phase(full0 + 8 * (k % kStages), (k / kStages) & 1u);
    } else if (warp == 9 && elect_one()) {
        // ---------------- MMA issuer
        constexpr uint32_t kIdescS = f16_idesc(kF == Fused::kBF16, kAttnRows, kAttnRows, false);
        constexpr uint32_t kIdescO = f16_idesc(kF == Fused::kBF16, kAttnRows, kD, true);
        const uint32_t q_low = desc_low(q_smem), k_low = desc_low(ring), v_low = desc_low(ring, kHalfTile);
        auto scores = [&](int t, uint32_t s) {
            tc_product<kD, kHalfTile, kHalfTile>(tmem + t * kAttnRows, q_low + t * (kTile >> 4), k_low + s * (kTile >> 4), kIdescS);
            tc_commit(s_full0 + 8 * t);
        };
        // the ring's next tile: stage and phase
        uint32_t s = 0, phase = 0;
        auto landed = [&]() { return bounded_wait(full0 + 8 * s, phase, abort_flag, &g_attention_status); };
        auto advance = [&]() {
            if (++s == uint32_t(kStages)) s = 0, phase ^= 1u;
        };
        int i = 0;  // key tiles finished
        int j = it.next();
        bool ok = j < 0 || (bounded_wait(q_full, 0, abort_flag, &g_attention_status) && landed());
        if (ok && j >= 0) {
            tc_fence_after();
            for (int t = 0; t < tiles; ++t) scores(t, 0);
            tc_commit(empty0);
            advance();
        }
        for (; ok && j >= 0; ++i) {
            j = it.next();
            if (!(ok = landed())) break;
            const uint32_t v = s;
            advance();
            for (int t = 0; t < tiles; ++t) {
                // P of the first 64 keys while the weights of the others are computed
                for (int x = 0; ok && x < 2; ++x) {
                    ok = bounded_wait(p_half0 + 16 * t + 8 * x, i & 1u, abort_flag, &g_attention_status);
                    if (!ok) break;
                    tc_fence_after();
                    tc_product_ts<kAttnRows / 2>(o_tmem + t * kD, tmem + t * kAttnRows + x * 32,
                                                 v_low + v * (kTile >> 4) + x * (64 * kSwizzleRow >> 4), kIdescO, uint32_t(i | x));
                }
                if (!ok) break;
                if (j >= 0) {
                    if (t == 0 && !(ok = landed())) break;
                    tc_fence_after();
                    scores(t, s);
                }
            }
            if (!ok) break;
            tc_commit(empty0 + 8 * v);
            if (j >= 0) {
                tc_commit(empty0 + 8 * s);
                advance();
            }
        }
        tc_commit(o_full);
        drain_phase(o_full, 0);  // every MMA of this CTA has completed
    }
    } else {
        // ---------------- softmax and epilogue: a thread per query row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const uint32_t t = warp / 4, quarter = warp % 4;
        const int i = row0 + int(t * kAttnRows + quarter * 32 + lane);
        const bool valid = i < int(p.Sq);
        const uint32_t lane_base = (quarter * 32u) << 16;
        const uint32_t s_tmem = tmem + t * kAttnRows + lane_base, o_row = o_tmem + t * kD + lane_base;
        int bound = valid ? key_bound(p, b, i) : 0;
        int32_t doc = -1;
        if (p.plan) {
            doc = valid ? p.q_docs[int64_t(b) * p.Sq + i] : -1;
            if (doc < 0) bound = 0;
        }
        const float slope = kScore == Score::kAny && p.slopes ? p.slopes[g * p.Hl + h] : 0.f;
        const float c = kScore == Score::kPlain ? p.scale * kLog2e : 1.0f;
        float m = -INFINITY, l = 0.f;
        int n = 0;  // key tiles done
        bool ok = true;
        for (int j = int(t) < tiles ? it.next() : -1; j >= 0; j = it.next(), ++n) {
            ok = bounded_wait(s_full0 + 8 * t, n & 1u, abort_flag, &g_attention_status);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float s[128];
            load_row<128>(s_tmem, s);
            const int j0 = j * int(kAttnRows);
            const bool whole = __all_sync(0xffffffffu, plan ? (__ldg(plan + words + (j >> 5)) >> (j & 31)) & 1u
                                                            : j0 + int(kAttnRows) <= bound);
            if (kScore == Score::kCap && whole &&
                fold_capped_tile<kF, kD, true>(s, p.scale, p.cap, 1.0f, n > 0, m, l, s_tmem, o_row, p_half0 + 16 * t))
                continue;
            const int pos0 = row0 + int(t * kAttnRows) + int(p.Sk) - int(p.Sq);
            if (kScore != Score::kPlain)
                finish_scores<kScore>(s, p.scale, p.cap, slope, float(i + (int(p.Sk) - int(p.Sq)) - j0),
                                      bias_side(pos0, int(kAttnRows), j0, int(kAttnRows), p.causal && !p.prefix));
            if (!whole) {
                uint32_t bits[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) bits[x] = bound_bits(bound, j0 + 32 * x);
                if (plan) {
                    int32_t kd[4];  // the tile's documents, four keys a lane
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = j0 + x * 32 + int(lane);
                        kd[x] = key < int(p.Sk) ? __ldg(p.k_docs + int64_t(b) * p.Sk + key) : -1;
                    }
                    keep_document(bits, kd, doc);
                    // the warps of tile 0 clear the V rows of padding, whose contents may be anything
                    int32_t own = kd[0];
#pragma unroll
                    for (int x = 1; x < 4; ++x) own = quarter == uint32_t(x) ? kd[x] : own;
                    if (t == 0 && __any_sync(0xffffffffu, own < 0)) {
                        const uint32_t vn = 2 * uint32_t(n) + 1;
                        ok = bounded_wait(full0 + 8 * (vn % kStages), (vn / kStages) & 1u, abort_flag, &g_attention_status);
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        if (own < 0) {
                            uint4* v = reinterpret_cast<uint4*>(smem + (2 + vn % kStages) * size_t(kTile) +
                                                                (quarter * 32 + lane) * kSwizzleRow);
                            for (int x = 0; x < kD / 64; ++x)
                                for (int y = 0; y < 8; ++y) v[x * (kHalfTile / 16) + y] = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_shared();
                    }
                }
#pragma unroll
                for (int x = 0; x < 128; ++x) s[x] = (bits[x / 32] >> (x % 32)) & 1u ? s[x] : -INFINITY;
            }
            fold_tile<kF, kD>(s, c, 1.0f, n > 0, m, l, s_tmem, o_row, p_half0 + 16 * t);
        }
        if (int(t) < tiles && ok) {
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            uint8_t* dst = p.out.base[g] + int64_t(b) * p.out.b + int64_t(valid ? i : 0) * p.out.t + int64_t(h) * p.out.h;
            const int64_t row = int64_t(unit.slot) * kAttnPair + t * kAttnRows + quarter * 32 + lane;  // of a part's sums
            if (n > 0) ok = bounded_wait(o_full, 0, abort_flag, &g_attention_status);
            if (__all_sync(0xffffffffu, ok) && !*abort_flag) {
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < kD; x += 32) {
                    uint32_t r[32];
                    if (n > 0) {
                        tc_ld32(o_row + x, r);
                        tc_wait_ld();
                        tc_landed(r);
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) r[y] = 0;
                    }
                    if (unit.parts > 1) {
#pragma unroll
                        for (int y = 0; y < 32; y += 4)
                            *reinterpret_cast<uint4*>(fp.split.part + row * kD + x + y) = make_uint4(r[y], r[y + 1], r[y + 2], r[y + 3]);
                        continue;
                    }
#pragma unroll
                    for (int y = 0; y < 32; y += 8) {
                        uint4 w;
                        uint32_t* o = &w.x;
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            o[z] = l == 0.f ? 0u
                                            : pack2<kF>(__uint_as_float(r[y + 2 * z]) * inv, __uint_as_float(r[y + 2 * z + 1]) * inv);
                        if (valid) *reinterpret_cast<uint4*>(dst + (x + y) * 2) = w;
                    }
                }
                if (unit.parts > 1)
                    fp.split.stat[row] = make_float2(m, l);
                else if (valid && p.lse[g])
                    p.lse[g][(int64_t(b) * p.Hl + h) * p.Sq + i] = (m == -INFINITY ? 0.f : m * kLn2) + logf(l);
            }
        }
    }
    // teardown: every MMA has completed (warp 9 drained o_full) and every TMEM access
    // has finished before the columns are freed
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <Fused kF, int kD, Score kScore>
cudaError_t launch(const ForwardParams& p, cudaStream_t stream) {
    const size_t smem = Shape<kD>::kSmem;
    auto kernel = attention_kernel<kF, kD, kScore>;
    // setting it twice is harmless; the cost is a fraction of a microsecond
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const uint32_t units = p.q_tiles * p.a.P * p.a.B * p.a.Hl;
    return launch_overlapped(kernel, p.split.whole + (units - p.split.whole) * p.split.parts, kThreadsA, smem, stream, p);
}

template <Fused kF, int kD>
cudaError_t launch_scored(const ForwardParams& p, cudaStream_t stream) {
    if (p.a.slopes || !(p.a.scale >= 0x1p-120f)) return launch<kF, kD, Score::kAny>(p, stream);
    return p.a.cap != 0.f ? launch<kF, kD, Score::kCap>(p, stream) : launch<kF, kD, Score::kPlain>(p, stream);
}

}  // namespace

cudaError_t launch_attention(const ForwardParams& p, bool bf16, cudaStream_t stream, int* launches) {
    *launches = 0;
    if (p.a.plan) {
        const cudaError_t e = launch_plan(p.a, p.a.plan, false, kAttnPair, stream);
        if (e != cudaSuccess) return e;
        *launches = 1;
    }
    cudaError_t e = p.a.D == 64 ? (bf16 ? launch_scored<Fused::kBF16, 64>(p, stream) : launch_scored<Fused::kFP16, 64>(p, stream))
                                : (bf16 ? launch_scored<Fused::kBF16, 128>(p, stream) : launch_scored<Fused::kFP16, 128>(p, stream));
    if (e != cudaSuccess) return e;
    *launches += 1;
    if (p.split.parts > 1) {
        if ((e = launch_join_forward(p, bf16, stream)) != cudaSuccess) return e;
        *launches += 1;
    }
    return cudaSuccess;
}

cudaError_t read_attention_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
