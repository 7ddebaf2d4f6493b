// kv_attend_tiles.cu -- attention over the paged 8-bit cache for many rows of a key head
// (whole chunks of new tokens): bound by the products, so they run on the 5th-generation
// tensor cores as in attention_forward.cu, in fp16.
//
// A CTA of 512 threads takes two tiles of 128 rows -- row r of a key head is token
// r / shared, query head r % shared of its group -- and a chunk of the keys:
//  * warp 13: looks up the pages of the tiles to come and copies their codes into a ring in
//    shared memory (bulk copies of a group of 16 keys, which lies in one page).
//  * warps 8-11: turn codes into operand tiles in fp16 and the swizzled layout; K relative
//    to the tile's largest page scale, V relative to the largest one so far.  Exact for scales
//    within 2^15 of that; codes of smaller ones round to multiples of 2^-24 of it.
//    Before that they lay down Q, each row times a power of two (f16_factor).  Keys
//    behind the sequence become zeros, whatever the page holds.
//  * warp 12, one lane: the products, as in the forward kernel.
//  * warps 0-3 and 4-7: softmax, a thread a row.
// TMEM: S0 S1 (128 columns each, P on top of S), O0 O1 (D columns each).
//
// 1560 tokens over 32760 keys, 40 heads, D = 128: 1.01 ms, 1030 TFLOP/s, the matrix pipe busy about half of
// the cycles.  Every 256 rows convert their chunk's codes anew, and the converting warps share issue slots
// with the softmax: without conversion (zeros) the kernel takes 0.85 ms.  Converters that loaded their codes
// themselves waited for them (1.67 ms from registers, 1.20 ms from their own copies ahead).
#include "kv_common.cuh"

namespace tfu {

__device__ unsigned g_kv_tiles_status;  // out-of-range lengths, starts, pages
__device__ unsigned g_kv_tiles_waits;   // bounded waits that gave up

namespace {

using namespace dev;

constexpr int kThreadsT = 512;
constexpr uint32_t kHalfTile = kAttnRows * kSwizzleRow;  // 128 rows of 64 elements: 16 KiB
constexpr int kStages = 3;                               // operand tiles: K V K, V K V, ...
constexpr int kSlots = 4;                                // tiles of codes: K V K V
// Warp 13 is at most kSlots / 2 tiles ahead of the converters, and those at most
// kStages / 2 ahead of the slowest softmax warp.
constexpr int kInfos = 8;

struct TileInfo {
    uint32_t factor[2][8];  // K's and V's groups of 16 keys: the page's scale over the tile's, a pair of fp16
    float k_ref, v_ref;     // scales that the tile's K and V are relative to
    uint32_t bad;           // groups of 16 keys whose page is out of range
    int left;               // keys of the sequence in the tile
};

template <int kD>
struct TilesShape {
    static constexpr uint32_t kTile = kHalfTile * (kD / 64);
    static constexpr uint32_t kSlot = kAttnRows * kD;
    static constexpr size_t kSmem = (2 + kStages) * size_t(kTile) + kSlots * size_t(kSlot) + 2 * kAttnRows * sizeof(float) +
                                    kInfos * sizeof(TileInfo) + 256 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return bounded_wait(bar, parity, abort_flag, &g_kv_tiles_waits);
}

// A bulk copy from device memory, counted in bytes on `bar`.
__device__ __forceinline__ void bulk_copy(uint32_t smem, const void* global, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem), "l"(global), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// 16 values of row `row` from element 16 * piece on, as two swizzled 16-byte chunks.  The
// upper half's lanes store their second chunk first: the halves lie on the same banks.
template <int kD>
__device__ __forceinline__ void store_piece(uint8_t* tile, uint32_t row, uint32_t piece, const uint32_t (&h)[8]) {
    uint8_t* base = tile + piece / 4 * kHalfTile + row * kSwizzleRow;
    const uint32_t chunk = piece % 4 * 2, flip = piece / 4 & 1u;
#pragma unroll
    for (uint32_t x = 0; x < 2; ++x) {
        const uint32_t y = x ^ flip;
        *reinterpret_cast<uint4*>(base + ((chunk + y) ^ (row & 7u)) * 16) =
            y ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(h[0], h[1], h[2], h[3]);
    }
}

template <Fused kF, int kD, Score kScore>
__global__ void __launch_bounds__(kThreadsT, 1) kv_tiles_kernel(const __grid_constant__ KvAttendParams p) {
    constexpr uint32_t kTile = TilesShape<kD>::kTile;
    constexpr uint32_t kPieces = kD / 16;             // pieces of 16 codes in a row
    constexpr int kLoads = kAttnRows * kPieces / 128;  // pieces of a thread in a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr uint32_t kSlot = TilesShape<kD>::kSlot;
    uint8_t* slots = smem + (2 + kStages) * size_t(kTile);
    float* factors = reinterpret_cast<float*>(slots + kSlots * size_t(kSlot));  // scale / Q's factor, by row
    TileInfo* infos = reinterpret_cast<TileInfo*>(factors + 2 * kAttnRows);
    uint64_t* bars = reinterpret_cast<uint64_t*>(infos + kInfos);
    const uint32_t q_smem = smem_u32(smem), ring = q_smem + 2 * kTile, slot_smem = smem_u32(slots);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, q_full = empty0 + 8 * kStages;
    const uint32_t s_full0 = q_full + 8, p_half0 = s_full0 + 16, o_full = p_half0 + 32, info_full0 = o_full + 8;
    const uint32_t code_full0 = info_full0 + 8 * kInfos, code_empty0 = code_full0 + 8 * kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 8 + kInfos + 2 * kSlots);
    static_assert((2 * kStages + 8 + kInfos + 2 * kSlots) * 8 + 8 <= 256, "the barriers' room");
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const KvCache& c = p.c;

    // the chunk, the row tile pair, the key head and the sequence of this CTA
    const uint32_t pairs = (p.row_cap + kAttnPair - 1) / kAttnPair;
    uint32_t u = blockIdx.x;
    const uint32_t chunk = u % p.chunks;
    u /= p.chunks;
    const uint32_t row0 = u % pairs * kAttnPair;
    u /= pairs;
    const uint32_t kh = u % c.Hkv, n = u / c.Hkv;
    grid_dependency_wait();
    const Sequence seq = sequence_of(p, n, &g_kv_tiles_status);
    if (!seq.ok || int(chunk) >= seq.chunks) return;
    const uint32_t rows = uint32_t(seq.tokens) * p.shared;
    if (row0 >= rows) return;
    const int tiles = row0 + kAttnRows < rows ? 2 : 1;
    const int key0 = int(chunk * p.chunk);
    // keys in reach of the last row
    const uint32_t last_row = min(row0 + kAttnPair, rows) - 1;
    const int reach = p.causal ? seq.len - seq.tokens + int(last_row / p.shared) + 1 : seq.len;
    const int key1 = min(reach, key0 + int(p.chunk));
    const int n_tiles = key1 > key0 ? (key1 - key0 + int(kAttnRows) - 1) / int(kAttnRows) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 4);  // a warp each
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(q_full, 4);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full0 + 8 * t, 1);
            mbar_init(p_half0 + 16 * t, 4);  // a warp each
            mbar_init(p_half0 + 16 * t + 8, 4);
        }
        mbar_init(o_full, 1);
        for (int t = 0; t < kInfos; ++t) mbar_init(info_full0 + 8 * t, 1);
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(code_full0 + 8 * s, 1);
            mbar_init(code_empty0 + 8 * s, 4);  // a warp each
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t o_tmem = tmem + 2 * kAttnRows;

    // 512 * 128 registers at launch = 256 * 184 + 128 * 88 + 128 * 56
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 12 && n_tiles > 0 && elect_one()) {
            // ---------------- MMA issuer
            constexpr uint32_t kIdescS = f16_idesc(false, kAttnRows, kAttnRows, false);
            constexpr uint32_t kIdescO = f16_idesc(false, kAttnRows, kD, true);
            const uint32_t q_low = desc_low(q_smem), k_low = desc_low(ring), v_low = desc_low(ring, kHalfTile);
            auto scores = [&](int t, uint32_t s) {
                tc_product<kD, kHalfTile, kHalfTile>(tmem + t * kAttnRows, q_low + t * (kTile >> 4), k_low + s * (kTile >> 4), kIdescS);
                tc_commit(s_full0 + 8 * t);
            };
            auto landed = [&](uint32_t k) { return wait_for(full0 + 8 * (k % kStages), (k / kStages) & 1u, abort_flag); };
            bool ok = wait_for(q_full, 0, abort_flag) && landed(0);
            if (ok) {
                tc_fence_after();
                for (int t = 0; t < tiles; ++t) scores(t, 0);
                tc_commit(empty0);
            }
            for (int i = 0; ok && i < n_tiles; ++i) {
                const uint32_t v = 2 * i + 1, k = v + 1;
                const bool more = i + 1 < n_tiles;
                if (!(ok = landed(v))) break;
                for (int t = 0; t < tiles; ++t) {
                    for (int x = 0; x < 2; ++x) {
                        if (!(ok = wait_for(p_half0 + 16 * t + 8 * x, i & 1u, abort_flag))) break;
                        tc_fence_after();
                        tc_product_ts<kAttnRows / 2>(o_tmem + t * kD, tmem + t * kAttnRows + x * 32,
                                                     v_low + v % kStages * (kTile >> 4) + x * (64 * kSwizzleRow >> 4), kIdescO,
                                                     uint32_t(i | x));
                    }
                    if (!ok) break;
                    if (more) {
                        if (t == 0 && !(ok = landed(k))) break;
                        tc_fence_after();
                        scores(t, k % kStages);
                    }
                }
                if (!ok) break;
                tc_commit(empty0 + 8 * (v % kStages));
                if (more) tc_commit(empty0 + 8 * (k % kStages));
            }
            tc_commit(o_full);
            drain_phase(o_full, 0);  // every MMA of this CTA has completed
        } else if (warp == 13) {
            // ---------------- codes.  Lane l of sixteen has K (l < 8) or V of the group of keys
            // [key0 + 128 * tile + 16 (l % 8), + 16)
            const uint32_t kv = lane / 8 % 2, group = lane % 8;
            struct Group {
                int64_t at;  // where its codes start; -1: behind the sequence, or its page is out of range
                float scale;
            };
            auto group_of = [&](int tile) {
                Group d{-1, 0.f};
                const int key = key0 + tile * int(kAttnRows) + int(group) * 16;
                if (tile < n_tiles && key < seq.len) {
                    const int x = c.table[int64_t(n) * c.table_stride + uint32_t(key) / c.page];
                    if (x >= 0 && uint32_t(x) < c.pages) {
                        const int64_t slot = int64_t(x) * c.Hkv + kh;
                        d.at = (slot * c.page + uint32_t(key) % c.page) * kD;
                        d.scale = c.scales[kv][slot];
                    } else if (lane < 8) {
                        atomicOr(&g_kv_tiles_status, 1u);
                    }
                }
                return d;
            };
            Group now = group_of(0);
            float v_ref = 0x1p-126f;
            uint32_t asked = 0;
            bool ok = true;
            for (int j = 0; ok && j < n_tiles; ++j) {
                const Group next = group_of(j + 1);
                float most = now.scale;
#pragma unroll
                for (int w = 1; w < 8; w <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, w));
                const float k_ref = fmaxf(__shfl_sync(0xffffffffu, most, 0), 0x1p-126f);
                v_ref = fmaxf(v_ref, __shfl_sync(0xffffffffu, most, 8));
                const int left = min(seq.len - key0 - j * int(kAttnRows), int(kAttnRows));
                const uint32_t bad = __ballot_sync(0xffffffffu, lane < 8 && now.at < 0 && int(group) * 16 < left);
                const uint32_t bytes = now.at < 0 ? 0 : min(left - int(group) * 16, 16) * kD;
#pragma unroll
                for (uint32_t side = 0; side < 2; ++side) {
                    const uint32_t k = 2 * j + side, s = k % kSlots;
                    ok = k < uint32_t(kSlots) || wait_for(code_empty0 + 8 * s, (k / kSlots - 1) & 1u, abort_flag);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const bool own = lane < 16 && kv == side;
                    if (side == 0) {
                        TileInfo& info = infos[j % kInfos];
                        if (lane < 16) {
                            const __half2 f = __float2half2_rn(now.scale / (kv == 0 ? k_ref : v_ref));
                            info.factor[kv][group] = *reinterpret_cast<const uint32_t*>(&f);
                        }
                        if (lane == 0) {
                            info.k_ref = k_ref;
                            info.v_ref = v_ref;
                            info.bad = bad;
                            info.left = left;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(info_full0 + 8 * (j % kInfos));
                    }
                    const uint32_t total = __reduce_add_sync(0xffffffffu, own ? bytes : 0);
                    if (lane == 0) mbar_expect_tx(code_full0 + 8 * s, total);
                    __syncwarp();
                    if (own && bytes) bulk_copy(slot_smem + s * kSlot + group * 16 * kD, c.codes[kv] + now.at, bytes, code_full0 + 8 * s);
                    asked = k + 1;
                }
                now = next;
            }
            __syncwarp();
            for (uint32_t k = asked > kSlots ? asked - kSlots : 0; k < asked; ++k)
                drain_phase(code_full0 + 8 * (k % kSlots), (k / kSlots) & 1u);
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        // ---------------- converters
        const uint32_t i = threadIdx.x - 256;
        if (n_tiles > 0) {
            for (int t = 0; t < tiles; ++t) {  // Q: a row a thread
                const uint32_t r = row0 + t * kAttnRows + i;
                const bool in = r < rows;
                const uint32_t token = in ? r / p.shared : 0, head = kh * p.shared + (in ? r % p.shared : 0);
                const uint4* src = reinterpret_cast<const uint4*>(p.q.base[head / p.Hl] + (seq.s0 + token) * p.q.t +
                                                                  int64_t(head % p.Hl) * p.q.h);
                float most = 0.f;
#pragma unroll
                for (int x = 0; x < kD / 8; ++x) {
                    const uint4 w = in ? src[x] : make_uint4(0, 0, 0, 0);
                    const uint32_t* v = &w.x;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float a, b;
                        unpack2<kF>(v[y], a, b);
                        most = fmaxf(most, fmaxf(fabsf(a), fabsf(b)));
                    }
                }
                const float up = f16_factor(most);
                factors[t * kAttnRows + i] = p.scale / up;
#pragma unroll 2
                for (uint32_t x = 0; x < kPieces; ++x) {
                    uint32_t h[8];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint4 w = in ? src[2 * x + z] : make_uint4(0, 0, 0, 0);
                        const uint32_t* v = &w.x;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            float a, b;
                            unpack2<kF>(v[y], a, b);
                            h[4 * z + y] = pack2<Fused::kFP16>(a * up, b * up);
                        }
                    }
                    store_piece<kD>(smem + t * kTile, i, x, h);
                }
            }
            fence_async_shared();
            warp_arrive(q_full);
        }
        // a thread's piece x: 16 codes of key x * kRowsPer + i / kPieces of the tile
        constexpr uint32_t kRowsPer = 128 / kPieces;  // keys that a pass of the 128 threads covers
        const uint32_t piece = i % kPieces, key_in = i / kPieces;
        for (uint32_t k = 0; k < 2 * uint32_t(n_tiles); ++k) {  // K of tile k / 2, then V
            bool ok = wait_for(code_full0 + 8 * (k % kSlots), (k / kSlots) & 1u, abort_flag);
            ok = ok && (k < uint32_t(kStages) || wait_for(empty0 + 8 * (k % kStages), (k / kStages - 1) & 1u, abort_flag));
            if (!__all_sync(0xffffffffu, ok)) break;
            const TileInfo& info = infos[k / 2 % kInfos];
            const int left = info.left;
            const uint32_t bad = info.bad;
            const bool whole = left == int(kAttnRows) && bad == 0;
            uint8_t* tile = smem + (2 + k % kStages) * size_t(kTile);
            const uint8_t* codes = slots + k % kSlots * kSlot + i * 16;
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                const uint32_t row = x * kRowsPer + key_in, f = info.factor[k % 2][row / 16];
                uint4 d = *reinterpret_cast<const uint4*>(codes + x * 2048);
                if (!whole && (int(row) >= left || (bad >> (row / 16)) & 1u)) d = make_uint4(0, 0, 0, 0);
                const uint32_t* w = &d.x;
                uint32_t h[8];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t v = to_f16x2(w[y] >> (16 * z));
                        const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&f));
                        h[2 * y + z] = *reinterpret_cast<const uint32_t*>(&r);
                    }
                }
                store_piece<kD>(tile, row, piece, h);
            }
            fence_async_shared();
            warp_arrive(full0 + 8 * (k % kStages));
            warp_arrive(code_empty0 + 8 * (k % kSlots));
        }
    } else {
        // ---------------- softmax: a thread per row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const uint32_t t = warp / 4, quarter = warp % 4, at = t * kAttnRows + quarter * 32 + lane;
        const uint32_t r = row0 + at;
        const bool valid = r < rows;
        const uint32_t token = valid ? r / p.shared : 0, head = kh * p.shared + (valid ? r % p.shared : 0);
        const uint32_t lane_base = (quarter * 32u) << 16;
        const uint32_t s_tmem = tmem + t * kAttnRows + lane_base, o_row = o_tmem + t * kD + lane_base;
        const int pos = seq.len - seq.tokens + int(token);
        const int bound = !valid ? 0 : p.causal ? pos + 1 : seq.len;
        const float slope = kScore == Score::kAny && p.slopes ? p.slopes[head] : 0.f;
        // positions of the warp's rows (those behind the last row count as its first one)
        const int pos_lo = __reduce_min_sync(0xffffffffu, pos), pos_hi = __reduce_max_sync(0xffffffffu, pos);
        float m = -INFINITY, l = 0.f, v_ref = 0x1p-126f, factor = 0.f;
        bool ok = true;
        for (int j = 0; j < (int(t) < tiles ? n_tiles : 0); ++j) {
            ok = wait_for(s_full0 + 8 * t, j & 1u, abort_flag) &&
                 wait_for(info_full0 + 8 * (j % kInfos), (j / kInfos) & 1u, abort_flag);
            if (j == 0) {
                ok = ok && wait_for(q_full, 0, abort_flag);  // the rows' factors
                factor = factors[at];
            }
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const TileInfo info = infos[j % kInfos];
            float s[128];
            load_row<128>(s_tmem, s);
            const int j0 = key0 + j * int(kAttnRows);
            const float f = factor * info.k_ref;
            const float down = v_ref / info.v_ref;
            v_ref = info.v_ref;
            const bool whole = __all_sync(0xffffffffu, j0 + int(kAttnRows) <= bound && info.bad == 0);
            if (kScore == Score::kCap && whole &&
                fold_capped_tile<Fused::kFP16, kD, false>(s, f, p.cap, down, j > 0, m, l, s_tmem, o_row, p_half0 + 16 * t))
                continue;
            if (kScore != Score::kPlain)
                finish_scores<kScore>(s, f, p.cap, slope, float(pos - j0), bias_side(pos_lo, pos_hi - pos_lo + 1, j0, int(kAttnRows), p.causal));
            const float to_z = kScore == Score::kPlain ? fmaxf(f * kLog2e, 0x1p-126f) : 1.0f;
            if (!whole) {
                uint32_t bits[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    bits[x] = bound_bits(bound, j0 + 32 * x);
                    if ((info.bad >> (2 * x)) & 1u) bits[x] &= 0xffff0000u;
                    if ((info.bad >> (2 * x)) & 2u) bits[x] &= 0x0000ffffu;
                }
#pragma unroll
                for (int x = 0; x < 128; ++x) s[x] = (bits[x / 32] >> (x % 32)) & 1u ? s[x] : -INFINITY;
            }
            fold_tile<Fused::kFP16, kD>(s, to_z, down, j > 0, m, l, s_tmem, o_row, p_half0 + 16 * t);
        }
        if (int(t) < tiles && ok) {
            if (n_tiles > 0) ok = wait_for(o_full, 0, abort_flag);
            if (__all_sync(0xffffffffu, ok) && !*abort_flag) {
                tc_fence_after();
                const bool joined = seq.chunks > 1;
                const int64_t slot = ((int64_t(n) * c.Hkv + kh) * p.row_cap + (valid ? r : 0)) * p.chunks + chunk;
                const float inv = joined ? v_ref : l > 0.f ? v_ref / l : (l == 0.f ? 0.f : l);
                uint8_t* dst = joined ? reinterpret_cast<uint8_t*>(p.part + slot * kD)
                                      : p.out.base[head / p.Hl] + (seq.s0 + token) * p.out.t + int64_t(head % p.Hl) * p.out.h;
                if (n_tiles > 0 || !joined) {
#pragma unroll 1
                    for (int x = 0; x < kD; x += 32) {
                        uint32_t o[32];
                        if (n_tiles > 0) {
                            tc_ld32(o_row + x, o);
                            tc_wait_ld();
                            tc_landed(o);
                        }
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            o[y] = n_tiles == 0 || (l == 0.f && !joined) ? 0u : __float_as_uint(__uint_as_float(o[y]) * inv);
                        if (!valid) continue;
                        if (joined) {
#pragma unroll
                            for (int y = 0; y < 32; y += 4)
                                *reinterpret_cast<uint4*>(dst + (x + y) * 4) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
                        } else {
#pragma unroll
                            for (int y = 0; y < 32; y += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    w[z] = pack2<kF>(__uint_as_float(o[y + 2 * z]), __uint_as_float(o[y + 2 * z + 1]));
                                *reinterpret_cast<uint4*>(dst + (x + y) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                }
                if (valid && joined) {
                    p.part_stat[slot] = make_float2(m, l);
                } else if (valid && p.lse[head / p.Hl]) {
                    p.lse[head / p.Hl][int64_t(head % p.Hl) * p.T + seq.s0 + token] = (m == -INFINITY ? 0.f : m * kLn2) + logf(l);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <Fused kF, int kD, Score kScore>
cudaError_t launch(const KvAttendParams& p, cudaStream_t stream) {
    auto kernel = kv_tiles_kernel<kF, kD, kScore>;
    constexpr size_t smem = TilesShape<kD>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const uint32_t pairs = (p.row_cap + kAttnPair - 1) / kAttnPair;
    return launch_overlapped(kernel, p.chunks * pairs * p.c.Hkv * p.c.N, kThreadsT, smem, stream, p);
}

template <Fused kF, int kD>
cudaError_t launch_scored(const KvAttendParams& p, cudaStream_t stream) {
    if (p.slopes || !(p.scale > 0.f)) return launch<kF, kD, Score::kAny>(p, stream);
    return p.cap != 0.f ? launch<kF, kD, Score::kCap>(p, stream) : launch<kF, kD, Score::kPlain>(p, stream);
}

}  // namespace

cudaError_t launch_kv_tiles(const KvAttendParams& p, bool bf16, cudaStream_t stream) {
    if (p.c.D == 64) return bf16 ? launch_scored<Fused::kBF16, 64>(p, stream) : launch_scored<Fused::kFP16, 64>(p, stream);
    return bf16 ? launch_scored<Fused::kBF16, 128>(p, stream) : launch_scored<Fused::kFP16, 128>(p, stream);
}

cudaError_t read_kv_tiles_status(unsigned* out, unsigned* waits, bool clear) {
    const unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv_tiles_status, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(waits, g_kv_tiles_waits, sizeof(unsigned));
    if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_kv_tiles_status, &zero, sizeof(unsigned));
    if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_kv_tiles_waits, &zero, sizeof(unsigned));
    return e;
}

}  // namespace tfu
