// kv_attend_tiles.cu -- attention over the paged 8-bit cache for many rows of a key head
// (whole chunks of new tokens): bound by the products, so they run on the 5th-generation
// tensor cores as in attention_forward.cu, in fp16.
//
// A CTA of 512 threads takes two tiles of 128 rows -- row r of a key head is token
// r / shared, query head r % shared of its group -- and a chunk of the keys:
//  * warps 8-11: turn codes into operand tiles.  A thread copies its pieces of 16 codes of the
//    next tile ahead into shared memory and converts the present ones, exactly, to fp16 in the swizzled
//    layout; K relative to the tile's largest page scale, V relative to the largest
//    one so far.  Before that they lay down Q, each row times a power of two
//    (f16_factor).  Keys behind the sequence become zeros, whatever the page holds.
//  * warp 12, one lane: the products, as in the forward kernel.
//  * warps 0-3 and 4-7: softmax, a thread a row.
// TMEM: S0 S1 (128 columns each, P on top of S), O0 O1 (D columns each).
#include "kv_common.cuh"

namespace tfu {

__device__ unsigned g_kv_tiles_status;  // out-of-range lengths, starts, pages
__device__ unsigned g_kv_tiles_waits;   // bounded waits that gave up

namespace {

using namespace dev;

constexpr int kThreadsT = 512;
constexpr uint32_t kHalfTile = kAttnRows * kSwizzleRow;  // 128 rows of 64 elements: 16 KiB
constexpr int kStages = 4;                               // K V K V
constexpr int kInfos = 4;  // the converters are at most two K tiles ahead of the slowest reader

struct TileInfo {
    float k_ref, v_ref;  // scales that the tile's K and V are relative to
    uint32_t bad;        // groups of 16 keys whose page is out of range
};

template <int kD>
struct TilesShape {
    static constexpr uint32_t kTile = kHalfTile * (kD / 64);
    static constexpr int kSlots = kD == 64 ? 4 : 2;              // code tiles under way
    static constexpr uint32_t kSlot = kAttnRows * kD;
    static constexpr size_t kSmem = (2 + kStages) * size_t(kTile) + kSlots * size_t(kSlot) + 2 * kAttnRows * sizeof(float) + kInfos * sizeof(TileInfo) + 512 + 1024;
};

__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return bounded_wait(bar, parity, abort_flag, &g_kv_tiles_waits);
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
    constexpr int kSlots = TilesShape<kD>::kSlots;
    uint8_t* slots = smem + (2 + kStages) * size_t(kTile);
    float* factors = reinterpret_cast<float*>(slots + kSlots * size_t(TilesShape<kD>::kSlot));  // scale / Q's factor, by row
    TileInfo* infos = reinterpret_cast<TileInfo*>(factors + 2 * kAttnRows);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(infos) + 64);
    static_assert(kInfos * sizeof(TileInfo) <= 64, "the barriers follow the tile infos");
    const uint32_t q_smem = smem_u32(smem), ring = q_smem + 2 * kTile;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, q_full = empty0 + 8 * kStages;
    const uint32_t s_full0 = q_full + 8, p_half0 = s_full0 + 16, o_full = p_half0 + 32, info_full0 = o_full + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 8 + kInfos);
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
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        // ---------------- converters
        const uint32_t i = threadIdx.x - 256, slot_smem = smem_u32(slots) + i * 16;
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
        // lane l of eight: the group of keys [key0 + 128 * tile + 16 l, + 16), which lies in one page:
        // whether there is one, where its K codes start (V's at the same offset), its scales
        struct Group {
            int64_t at;  // -1: behind the sequence, or its page is out of range
            float scale[2];
        };
        auto group_of = [&](int tile) {
            Group d{-1, {0.f, 0.f}};
            const int key = key0 + tile * int(kAttnRows) + int(lane % 8) * 16;
            if (tile < n_tiles && key < seq.len) {
                const int x = c.table[int64_t(n) * c.table_stride + uint32_t(key) / c.page];
                if (x >= 0 && uint32_t(x) < c.pages) {
                    const int64_t slot = int64_t(x) * c.Hkv + kh;
                    d.at = (slot * c.page + uint32_t(key) % c.page) * kD;
                    d.scale[0] = c.scales[0][slot];
                    d.scale[1] = c.scales[1][slot];
                } else {
                    atomicOr(&g_kv_tiles_status, 1u);
                }
            }
            return d;
        };
        // piece x of a thread: 16 codes of a key
        constexpr uint32_t kRowsPer = 128 / kPieces;  // keys that a pass of the 128 threads covers
        const uint32_t piece = i % kPieces, key_in = i / kPieces;
        const uint32_t own = key_in % 16 * kD + piece * 16;  // in a group
        // ask for piece x of tile `tile`; only this thread reads what lands in its 16 bytes
        auto ask = [&](int x, int tile, int kv, int64_t at) {
            const uint32_t row = x * kRowsPer + key_in;
            const int64_t from = __shfl_sync(0xffffffffu, at, row / 16);
            const bool there = from >= 0 && int(row) < seq.len - key0 - tile * int(kAttnRows);
            copy_async16(slot_smem + (2 * tile + kv) % kSlots * TilesShape<kD>::kSlot + x * 2048, c.codes[kv] + (there ? from + own : 0), there);
        };
        // step k (tile k / 2; K, then V) into the ring, and the codes of step k + kSlots asked for
        auto convert = [&](uint32_t k, float scale, float ref, int64_t ahead) {
            uint8_t* tile = smem + (2 + k % kStages) * size_t(kTile);
            const __half2 own_factor = __float2half2_rn(scale / ref);
            const uint32_t factor = *reinterpret_cast<const uint32_t*>(&own_factor);
            copy_async_wait<kSlots - 1>();
            const uint8_t* codes = slots + k % kSlots * TilesShape<kD>::kSlot + i * 16;
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                const uint32_t row = x * kRowsPer + key_in, f = __shfl_sync(0xffffffffu, factor, row / 16);
                const uint4 d = *reinterpret_cast<const uint4*>(codes + x * 2048);
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
                ask(x, k / 2 + kSlots / 2, k % 2, ahead);  // the piece has been read
            }
            copy_async_commit();
            fence_async_shared();
        };
        auto largest = [&](float v) {
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        };
        constexpr int kAhead = kSlots / 2;  // tiles
        Group groups[kAhead + 1];  // of tiles j .. j + kAhead
#pragma unroll
        for (int t = 0; t < kAhead; ++t) {
            groups[t] = group_of(t);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
                for (int x = 0; x < kLoads; ++x) ask(x, t, kv, groups[t].at);
                copy_async_commit();
            }
        }
        groups[kAhead] = group_of(kAhead);
        float v_ref = 0x1p-126f;
        for (int j = 0; j < n_tiles; ++j) {
            const Group now = groups[0];
            const int64_t ahead = groups[kAhead].at;
#pragma unroll
            for (int t = 0; t < kAhead; ++t) groups[t] = groups[t + 1];
            groups[kAhead] = group_of(j + 1 + kAhead);
            const float k_ref = fmaxf(largest(now.scale[0]), 0x1p-126f);
            v_ref = fmaxf(v_ref, largest(now.scale[1]));
            const int key = key0 + j * int(kAttnRows) + int(lane % 8) * 16;
            const uint32_t bad = __ballot_sync(0xffffffffu, lane < 8 && now.at < 0 && key < seq.len);
            const uint32_t k = 2 * j;
            auto stage_free = [&](uint32_t k) {
                return __all_sync(0xffffffffu, k < uint32_t(kStages) || wait_for(empty0 + 8 * (k % kStages), (k / kStages - 1) & 1u, abort_flag));
            };
            if (!stage_free(k)) break;
            convert(k, now.scale[0], k_ref, ahead);
            if (i == 0) {
                infos[j % kInfos] = TileInfo{k_ref, v_ref, bad};
                mbar_arrive(info_full0 + 8 * (j % kInfos));
            }
            warp_arrive(full0 + 8 * (k % kStages));
            if (!stage_free(k + 1)) break;
            convert(k + 1, now.scale[1], v_ref, ahead);
            warp_arrive(full0 + 8 * ((k + 1) % kStages));
        }
        copy_async_wait<0>();
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
