// kv_attend.cu -- attention of each sequence's newest tokens over the paged 8-bit cache.
//
// The scores and the softmax are those of attention_common.cuh with K = code * scale and
// V = code * scale of the page's head; key j of a sequence is in page j / page_size of its
// table row.  Few rows (tokens times shared heads) for each key: the bound is
// reading the codes once, 2 D bytes a key and head.
//
// kv_decode_kernel: a CTA of 4 warps takes 8 or 16 rows of one key head and a chunk of the
// keys; each warp walks its own part in steps of 16 keys, copied ahead into a ring of its own in
// shared memory, and the warps join at the end.  The products are mma.m16n8k16 in the
// transposed form, S^T = K Q^T and O^T = V^T P^T: 16 keys or dimensions fill the tile's 16
// rows and the few query rows its 8 columns.  The order of the summed dimensions is free, so
// lane (g, t) takes 16 consecutive bytes of keys g and g + 8 for S^T, and of keys 2t, 2t+1,
// 2t+8, 2t+9 for O^T, where bytes of two keys are paired by a permute; codes become fp16
// exactly (e4m3 fits), and P^T comes from S^T by two 8 x 8 transposes.
//  * Q in fp16 times a power of two for each row that puts its largest value at 2^14: exact
//    but for values 2^28 below it; the factor goes into the score's scale.
//  * P in fp16 times the page's V scale relative to the largest one so far (O is rescaled
//    when that grows), so O sums codes times weights of at most 2^8.
//  * The reference m of a row follows its maximum when that outgrows it by 2^8.
//
// 24 sequences of up to 65536 keys, 4 key heads, 4 query heads each, D = 128: 140 us, 6.0 TB/s of codes (a
// plain copy 6.8).  What it took: codes loaded into registers a step ahead 302 us; through
// the ring, three steps ahead, 174; transposed products, whose tile the keys fill, 140.  64 sequences of up to 8192
// keys, 8 query heads to a key head, capped: 64 us, 4.3 TB/s, the short sequences' chunks end early.
#include "kv_common.cuh"

namespace tfu {

__device__ unsigned g_kv_attend_status;

namespace {

using namespace dev;

constexpr int kWarps = 4;
constexpr int kStep = 16;      // keys of a warp's step; a page is a whole number of steps
constexpr int kRing = 4;       // steps of a warp in shared memory: one computed, three on their way

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A step in shared memory: 16 keys of K, then of V, rows of kD codes in 16-byte chunks that are
// swapped about so that the fragments' reads meet no bank twice: K by rows g with chunks
// t, V by rows 2t with chunks g.
template <int kD>
struct StepLayout {
    static constexpr uint32_t kHalf = kStep * kD, kBytes = 2 * kHalf;
    static constexpr uint32_t kChunks = kD / 16;  // of a row
    __device__ static __forceinline__ uint32_t k(uint32_t row, uint32_t chunk) {
        if constexpr (kD == 128) return row * 128 + ((chunk ^ ((row & 1u) * 4 | (row >> 1 & 3u))) * 16);
        return row * 64 + chunk * 16;
    }
    __device__ static __forceinline__ uint32_t v(uint32_t row, uint32_t chunk) {
        if constexpr (kD == 128) return kHalf + row * 128 + ((chunk ^ (row >> 1 & 3u) * 2) * 16);
        return kHalf + (row >> 1) * 128 + ((((row & 1u) * 4 + chunk) ^ (row >> 1 & 3u) * 2) * 16);
    }
};

// What a step needs beside its codes.
struct StepInfo {
    float ks, vs;
    int keys;  // visible ones; 0: its page is out of range
};

// The 8 x 8 matrix of 16-bit values whose row g the lanes (g, t) hold in pairs, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// kTiles: tiles of 8 rows.
template <Fused kF, int kD, int kTiles>
__global__ void __launch_bounds__(kWarps * 32, 3) kv_decode_kernel(const __grid_constant__ KvAttendParams p) {
    using Layout = StepLayout<kD>;
    constexpr int kSteps = kD / 16;   // k-steps of K Q^T
    constexpr int kTilesO = kD / 16;  // tiles of 16 dimensions of V^T P^T
    constexpr int kRows = 8 * kTiles;
    // the rings; at the end the warps' sums
    extern __shared__ __align__(16) uint8_t rings[];
    auto o_all = reinterpret_cast<float(*)[kRows][kD + 4]>(rings);
    static_assert(sizeof(float) * kRows * (kD + 4) <= kRing * Layout::kBytes, "the sums take the rings' place");
    __shared__ float m_all[kWarps][kRows], l_all[kWarps][kRows];
    __shared__ StepInfo infos[kWarps][kRing];
    grid_dependency_wait();
    const KvCache& c = p.c;
    const uint32_t n = blockIdx.z, row_tiles = gridDim.y / c.Hkv, kh = blockIdx.y / row_tiles;
    const uint32_t row0 = blockIdx.y % row_tiles * kRows;
    const Sequence seq = sequence_of(p, n, &g_kv_attend_status);
    if (!seq.ok || int(blockIdx.x) >= seq.chunks) return;
    const uint32_t rows = uint32_t(seq.tokens) * p.shared;
    if (row0 >= rows) return;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;

    const int lo = int(blockIdx.x * p.chunk), hi = min(seq.len, lo + int(p.chunk));
    const int steps = (hi - lo + kStep - 1) / kStep, per = (steps + kWarps - 1) / kWarps;
    const int first = lo + int(warp) * per * kStep, last = min(hi, first + per * kStep);

    // the pages of 32 steps, one a lane, and of the 32 after them
    struct Pages {
        int id;
        float ks, vs;
    };
    auto pages = [&](int j) {
        Pages d{-1, 0.f, 0.f};
        const int key = j + int(lane) * kStep;
        if (key < last) {
            const int id = c.table[int64_t(n) * c.table_stride + uint32_t(key) / c.page];
            if (id >= 0 && uint32_t(id) < c.pages) {
                d.id = id;
                d.ks = c.scales[0][int64_t(id) * c.Hkv + kh];
                d.vs = c.scales[1][int64_t(id) * c.Hkv + kh];
            } else {
                atomicOr(&g_kv_attend_status, 1u);
            }
        }
        return d;
    };
    const uint32_t ring = smem_u32(rings) + warp * (kRing * Layout::kBytes);
    uint32_t k_to[Layout::kHalf / 512], v_to[Layout::kHalf / 512];  // where this lane's pieces of a step go
#pragma unroll
    for (uint32_t x = 0; x < Layout::kHalf / 512; ++x) {
        const uint32_t piece = x * 32 + lane;
        k_to[x] = Layout::k(piece / Layout::kChunks, piece % Layout::kChunks);
        v_to[x] = Layout::v(piece / Layout::kChunks, piece % Layout::kChunks);
    }
    Pages now = pages(first), next = pages(first + 32 * kStep);
    auto load = [&](int s) {  // step s of this warp; always one group
        const int j = first + s * kStep;
        if (j < last) {
            if (s > 0 && s % 32 == 0) {
                now = next;
                next = pages(j + 32 * kStep);
            }
            const int id = __shfl_sync(0xffffffffu, now.id, s % 32);
            if (int(lane) == s % 32) infos[warp][s % kRing] = StepInfo{now.ks, now.vs, id < 0 ? 0 : min(kStep, last - j)};
            if (id >= 0) {
                const int64_t at = ((int64_t(id) * c.Hkv + kh) * c.page + (uint32_t(j) & (c.page - 1))) * kD + lane * 16;
                const uint32_t to = ring + s % kRing * Layout::kBytes;
#pragma unroll
                for (uint32_t x = 0; x < Layout::kHalf / 512; ++x) {
                    copy_async16(to + k_to[x], c.codes[0] + at + x * 512);
                    copy_async16(to + v_to[x], c.codes[1] + at + x * 512);
                }
            }
        }
        copy_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) load(s);

    // Q: this lane's part of row 8y + g in fragments; what belongs to the score columns, rows
    // 8y + 2t + e: factors, bounds, positions
    uint32_t qf[kTiles][kSteps][2];
    float factor[kTiles][2], slope[kTiles][2];
    int bound[kTiles][2], pos[kTiles][2];
#pragma unroll
    for (int y = 0; y < kTiles; ++y) {
        const uint32_t r = row0 + 8 * y + g;
        const bool in = r < rows;
        const uint32_t token = in ? r / p.shared : 0, head = kh * p.shared + (in ? r % p.shared : 0);
        const uint8_t* src = p.q.base[head / p.Hl] + (seq.s0 + token) * p.q.t + int64_t(head % p.Hl) * p.q.h;
        uint2 w[kSteps];
        float most = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            w[s] = in ? *reinterpret_cast<const uint2*>(src + 2 * (s / 4 * 64 + t * 16 + s % 4 * 4)) : make_uint2(0, 0);
            float f[4];
            unpack2<kF>(w[s].x, f[0], f[1]);
            unpack2<kF>(w[s].y, f[2], f[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) most = fmaxf(most, fabsf(f[x]));
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const float up = f16_factor(most), own = p.scale / up;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            float f[4];
            unpack2<kF>(w[s].x, f[0], f[1]);
            unpack2<kF>(w[s].y, f[2], f[3]);
            qf[y][s][0] = pack2<Fused::kFP16>(f[0] * up, f[1] * up);
            qf[y][s][1] = pack2<Fused::kFP16>(f[2] * up, f[3] * up);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            factor[y][e] = __shfl_sync(0xffffffffu, own, (2 * t + e) * 4);
            const uint32_t rc = row0 + 8 * y + 2 * t + e;
            const bool col = rc < rows;
            pos[y][e] = seq.len - seq.tokens + int(col ? rc / p.shared : 0);
            bound[y][e] = !col ? 0 : p.causal ? pos[y][e] + 1 : seq.len;
            slope[y][e] = p.slopes && col ? p.slopes[kh * p.shared + rc % p.shared] * kLog2e : 0.f;
        }
    }
    int least = seq.len;  // keys below it are visible to every row
#pragma unroll
    for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) least = min(least, bound[y][e] == 0 ? least : bound[y][e]);
    least = __reduce_min_sync(0xffffffffu, least);

    float o[kTiles][kTilesO][4], m[kTiles][2], l[kTiles][2], v_ref = 0x1p-126f;
#pragma unroll
    for (int y = 0; y < kTiles; ++y) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[y][e] = -INFINITY;
            l[y][e] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kTilesO; ++s)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[y][s][x] = 0.f;
    }

    auto step = [&](int number) {
        const int j = first + number * kStep;
        const StepInfo d = infos[warp][number % kRing];
        if (d.keys == 0) return;
        const uint8_t* codes = rings + warp * (kRing * Layout::kBytes) + number % kRing * Layout::kBytes;
        // s[y][2x + e]: key j + 8x + g, row 8y + 2t + e
        float s[kTiles][4];
#pragma unroll
        for (int y = 0; y < kTiles; ++y) s[y][0] = s[y][1] = s[y][2] = s[y][3] = 0.f;
#pragma unroll
        for (int z = 0; z < kD / 64; ++z) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(codes + Layout::k(g, 4 * z + t)),
                        u4 = *reinterpret_cast<const uint4*>(codes + Layout::k(g + 8, 4 * z + t));
            const uint32_t* w = &w4.x;
            const uint32_t* u = &u4.x;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t a[4] = {to_f16x2(w[x]), to_f16x2(u[x]), to_f16x2(w[x] >> 16), to_f16x2(u[x] >> 16)};
#pragma unroll
                for (int y = 0; y < kTiles; ++y) mma_f16(s[y], a, qf[y][4 * z + x][0], qf[y][4 * z + x][1]);
            }
        }
        const bool whole = j + kStep <= least;  // d.keys is kStep then
        bool up = false;
        float top[kTiles][2];
#pragma unroll
        for (int y = 0; y < kTiles; ++y) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = factor[y][e] * d.ks;
                float a = s[y][e], b = s[y][2 + e];
                if (p.cap != 0.f) {
                    const float to_x = f / p.cap, to_z = p.cap * kLog2e;
                    a *= to_x;
                    b *= to_x;
                    if (__all_sync(0xffffffffu, fmaxf(fabsf(a), fabsf(b)) <= kTanhNear)) {
                        const uint64_t v = f2_pack(a, b);
                        f2_unpack(f2_mul(f2_mul(v, f2_pack(to_z, to_z)), tanh_over_x(f2_mul(v, v))), a, b);
                    } else {
                        a = to_z * tanh_wide(a);
                        b = to_z * tanh_wide(b);
                    }
                } else {
                    a *= f * kLog2e;
                    b *= f * kLog2e;
                }
                if (p.slopes) {
                    a = fmaf(-slope[y][e], fabsf(float(pos[y][e] - (j + int(g)))), a);
                    b = fmaf(-slope[y][e], fabsf(float(pos[y][e] - (j + 8 + int(g)))), b);
                }
                if (!whole) {
                    a = j + int(g) < bound[y][e] ? a : -INFINITY;
                    b = j + 8 + int(g) < bound[y][e] ? b : -INFINITY;
                }
                s[y][e] = a;
                s[y][2 + e] = b;
                top[y][e] = fmaxf(a, b);
                up |= top[y][e] > m[y][e] + kSlack;
            }
        }
        if (__any_sync(0xffffffffu, up) || d.vs > v_ref) {  // the same for the whole warp
            const float v_new = fmaxf(v_ref, d.vs), down = v_ref / v_new;
            v_ref = v_new;
#pragma unroll
            for (int y = 0; y < kTiles; ++y) {
                float shrink[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float most = top[y][e];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, w));
                    shrink[e] = 1.f;
                    if (most > m[y][e] + kSlack) {
                        shrink[e] = ex2(m[y][e] - most);
                        m[y][e] = most;
                        l[y][e] *= shrink[e];
                    }
                    shrink[e] *= down;
                }
#pragma unroll
                for (int z = 0; z < kTilesO; ++z) {
                    o[y][z][0] *= shrink[0], o[y][z][1] *= shrink[1];
                    o[y][z][2] *= shrink[0], o[y][z][3] *= shrink[1];
                }
            }
        }
        const float fv = d.vs / v_ref;
        uint32_t pf[kTiles][2];  // P^T: keys 2t, 2t + 1 (+ 8) of row 8y + g
#pragma unroll
        for (int y = 0; y < kTiles; ++y) {
            const float b0 = m[y][0] == -INFINITY ? 0.f : m[y][0], b1 = m[y][1] == -INFINITY ? 0.f : m[y][1];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float e0 = ex2(s[y][2 * x] - b0), e1 = ex2(s[y][2 * x + 1] - b1);
                l[y][0] += e0;
                l[y][1] += e1;
                pf[y][x] = transpose8(pack2<Fused::kFP16>(e0 * fv, e1 * fv));
            }
        }
        uint32_t v[4][kD / 32];  // keys 2t, 2t + 1, 2t + 8, 2t + 9: kD / 8 codes from dimension g * kD / 8 on
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t row = 2 * t + x % 2 + x / 2 * 8;
            if constexpr (kD == 128)
                *reinterpret_cast<uint4*>(v[x]) = *reinterpret_cast<const uint4*>(codes + Layout::v(row, g));
            else
                *reinterpret_cast<uint2*>(v[x]) = *reinterpret_cast<const uint2*>(codes + Layout::v(row, g / 2) + g % 2 * 8);
        }
        if (d.keys < kStep) {  // what lies behind the sequence may be anything
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (2 * int(t) + x % 2 + x / 2 * 8 >= d.keys) {
#pragma unroll
                    for (int z = 0; z < kD / 32; ++z) v[x][z] = 0;
                }
        }
        // V^T: tile z of dimensions g * kD / 8 + 2z (its rows g) and + 1 (rows g + 8)
#pragma unroll
        for (int z = 0; z < kD / 32; ++z) {
            const uint32_t lo0 = __byte_perm(v[0][z], v[1][z], 0x5140), hi0 = __byte_perm(v[0][z], v[1][z], 0x7362);
            const uint32_t lo1 = __byte_perm(v[2][z], v[3][z], 0x5140), hi1 = __byte_perm(v[2][z], v[3][z], 0x7362);
            const uint32_t a[4] = {to_f16x2(lo0), to_f16x2(lo0 >> 16), to_f16x2(lo1), to_f16x2(lo1 >> 16)};
            const uint32_t b[4] = {to_f16x2(hi0), to_f16x2(hi0 >> 16), to_f16x2(hi1), to_f16x2(hi1 >> 16)};
#pragma unroll
            for (int y = 0; y < kTiles; ++y) {
                mma_f16(o[y][2 * z], a, pf[y][0], pf[y][1]);
                mma_f16(o[y][2 * z + 1], b, pf[y][0], pf[y][1]);
            }
        }
    };

    const int mine = first < last ? (last - first + kStep - 1) / kStep : 0;
    for (int s = 0; s < mine; ++s) {
        copy_async_wait<kRing - 2>();
        __syncwarp();  // every lane's copies of step s have landed; step s - 1 has been read
        load(s + kRing - 1);
        step(s);
    }
    copy_async_wait<0>();
    __syncthreads();  // the sums take the rings' place

    // join the warps
#pragma unroll
    for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) l[y][e] += __shfl_xor_sync(0xffffffffu, l[y][e], w);
            const uint32_t row = 8 * y + 2 * t + e;
            if (g == 0) {
                m_all[warp][row] = m[y][e];
                l_all[warp][row] = l[y][e];
            }
#pragma unroll
            for (int z = 0; z < kTilesO; z += 2)
                *reinterpret_cast<float4*>(&o_all[warp][row][g * (kD / 8) + 2 * z]) =
                    make_float4(o[y][z][e] * v_ref, o[y][z][2 + e] * v_ref, o[y][z + 1][e] * v_ref, o[y][z + 1][2 + e] * v_ref);
        }
    __syncthreads();
    for (uint32_t x = threadIdx.x; x < kRows * (kD / 8); x += kWarps * 32) {
        const uint32_t row = x / (kD / 8), d = x % (kD / 8) * 8, r = row0 + row;
        if (r >= rows) break;
        float top = -INFINITY, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_all[w][row]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // nothing visible: 0, or the NaN of a row whose scores are
            const float f = m_all[w][row] == -INFINITY ? 0.f * l_all[w][row] : ex2(m_all[w][row] - top);
            if (f == 0.f) continue;
            sum = fmaf(f, l_all[w][row], sum);
#pragma unroll
            for (int y = 0; y < 8; ++y) acc[y] = fmaf(f, o_all[w][row][d + y], acc[y]);
        }
        if (seq.chunks > 1) {
            const int64_t at = ((int64_t(n) * c.Hkv + kh) * p.row_cap + r) * p.chunks + blockIdx.x;
            float4* dst = reinterpret_cast<float4*>(p.part + at * kD + d);
            dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            if (d == 0) p.part_stat[at] = make_float2(top, sum);
            continue;
        }
        const uint32_t token = r / p.shared, head = kh * p.shared + r % p.shared;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        uint8_t* dst = p.out.base[head / p.Hl] + (seq.s0 + token) * p.out.t + int64_t(head % p.Hl) * p.out.h + d * 2;
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<kF>(acc[0] * inv, acc[1] * inv), pack2<kF>(acc[2] * inv, acc[3] * inv),
                                                    pack2<kF>(acc[4] * inv, acc[5] * inv), pack2<kF>(acc[6] * inv, acc[7] * inv));
        float* lse = p.lse[head / p.Hl];
        if (lse && d == 0) lse[int64_t(head % p.Hl) * p.T + seq.s0 + token] = (top == -INFINITY ? 0.f : top * kLn2) + logf(sum);
    }
}

// Joins the chunks of a row: four warps a row, which take every fourth chunk; kJoinAhead chunks
// of a warp are on their way at a time.
constexpr int kJoinWarps = 4, kJoinAhead = 8;
template <Fused kF, int kD>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_join_kernel(const __grid_constant__ KvAttendParams p) {
    constexpr int kPer = kD / 32;
    __shared__ float o_all[kJoinWarps][kD], l_all[kJoinWarps];
    grid_dependency_wait();
    const KvCache& c = p.c;
    const uint32_t n = blockIdx.z, kh = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32, r = blockIdx.x;
    const Sequence seq = sequence_of(p, n, &g_kv_attend_status);
    if (!seq.ok || seq.chunks <= 1 || r >= uint32_t(seq.tokens) * p.shared) return;
    const int64_t at = ((int64_t(n) * c.Hkv + kh) * p.row_cap + r) * p.chunks;
    float top = -INFINITY;
    for (int x = int(lane); x < seq.chunks; x += 32) top = fmaxf(top, p.part_stat[at + x].x);
#pragma unroll
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    float sum = 0.f, acc[kPer] = {};
    for (int x0 = int(warp); x0 < seq.chunks; x0 += kJoinWarps * kJoinAhead) {
        float v[kJoinAhead][kPer];
        float2 st[kJoinAhead];
#pragma unroll
        for (int a = 0; a < kJoinAhead; ++a) {
            const int x = x0 + a * kJoinWarps;
            st[a] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int y = 0; y < kPer; ++y) v[a][y] = 0.f;
            if (x < seq.chunks) {
                st[a] = p.part_stat[at + x];
                const float* src = p.part + (at + x) * kD + lane * kPer;
                if constexpr (kPer == 4)
                    *reinterpret_cast<float4*>(v[a]) = *reinterpret_cast<const float4*>(src);
                else
                    *reinterpret_cast<float2*>(v[a]) = *reinterpret_cast<const float2*>(src);
            }
        }
#pragma unroll
        for (int a = 0; a < kJoinAhead; ++a) {
            const float f = st[a].x == -INFINITY ? 0.f * st[a].y : ex2(st[a].x - top);
            if (f == 0.f) continue;  // what such a chunk left is not defined
            sum = fmaf(f, st[a].y, sum);
#pragma unroll
            for (int y = 0; y < kPer; ++y) acc[y] = fmaf(f, v[a][y], acc[y]);
        }
    }
#pragma unroll
    for (int y = 0; y < kPer; ++y) o_all[warp][lane * kPer + y] = acc[y];
    if (lane == 0) l_all[warp] = sum;
    __syncthreads();
    if (threadIdx.x * 2 >= kD) return;
    const uint32_t token = r / p.shared, head = kh * p.shared + r % p.shared, d = threadIdx.x * 2;
    float o0 = 0.f, o1 = 0.f;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        sum += l_all[w];
        o0 += o_all[w][d];
        o1 += o_all[w][d + 1];
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    uint8_t* dst = p.out.base[head / p.Hl] + (seq.s0 + token) * p.out.t + int64_t(head % p.Hl) * p.out.h + d * 2;
    *reinterpret_cast<uint32_t*>(dst) = pack2<kF>(o0 * inv, o1 * inv);
    float* lse = p.lse[head / p.Hl];
    if (lse && d == 0) lse[int64_t(head % p.Hl) * p.T + seq.s0 + token] = (top == -INFINITY ? 0.f : top * kLn2) + logf(sum);
}

template <typename... Args>
cudaError_t launch_grid(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <Fused kF, int kD>
cudaError_t launch(const KvAttendParams& p, cudaStream_t stream, int* launches) {
    const uint32_t rows = p.max_tokens * p.shared;
    cudaError_t e;
    if (p.tiles) {
        e = launch_kv_tiles(p, kF == Fused::kBF16, stream);
    } else {
        constexpr size_t smem = size_t(kWarps) * kRing * StepLayout<kD>::kBytes;
        auto kernel = p.unit == 8 ? kv_decode_kernel<kF, kD, 1> : kv_decode_kernel<kF, kD, 2>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        e = launch_grid(kernel, dim3(p.chunks, p.c.Hkv * (p.row_cap / p.unit), p.c.N), kWarps * 32, smem, stream, p);
    }
    if (e != cudaSuccess) return e;
    *launches += 1;
    if (p.chunks > 1) {
        e = launch_grid(kv_join_kernel<kF, kD>, dim3(rows, p.c.Hkv, p.c.N), kJoinWarps * 32, 0, stream, p);
        if (e != cudaSuccess) return e;
        *launches += 1;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendParams& p, bool bf16, cudaStream_t stream, int* launches) {
    *launches = 0;
    if (p.c.D == 64)
        return bf16 ? launch<Fused::kBF16, 64>(p, stream, launches) : launch<Fused::kFP16, 64>(p, stream, launches);
    return bf16 ? launch<Fused::kBF16, 128>(p, stream, launches) : launch<Fused::kFP16, 128>(p, stream, launches);
}

cudaError_t read_kv_attend_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv_attend_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_kv_attend_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
