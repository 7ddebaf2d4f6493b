// linear_chunks.cu -- linear attention chunk by chunk on the 5th-generation tensor cores.
//
// For a chunk of L <= 128 tokens, rows a and columns b, and the state S in front of it:
//
//   out_a = out_scale ( kv_scale sum_(b <= a) lambda^(a - b) (q_a . k_b) v_b + lambda^(a + 1) q_a S )
//   S    <- lambda^L S + kv_scale sum_b (lambda^(L - 1 - b) k_b)^T v_b
//   reverse, the last chunk first: b >= a, lambda^(b - a), lambda^(L - 1 - a) q_a S, lambda^(b + 1) k_b
//
// -- four products of 128 x 128 x D or 128 x D x D.  A CTA of six warpgroups walks the chunks of one head (or of a segment
// of them, below), each of them at its own step:
//  * warps 0-3: a thread a row of the chunk.  P = X times the decays and the mask, in 16 bits over the scores.
//  * warps 4-7: a thread a row of the output, O1 + lambda^(a + 1) O2, to memory.
//  * warps 8-11: a thread a row of S (D = 64: half a row; dS comes twice then), in registers in fp32.  S in 16 bits into
//    shared memory for O2, and dS into S.
//  * warps 12-19: a thread half a row of the chunk's keys, K_w = K times its decay, in place and the rest in tiles beside.
//  * warp 20, one lane: TMA producer.  Q, K, V tiles through a ring of stages.
//  * warp 21, one lane: X = Q K^T, then O1 = P V with P from TMEM.
//  * warp 22, one lane: O2 = Q S.  Warp 23, one lane: dS = K_w^T V.
// Each chunk's dS starts at zero and is added to S in fp32 with one rounding, so what the tensor cores' sums drop does not
// add up over the chunks.  K_w is a sum of several 16-bit numbers, because S is fp32 and outlives the chunk: two fp16 ones, two
// bf16 ones (2^-16 of a key: S is 2.4e-6 off) for states that only enter outputs, three (S 3e-7 off) for those handed
// out.  P and S only enter the chunk's own output, in 16 bits like it.
// fp16: powers of two bring the largest value of each row of P, of S and of each channel (column) of K_w into [2^13, 2^14), so that
// what is smaller keeps its 11 bits down to 2^-27 of it, K_w its 22 down to 2^-16 of it, and below is off by 2^-38 of it at
// most.  A channel's factor comes out as that of a row of dS, where S takes it in.
//
// Segments: where there are fewer heads than SMs, each sequence is cut.  A first launch finds what every segment but the
// last adds to the state (K and V only), a second one runs these sums up to the states in front of the
// segments, and the segments then go on their own.
//
// Bound: DRAM, q, k, v and out once -- 1 KB a token of D = 128, 2.9 us of an SM's share a chunk.  152 heads of 8192 tokens,
// D = 128: bf16 231 us (5.5 TB/s, 0.81 of the copy bandwidth), handing its state on (three parts of the keys, a ring of four
// stages) 263, fp16 299; D = 64: 129, 140 and 205 us.  A chunk takes 3.3 us at D = 128 in bf16, 6650 cycles: 4500 from the
// scores to P, set by the rows that see four blocks of 32 columns (1100 each), 700 to the product with P, 1500 to the next
// scores; the keys 3400, the output 2700 and dS 1300 go beside that.  The matrix pipe is busy 31 % of the cycles, issue
// slots 35 %; what stalls a group is its own latency (TMEM and shared memory, whose bandwidth the products with both operands
// there take half of) and instruction fetches of six different codes.  fp16 reads its scores twice, for each row's power of two.
// 40 heads of 32760 tokens: 384 us, 105 of them the segments' sums, 8 their join; 425 with decays so slow that the sums leave
// nothing out.
// Measured on the way to this split (152 heads of 8192 tokens, bf16, D = 128): keys weighted by the state's warps 598 us at
// the video shape, by four warps of their own 559, by eight 477; the parts rounded one from another instead of cut 281 us
// here, cut 236; P and output shared by both groups, half of the columns each, 254; a block of P of the rows
// with the most taken by the output's warps 250; D = 64 with scores of one chunk in TMEM 152, of two
// 140, with two chunks' rest tiles 130.
// Registers: the groups' shares are what they hold; up to 48 bytes a thread are spilled (0.1 to 0.3 % of the instructions).
#include "attention_common.cuh"
#include "linear.h"

namespace tfu {

__device__ unsigned g_linear_chunks_status, g_linear_chunks_waits;

namespace {

using namespace dev;

constexpr int kThreadsC = 768;
constexpr uint32_t kChunk = kLinearChunk;
constexpr uint32_t kHalfTile = kChunk * kSwizzleRow;  // 128 rows of 64 elements: 16 KiB

// kRests: tiles that hold what the first part of K_w leaves
template <int kD, bool kOutputs, int kRests>
struct Shape {
    static constexpr uint32_t kTile = kHalfTile * (kD / 64);
    static constexpr uint32_t kStateTile = kD * kSwizzleRow * (kD / 64);
    static constexpr int kTiles = kOutputs ? 3 : 2;                      // a chunk's
    static constexpr int kStages = kD == 128 ? (kOutputs ? 6 : 7) - kRests : 9;
    static constexpr size_t kBars = 2048;
    // D = 64 has room for two chunks' rest tiles, so that the keys of a chunk are weighted beside the product before it
    static constexpr int kSets = kD == 64 ? 2 : 1;
    static constexpr size_t kSmem = (kStages + kSets * kRests) * size_t(kTile) + (kOutputs ? kStateTile : 0) + kBars + 1024;  // and alignment
};

constexpr uint32_t kRowsTransposed = 1u << 15;  // of f16_idesc: A MN-major

// The largest value of kWarps warps through shared memory; false if a wait gave up.
template <int kWarps>
struct Largest {
    float* slots;  // [2][kWarps]
    uint32_t bar, phase;
    __device__ bool of(float& v, uint32_t warp, uint32_t lane, volatile int* abort_flag) {
        v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
        float* at = slots + phase * kWarps;
        if (lane == 0) {
            at[warp] = v;
            mbar_arrive(bar);
        }
        const bool ok = __all_sync(0xffffffffu, bounded_wait(bar, phase, abort_flag, &g_linear_chunks_waits));
        phase ^= 1u;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) v = fmaxf(v, at[x]);
        return ok;
    }
};

// A power of two that takes a largest magnitude v into [2^13, 2^14), as far as fp32's range goes.  1 for 0, infinities and NaN.
__device__ __forceinline__ float up_scale(float v) {
    const int e = int(__float_as_uint(v) >> 23);  // biased; 0: below the normal range
    if (!(v > 0.f) || e == 255) return 1.f;
    const int to = 127 + 13 - (e - 127);
    return __uint_as_float(uint32_t(min(to, 253)) << 23);
}
__device__ __forceinline__ float power_of(uint8_t exponent) { return __uint_as_float(uint32_t(exponent) << 23); }
__device__ __forceinline__ float inverse(float power_of_two) { return __uint_as_float((254u << 23) - __float_as_uint(power_of_two)); }

// 16 consecutive 32-bit columns of this thread's TMEM lane
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// tcgen05.wait::ld orders the registers of loads in flight for the compiler too (tc_landed in 16s)
__device__ __forceinline__ void landed16(uint32_t (&r)[16]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// Takes 16 bits off two numbers and leaves the rest: bf16 by cutting (three parts of 8 bits hold a number of 24), fp16 rounded.
template <Fused kF>
__device__ __forceinline__ uint32_t take_part(uint64_t& v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    uint32_t part;
    if constexpr (kF == Fused::kBF16) {
        part = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
        v = f2_sub(v, f2_pack(__uint_as_float(__float_as_uint(lo) & 0xffff0000u), __uint_as_float(__float_as_uint(hi) & 0xffff0000u)));
    } else {
        part = pack2<kF>(lo, hi);
        unpack2<kF>(part, lo, hi);
        v = f2_sub(v, f2_pack(lo, hi));
    }
    return part;
}

// Eight floats of a state's row, a sector of memory: a thread's rows lie 4 D bytes apart, and with 16 bytes at a time the
// L1, small beside the shared memory taken, would read every sector twice.  Not the read-only path: the state may be written
// where it was read.
__device__ __forceinline__ void load_sector(const float* p, uint64_t* s) {
    asm volatile("ld.global.L1::no_allocate.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(s[0]), "=l"(s[1]), "=l"(s[2]), "=l"(s[3]) : "l"(p) : "memory");
}
__device__ __forceinline__ void store_sector(float* p, const uint64_t* s) {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(s[0]), "l"(s[1]), "l"(s[2]), "l"(s[3]) : "memory");
}

// This warpgroup's registers a thread, of the kLaunched that the CTA was launched with.
constexpr int kLaunched = 80;  // 65536 / kThreadsC, in eights
template <int kRegisters>
__device__ __forceinline__ void registers() {
    if constexpr (kRegisters < kLaunched) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegisters));
    if constexpr (kRegisters > kLaunched) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegisters));
}
// S is 128 registers of a thread at D = 128 and 32 at D = 64.
template <int kD>
struct Registers {
    static constexpr int kP = kD == 128 ? 72 : 112, kO = kD == 128 ? 64 : 80, kS = kD == 128 ? 192 : 96, kK = kD == 128 ? 56 : 72,
                         kIssue = kD == 128 ? 40 : 48;
    static_assert(kP + kO + kS + 2 * kK + kIssue == 6 * kLaunched, "what some take, others give");
};

// kOne: a single pass, whose parameters lie at constant addresses (an index there cost 5 %), forward
template <Fused kF, int kD, bool kOutputs, int kRests, bool kOne>
__global__ void __launch_bounds__(kThreadsC, 1) linear_chunks_kernel(const __grid_constant__ LinearChunkParams cp) {
    using Sh = Shape<kD, kOutputs, kRests>;
    constexpr uint32_t kTile = Sh::kTile;
    constexpr int kStages = Sh::kStages, kTiles = Sh::kTiles, kSets = Sh::kSets;
    constexpr uint32_t kScores = kD == 64 ? 2 : 1;  // chunks whose scores TMEM holds: D = 128 fills its 512 columns with one
    constexpr uint32_t kFactors = 2 * kScores;      // P is up to kScores chunks ahead of the output
    constexpr bool kFp16 = kF == Fused::kFP16;
    const uint32_t which = kOne ? 0 : blockIdx.x % cp.passes, block = kOne ? blockIdx.x : blockIdx.x / cp.passes;
    const LinearPass& p = cp.pass[which];
    // several passes are the gradients' (of batch rows), a single one goes forward
    const bool reverse = !kOne && p.reverse, rows_of_sequences = kOne && p.starts;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* rest_tiles = smem + kStages * size_t(kTile);  // of K_w
    uint8_t* state_tile = rest_tiles + kSets * kRests * kTile;
    uint64_t* bars = reinterpret_cast<uint64_t*>(state_tile + (kOutputs ? Sh::kStateTile : 0));
    const uint32_t ring = smem_u32(smem);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
    const uint32_t x_full0 = empty0 + 8 * kStages, p_ready0 = x_full0 + 16, o1_full = p_ready0 + 16, o2_full = o1_full + 8,
                   o_free = o2_full + 8, s_ready = o_free + 8, k_ready0 = s_ready + 8, ds_full0 = k_ready0 + 16, ds_free = ds_full0 + 16,
                   done_a = ds_free + 8, done_b = done_a + 8, done_c = done_b + 8, state_largest = done_c + 8, keys_met = state_largest + 8,
                   k_begun0 = keys_met + 8;
    constexpr int kFixedBars = 20;  // an even number
    float* floats = reinterpret_cast<float*>(bars + 2 * kStages + kFixedBars);  // 16-byte aligned
    float* decays = floats;             // [64]: lambda^(31 - r), reverse: lambda^(r - 32), 0 where that is no decay
    float* state_factor = floats + 64;  // fp16: what O2 is to be multiplied by, [2] by parity of the chunk
    float* largest = floats + 66;       // [2][4]
    // fp16: biased exponents of the channels' powers of two, [kExponents][D] by chunk: the keys of chunk x + kExponents wait for the
    // product of x + kExponents - kSets, which waits for the state to have taken the chunk before that one, x at the least
    constexpr uint32_t kExponents = 256 / kD;
    static_assert(kExponents > kSets, "a factor is overwritten behind its reader");
    uint8_t* key_exponents = reinterpret_cast<uint8_t*>(floats + 74);
    uint8_t* row_exponents = key_exponents + 256;  // of the powers of two of P's rows, [kFactors][128]
    float* key_scale = floats + 140 + kFactors * kChunk / 4;  // this chunk's powers of two by channel, [D]; 16-byte aligned
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(key_scale + kD);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kStages + kFixedBars) * 8 + (142 + kFactors * kChunk / 4 + kD) * 4 <= int(Sh::kBars), "barriers and factors");
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, quarter = warp % 4, group = warp / 4;

    // the unit: sequence, head, segment.  In the grid's order the passes of a unit lie beside one another, then the
    // segments of a head, a reverse pass's from its last on: what runs together reads the same tokens
    const uint32_t heads = p.P * p.Hl, here = kOutputs ? cp.segments : cp.segments - 1;
    const uint32_t seg = reverse ? here - 1 - block % here : block % here, unit = block / here, head = unit % heads, n = unit / heads;
    const uint32_t g = head / p.Hl, h = head % p.Hl;

    if (threadIdx.x == 640)  // the producer's thread
        for (int y = 3 - kTiles; y < 3; ++y)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&cp.maps[cp.tensor[which][y]].m[g])) : "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kOutputs ? 2 : 1);
        }
        for (uint32_t s = 0; s < kScores; ++s) {  // by the chunk
            mbar_init(x_full0 + 8 * s, 1);
            mbar_init(p_ready0 + 8 * s, 4);  // a warp each
            mbar_init(k_ready0 + 8 * s, 8);
            mbar_init(k_begun0 + 8 * s, 8);
        }
        mbar_init(o1_full, 1);
        mbar_init(o2_full, 1);
        mbar_init(o_free, 4);
        mbar_init(s_ready, 4);
        for (uint32_t s = 0; s < uint32_t(kSets); ++s) mbar_init(ds_full0 + 8 * s, 1);
        mbar_init(ds_free, 4);
        mbar_init(done_a, 1);
        mbar_init(done_b, 1);
        mbar_init(done_c, 1);
        mbar_init(state_largest, 4);
        mbar_init(keys_met, 8);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 21) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    const uint32_t tmem = *tmem_slot, o1_tmem = tmem + kScores * kChunk, o2_tmem = o1_tmem + kD, ds_tmem = o2_tmem + kD;

    const LinearSequence seq = linear_sequence(p, n, &g_linear_chunks_status);
    const uint32_t chunks = (seq.len + kChunk - 1) / kChunk, first = seg * cp.seg_chunks;
    const uint32_t count = seq.ok && chunks > first ? min(chunks - first, cp.seg_chunks) : 0;
    const bool last = first + count == chunks;  // of this sequence's segments
    const bool work = count > 0 && (kOutputs || !last);
    // a decay that leaves nothing of the token before is as good as any larger one, and times log2 e it stays finite: 0 times it is 0
    constexpr float kMostDecay = 256.f;
    const float decay = p.decay[head] > kMostDecay ? kMostDecay : p.decay[head];
    // a segment's sum: what is more than kGone / decay tokens in front of its end counts for less than fp32's least number, whatever
    // its key and value are (2^128 e^-193 < 2^-149)
    constexpr float kGone = 193.f;
    const float reach = kGone / (decay * float(kChunk));  // chunks; the last ones of a segment are whole
    const uint32_t skipped = !kOutputs && decay > 0.f && reach + 1.f < float(count) ? count - uint32_t(reach) - 1 : 0;
    const uint32_t visits = count - skipped;
    // chunk x of those visited: its first token and how many it has
    auto chunk_at = [&](uint32_t x) { return (reverse ? chunks - 1 - first - skipped - x : first + skipped + x) * kChunk; };
    auto chunk_len = [&](uint32_t at) { return min(seq.len - at, kChunk); };
    auto wait = [&](uint32_t bar, uint32_t x) { return bounded_wait(bar, x & 1u, abort_flag, &g_linear_chunks_waits); };
    auto all_wait = [&](uint32_t bar, uint32_t x) { return bool(__all_sync(0xffffffffu, wait(bar, x))); };
    auto wait2 = [&](uint32_t bar0, uint32_t x) { return wait(bar0 + 8 * (x % kScores), x / kScores); };
    auto all_wait2 = [&](uint32_t bar0, uint32_t x) { return all_wait(bar0 + 8 * (x % kScores), x / kScores); };
    auto ds_full = [&](uint32_t x) { return ds_full0 + 8 * (x % kSets); };
    auto all_wait_ds = [&](uint32_t x) { return all_wait(ds_full(x), x / kSets); };
    auto scores_of = [&](uint32_t x) { return tmem + x % kScores * kChunk; };
    auto landed = [&](uint32_t m) { return wait(full0 + 8 * (m % kStages), m / kStages); };  // the ring's tile m
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (!work) {
    } else if (group == 5) {
        registers<Registers<kD>::kIssue>();
        if (warp == 20 && elect_one()) {
            // ---------------- TMA producer
            const uint32_t* tensor = cp.tensor[which];
            const CUtensorMap* maps[3] = {&cp.maps[tensor[0]].m[g], &cp.maps[tensor[1]].m[g], &cp.maps[tensor[2]].m[g]};
            uint32_t m = 0;  // tiles loaded
            bool ok = true;
            for (uint32_t x = 0; ok && x < visits; ++x) {
                const int token = int(seq.first + chunk_at(x));
                for (int y = 0; y < kTiles; ++y, ++m) {
                    const uint32_t s = m % kStages, use = m / kStages;
                    if (use > 0 && !wait(empty0 + 8 * s, use - 1)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(full0 + 8 * s, kTile);
                    for (int z = 0; z < kD / 64; ++z)
                        tma_load_4d(ring + s * kTile + z * kHalfTile, maps[3 - kTiles + y], z * 64, int(h), token, int(seq.b), full0 + 8 * s);
                }
            }
            // every load has landed before the CTA exits
            for (uint32_t k = m > uint32_t(kStages) ? m - kStages : 0; k < m; ++k)
                drain_phase(full0 + 8 * (k % kStages), (k / kStages) & 1u);
        } else if (kOutputs && warp == 21 && elect_one()) {
            // ---------------- X = Q K^T, O1 = P V
            constexpr uint32_t kIdescX = f16_idesc(!kFp16, kChunk, kChunk, false);
            constexpr uint32_t kIdescO = f16_idesc(!kFp16, kChunk, kD, true);
            const uint32_t low = desc_low(ring), v_low = desc_low(ring, kHalfTile);
            auto scores = [&](uint32_t x) {
                const uint32_t m = x * kTiles, qs = m % kStages, ks = (m + 1) % kStages;
                if (!landed(m) || !landed(m + 1)) return false;
                // no arrival on x_full runs two phases ahead of the warps that wait for it to weight the keys
                if (x >= kScores && !wait2(k_begun0, x - kScores)) return false;
                tc_fence_after();
                tc_product<kD, kHalfTile, kHalfTile>(scores_of(x), low + qs * (kTile >> 4), low + ks * (kTile >> 4), kIdescX);
                tc_commit(x_full0 + 8 * (x % kScores));
                tc_commit(empty0 + 8 * qs);
                tc_commit(empty0 + 8 * ks);
                return true;
            };
            bool ok = true;
            for (uint32_t x = 0; ok && x < kScores && x < visits; ++x) ok = scores(x);
            for (uint32_t x = 0; ok && x < visits; ++x) {
                const uint32_t m = x * kTiles, vs = (m + 2) % kStages;
                if (!wait2(p_ready0, x) || !landed(m + 2) || (x > 0 && !wait(o_free, x - 1))) break;
                tc_fence_after();
                tc_product_ts<kChunk>(o1_tmem, scores_of(x), v_low + vs * (kTile >> 4), kIdescO, 0u);
                tc_commit(o1_full);
                tc_commit(empty0 + 8 * vs);
                if (x + kScores < visits) ok = scores(x + kScores);  // over the weights that this product reads first
            }
            tc_commit(done_a);
            drain_phase(done_a, 0);  // every product of this thread has completed
        } else if (kOutputs && warp == 22 && elect_one()) {
            // ---------------- O2 = Q S
            constexpr uint32_t kIdesc2 = f16_idesc(!kFp16, kChunk, kD, true);
            const uint32_t q_low = desc_low(ring), state_low = desc_low(smem_u32(state_tile), kD * kSwizzleRow);
            for (uint32_t x = 0; x < visits; ++x) {
                const uint32_t m = x * kTiles, qs = m % kStages;
                if (!landed(m) || !wait(s_ready, x) || (x > 0 && !wait(o_free, x - 1))) break;
                tc_fence_after();
#pragma unroll
                for (uint32_t kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t a = q_low + qs * (kTile >> 4) + ((kk / 4 * kHalfTile + kk % 4 * 32) >> 4), b = state_low + kk * (2048 >> 4);
                    if (kk == 0)
                        tc_mma_low<false>(o2_tmem, a, b, kIdesc2);
                    else
                        tc_mma_low<true>(o2_tmem, a, b, kIdesc2);
                }
                tc_commit(o2_full);
                tc_commit(empty0 + 8 * qs);
            }
            tc_commit(done_b);
            drain_phase(done_b, 0);
        } else if (warp == 23 && elect_one()) {
            // ---------------- dS = K_w^T V
            constexpr uint32_t kIdescS = f16_idesc(!kFp16, kChunk, kD, true) | kRowsTransposed;
            const uint32_t v_low = desc_low(ring, kHalfTile);
            // 128 rows of K_w^T; D = 64: its 64 rows twice
            const uint32_t k_low = desc_low(ring, kD == 128 ? kHalfTile : 0), rest_low = desc_low(smem_u32(rest_tiles), kD == 128 ? kHalfTile : 0);
            for (uint32_t x = 0; x < visits; ++x) {
                const uint32_t m = x * kTiles, ks = (m + kTiles - 2) % kStages, vs = (m + kTiles - 1) % kStages;
                if (!landed(m + kTiles - 1) || !wait2(k_ready0, x) || (x > 0 && !wait(ds_free, x - 1))) break;
                // a short chunk among rows of other sequences: the rows behind it are cleared with P
                if (kOutputs && rows_of_sequences && chunk_len(chunk_at(x)) < kChunk && !wait2(p_ready0, x)) break;
                tc_fence_after();
                const uint32_t b = v_low + vs * (kTile >> 4), a = k_low + ks * (kTile >> 4), rests = rest_low + x % kSets * (kRests * kTile >> 4);
                tc_mma_low<false>(ds_tmem, a, b, kIdescS);
#pragma unroll
                for (uint32_t kk = 1; kk < kChunk / 16; ++kk) tc_mma_low<true>(ds_tmem, a + kk * (2048 >> 4), b + kk * (2048 >> 4), kIdescS);
#pragma unroll 1
                for (int r = 0; r < kRests; ++r)
#pragma unroll
                    for (uint32_t kk = 0; kk < kChunk / 16; ++kk)
                        tc_mma_low<true>(ds_tmem, rests + r * (kTile >> 4) + kk * (2048 >> 4), b + kk * (2048 >> 4), kIdescS);
                tc_commit(ds_full(x));
                tc_commit(empty0 + 8 * ks);
                tc_commit(empty0 + 8 * vs);
            }
            tc_commit(done_c);
            drain_phase(done_c, 0);
        }
    } else if (group == 0) {
        registers<Registers<kD>::kP>();
        if (kOutputs) {
            // ---------------- P: a thread a row
            const uint32_t a = quarter * 32 + lane, lane_base = (quarter * 32u) << 16;
            const float c = decay * kLog2e, both_scales = p.out_scale * p.kv_scale;
            if (warp < 2) {
                const uint32_t r = warp * 32 + lane;
                decays[r] = reverse ? (r < 32 ? 0.f : ex2(-c * float(r - 32))) : r < 32 ? ex2(-c * float(31 - r)) : 0.f;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");  // these four warps, before any wait
            const float* own_decays = decays + (reverse ? 32 - lane : 31 - lane);  // of columns in the row's own block
            const float* far_decays = decays + (reverse ? 32 : 0);                 // of others, up to a factor
            const uint32_t own_columns = reverse ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
            // of block j's columns, what far_decays leaves out
            auto far_factor = [&](uint32_t j) {
                const int gone = reverse ? int(32 * (j - quarter)) - int(lane) : int(32 * (quarter - j)) + int(lane) - 31;
                return ex2(-c * float(gone));
            };
            // scores of 32 columns times their decays, from column 32 j of the row on
            auto weighted = [&](uint32_t at, uint32_t j, uint64_t (&w)[16], const float scales) {
                uint32_t r[32];
                tc_ld32(at + j * 32, r);
                tc_wait_ld();
                tc_landed(r);
                if (j == quarter) {
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        // selected: a masked key may be anything
                        const float w0 = own_decays[2 * y] * scales, w1 = own_decays[2 * y + 1] * scales;
                        w[y] = f2_pack((own_columns >> (2 * y)) & 1u ? __uint_as_float(r[2 * y]) * w0 : 0.f,
                                       (own_columns >> (2 * y + 1)) & 1u ? __uint_as_float(r[2 * y + 1]) * w1 : 0.f);
                    }
                } else {
                    const float f = far_factor(j) * scales;
                    const uint64_t f2 = f2_pack(f, f);
#pragma unroll
                    for (int y = 0; y < 16; y += 2) {
                        const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(far_decays + 2 * y);
                        w[y] = f2_mul(f2_pack(__uint_as_float(r[2 * y]), __uint_as_float(r[2 * y + 1])), f2_mul(t.x, f2));
                        w[y + 1] = f2_mul(f2_pack(__uint_as_float(r[2 * y + 2]), __uint_as_float(r[2 * y + 3])), f2_mul(t.y, f2));
                    }
                }
            };
            auto seen = [&](uint32_t j) { return reverse ? j >= quarter : j <= quarter; };
            for (uint32_t x = 0; x < visits; ++x) {
                const uint32_t len = chunk_len(chunk_at(x));
                if (!all_wait2(x_full0, x)) break;
                tc_fence_after();
                const uint32_t at = scores_of(x) + lane_base;
                float f = both_scales;
                if (kFp16) {
                    // the row's power of two, from its weighted scores: one that has faded says nothing about the others
                    float most = 0.f;
#pragma unroll 1
                    for (uint32_t j = 0; j < 4; ++j) {
                        if (!seen(j)) continue;
                        uint32_t r[32];
                        tc_ld32(at + j * 32, r);
                        tc_wait_ld();
                        tc_landed(r);
                        // own_decays are 0 behind the row; fmaxf passes over NaN: a masked key that is not finite, times 0
                        const float* t = j == quarter ? own_decays : far_decays;
                        float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int y = 0; y < 32; ++y) m[y % 4] = fmaxf(m[y % 4], fabsf(__uint_as_float(r[y]) * t[y]));
                        most = fmaxf(most, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * (j == quarter ? 1.f : far_factor(j)));
                    }
                    const float to_half = up_scale(most * fabsf(both_scales));
                    row_exponents[x % kFactors * kChunk + a] = uint8_t(__float_as_uint(to_half) >> 23);
                    f *= to_half;
                }
#pragma unroll 1
                for (uint32_t j = 0; j < 4; ++j) {
                    uint32_t o[16];
                    if (seen(j)) {
                        uint64_t w[16];
                        weighted(at, j, w, f);
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            float lo, hi;
                            f2_unpack(w[y], lo, hi);
                            o[y] = pack2<kF>(lo, hi);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = 0u;
                    }
                    tc_st16(at + j * 16, o);
                }
                if (rows_of_sequences && len < kChunk) {  // rows of other sequences, whose V may be anything
                    const uint32_t m = x * kTiles + 2;
                    if (!__all_sync(0xffffffffu, landed(m))) break;
                    if (a >= len) {
                        uint4* v = reinterpret_cast<uint4*>(smem + (m % kStages) * size_t(kTile) + a * kSwizzleRow);
                        for (int z = 0; z < kD / 64; ++z)
                            for (int y = 0; y < 8; ++y) v[z * (kHalfTile / 16) + y] = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();
                    __syncwarp();  // tcgen05.wait is for a warp that has come together
                }
                tc_wait_st();
                tc_fence_before();
                arrive(p_ready0 + 8 * (x % kScores));
            }
        }
    } else if (group == 1) {
        registers<Registers<kD>::kO>();
        if (kOutputs) {
            // ---------------- the output: a thread a row
            const uint32_t a = quarter * 32 + lane, lane_base = (quarter * 32u) << 16;
            float age = p.out_scale * expf(-decay * float(a + 1));
            for (uint32_t x = 0; x < visits; ++x) {
                const uint32_t at = chunk_at(x), len = chunk_len(at);
                const bool valid = a < len;
                if (reverse) age = p.out_scale * expf(-decay * float(int(len) - 1 - int(a)));
                if (!all_wait(o1_full, x) || !all_wait(o2_full, x)) break;
                tc_fence_after();
                const float f1 = kFp16 ? inverse(power_of(row_exponents[x % kFactors * kChunk + a])) : 1.f, f2 = kFp16 ? age * state_factor[x & 1u] : age;
                const uint64_t f1_2 = f2_pack(f1, f1), f2_2 = f2_pack(f2, f2);
                uint8_t* dst = p.out.base[g] + int64_t(seq.b) * p.out.b + (seq.first + at + (valid ? a : 0)) * p.out.t + int64_t(h) * p.out.h;
#pragma unroll 1
                for (int z = 0; z < kD; z += 16) {
                    uint32_t r1[16], r2[16];
                    tc_ld16(o1_tmem + lane_base + z, r1);
                    tc_ld16(o2_tmem + lane_base + z, r2);
                    tc_wait_ld();
                    landed16(r1);
                    landed16(r2);
                    if (z + 16 == kD) {
                        tc_fence_before();
                        arrive(o_free);
                    }
                    Vec<32> w;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint64_t v = f2_pack(__uint_as_float(r1[2 * i]), __uint_as_float(r1[2 * i + 1]));
                        if (kFp16) v = f2_mul(v, f1_2);
                        v = f2_fma(f2_pack(__uint_as_float(r2[2 * i]), __uint_as_float(r2[2 * i + 1])), f2_2, v);
                        float lo, hi;
                        f2_unpack(v, lo, hi);
                        w.w[i] = pack2<kF>(lo, hi);
                    }
                    if (!valid) continue;
                    if (cp.wide_out[which]) {
                        st_stream<32>(dst + z * 2, w);
                    } else {
                        *reinterpret_cast<uint4*>(dst + z * 2) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
                        *reinterpret_cast<uint4*>(dst + z * 2 + 16) = make_uint4(w.w[4], w.w[5], w.w[6], w.w[7]);
                    }
                }
            }
        }
    } else if (group == 2) {
        registers<Registers<kD>::kS>();
        // ---------------- the state: a thread a row of it (D = 64: half a row)
        constexpr int kCols = kD == 128 ? 128 : 32;
        const uint32_t t = quarter * 32 + lane, lane_base = (quarter * 32u) << 16;
        const uint32_t row = t % kD, col = kD == 128 ? 0 : t / 64 * 32;
        Largest<4> most{largest, state_largest, 0};
        uint64_t s[kCols / 2];
        const int64_t own = (int64_t(seq.slot) * heads + head) * (kD * kD);
        // in front of a segment; the state itself only where there is one segment: another one's CTA may write it
        float* const parts = cp.parts + ((int64_t(which) * p.N * heads + unit) * cp.segments + seg) * (kD * kD);
        const bool joined = kOutputs && chunks > cp.seg_chunks;
        const float* from = joined ? (seg > 0 || p.state ? parts : nullptr) : kOutputs && p.state ? p.state + own : nullptr;
        if (!from) {
#pragma unroll
            for (int y = 0; y < kCols / 2; ++y) s[y] = 0;
        } else if (!kOne && !joined && p.transposed) {
#pragma unroll
            for (int y = 0; y < kCols / 2; ++y) s[y] = f2_pack(from[(col + 2 * y) * kD + row], from[(col + 2 * y + 1) * kD + row]);
        } else {
#pragma unroll
            for (int y = 0; y < kCols / 2; y += 4) load_sector(from + row * kD + col + 2 * y, &s[y]);
        }
        bool ok = true;
        for (uint32_t x = 0; x < visits; ++x) {
            const uint32_t len = chunk_len(chunk_at(x));
            if (kOutputs) {
                float to_half = 1.f;
                if (kFp16) {
                    float v = 0.f;
#pragma unroll
                    for (int y = 0; y < kCols / 2; ++y) {
                        float lo, hi;
                        f2_unpack(s[y], lo, hi);
                        v = fmaxf(v, fmaxf(fabsf(lo), fabsf(hi)));
                    }
                    if (!(ok = most.of(v, quarter, lane, abort_flag))) break;
                    to_half = up_scale(v);
                }
                // the product with the tile's last contents; it followed the output of the chunk before that one, which was the
                // last reader of the factor that is overwritten here
                if (x > 0 && !(ok = all_wait(o2_full, x - 1))) break;
                if (kFp16 && t == 0) state_factor[x & 1u] = inverse(to_half);
                uint8_t* dst = state_tile + row * kSwizzleRow;
#pragma unroll
                for (int y = 0; y < kCols; y += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float lo, hi;
                        f2_unpack(kFp16 ? f2_mul(s[y / 2 + i], f2_pack(to_half, to_half)) : s[y / 2 + i], lo, hi);
                        w[i] = pack2<kF>(lo, hi);
                    }
                    const uint32_t e = col + y;
                    *reinterpret_cast<uint4*>(dst + e / 64 * (kD * kSwizzleRow) + ((e % 64 / 8) ^ (row & 7u)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_async_shared();
                arrive(s_ready);
            }
            const Fade fade(decay * float(len));
            if (!(ok = all_wait_ds(x))) break;
            tc_fence_after();
            const float back =
                kFp16 ? p.kv_scale * inverse(power_of(key_exponents[x % kExponents * kD + row])) : p.kv_scale;
            const uint64_t back2 = f2_pack(back, back), factor2 = f2_pack(fade.factor, fade.factor), whole2 = f2_pack(fade.whole, fade.whole);
#pragma unroll
            for (int z = 0; z < kCols; z += 32) {
                uint32_t r[32];
                tc_ld32(ds_tmem + lane_base + col + z, r);
                tc_wait_ld();
                tc_landed(r);
                if (z + 32 == kCols) {
                    tc_fence_before();
                    arrive(ds_free);
                }
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const uint64_t add = f2_mul(f2_pack(__uint_as_float(r[2 * y]), __uint_as_float(r[2 * y + 1])), back2);
                    s[z / 2 + y] = f2_fma(whole2, s[z / 2 + y], f2_fma(s[z / 2 + y], factor2, add));
                }
            }
        }
        if (ok && !*abort_flag) {
            float* to = !kOutputs ? parts + kD * kD  // what is in front of the next one
                        : last && p.final_state ? p.final_state + own : nullptr;
            if (to) {
#pragma unroll
                for (int y = 0; y < kCols / 2; y += 4) store_sector(to + row * kD + col + 2 * y, &s[y]);
            }
        }
    } else {
        registers<Registers<kD>::kK>();
        // ---------------- the keys times their decay: a thread half a row of the chunk
        const uint32_t t = quarter * 32 + lane, half = group - 3;
        for (uint32_t x = 0; x < visits; ++x) {
            const uint32_t len = chunk_len(chunk_at(x)), m = x * kTiles + kTiles - 2;
            // the scores no longer need K as it came; the products with the rest tiles' last contents have completed
            if ((kOutputs && !all_wait2(x_full0, x)) || !__all_sync(0xffffffffu, landed(m)) || (x >= kSets && !all_wait_ds(x - kSets))) break;
            if (kOutputs) arrive(k_begun0 + 8 * (x % kScores));
            const bool valid = t < len;
            const float w = valid ? expf(-decay * float(reverse ? t + 1 : len - 1 - t)) : 0.f;
            // D = 128: 64 elements are a half of the tile; D = 64: 32 of the row
            uint8_t* key = smem + (m % kStages) * size_t(kTile) + t * kSwizzleRow;
            uint8_t* rest = rest_tiles + x % kSets * (kRests * kTile) + t * kSwizzleRow;
            auto vec = [&](int y) {
                return kD == 128 ? half * kHalfTile + ((uint32_t(y) ^ (t & 7u)) * 16) : ((half * 4 + uint32_t(y)) ^ (t & 7u)) * 16;
            };
            constexpr int kVecs = kD / 16;
            // the groups' codes share the instruction cache: fp16 by half of the vectors 329 -> 299 us (D = 64 216 -> 204), all rolled up 302
            constexpr int kAtOnce = kFp16 ? kVecs / 2 : kVecs;
            if (kFp16) {
                // every channel's largest weighted key: a lane takes two channels, a warp a part of the tokens; the parts meet where
                // the rests are written afterwards
                constexpr uint32_t kParts = kD == 128 ? 4 : 8, kEach = kChunk / kParts;
                const uint32_t part = kD == 128 ? quarter : quarter * 2 + half, channel = kD == 128 ? half * 64 : 0;
                float* const found = reinterpret_cast<float*>(rest_tiles + x % kSets * (kRests * kTile));  // [kParts][D]
                const uint8_t* from = smem + (m % kStages) * size_t(kTile) + channel / 64 * kHalfTile + part * kEach * kSwizzleRow + lane % 4 * 4;
                auto word = [&](uint32_t i) { return *reinterpret_cast<const __half2*>(from + i * kSwizzleRow + ((lane / 4) ^ (i & 7u)) * 16); };
                float most0 = 0.f, most1 = 0.f;  // fmaxf passes over NaN: rows of no token, times 0
                auto take = [&](__half2 two, uint32_t token) {
                    const float weight = __shfl_sync(0xffffffffu, w, token % 32);
                    const float2 k = __half22float2(two);
                    most0 = fmaxf(most0, fabsf(k.x) * weight);
                    most1 = fmaxf(most1, fabsf(k.y) * weight);
                };
                // Eight tokens may share the weight of the one that has faded least, e^7 too large at most (2^-27 and 2^-6 in place of 2^-38
                // and 2^-16 of a channel's largest): 152 heads of 8192 tokens 299 us, every token by its own 317.
                if (decay >= 0.f && decay <= 1.f && len == kChunk) {
                    const uint32_t nearest = reverse ? 0 : 7;
#pragma unroll
                    for (uint32_t i = 0; i < kEach; i += 8) {
                        __half2 eight = __habs2(word(i));
#pragma unroll
                        for (uint32_t z = 1; z < 8; ++z) eight = __hmax2(eight, __habs2(word(i + z)));
                        take(eight, part * kEach + i + nearest);
                    }
                } else {
#pragma unroll 8
                    for (uint32_t i = 0; i < kEach; ++i) take(word(i), part * kEach + i);
                }
                *reinterpret_cast<float2*>(found + part * kD + channel + lane * 2) = make_float2(most0, most1);
                arrive(keys_met);
                if (!all_wait(keys_met, 0)) break;
                const uint32_t c = half * 128 + t;
                if (c < kD) {
                    float v = found[c];
#pragma unroll
                    for (uint32_t y = 1; y < kParts; ++y) v = fmaxf(v, found[y * kD + c]);
                    const float to_half = up_scale(v);
                    key_scale[c] = to_half;
                    key_exponents[x % kExponents * kD + c] = uint8_t(__float_as_uint(to_half) >> 23);
                }
                arrive(keys_met);
                if (!all_wait(keys_met, 1)) break;
            }
            const uint64_t w2 = f2_pack(w, w);
#pragma unroll kAtOnce
            for (int y = 0; y < kVecs; ++y) {
                const uint4 k = *reinterpret_cast<const uint4*>(key + vec(y));
                const uint32_t kw[4] = {valid ? k.x : 0u, valid ? k.y : 0u, valid ? k.z : 0u, valid ? k.w : 0u};
                uint32_t part[1 + kRests][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    unpack2<kF>(kw[i], lo, hi);
                    uint64_t v = f2_mul(f2_pack(lo, hi), w2);
                    if (kFp16) v = f2_mul(v, *reinterpret_cast<const uint64_t*>(key_scale + half * (kD / 2) + y * 8 + i * 2));
#pragma unroll
                    for (int r = 0; r < kRests; ++r) part[r][i] = take_part<kF>(v);
                    f2_unpack(v, lo, hi);
                    part[kRests][i] = pack2<kF>(lo, hi);
                }
                *reinterpret_cast<uint4*>(key + vec(y)) = make_uint4(part[0][0], part[0][1], part[0][2], part[0][3]);
#pragma unroll
                for (int r = 0; r < kRests; ++r)
                    *reinterpret_cast<uint4*>(rest + r * kTile + vec(y)) = make_uint4(part[r + 1][0], part[r + 1][1], part[r + 1][2], part[r + 1][3]);
            }
            fence_async_shared();
            arrive(k_ready0 + 8 * (x % kScores));
        }
    }
    // teardown: every product has completed (their threads drained them) and every TMEM access has finished before
    // the columns are freed
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 21) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The sums of the segments, run up to the states in front of them: parts[0] of a head becomes the state that the sequence
// starts from (where there is one), parts[1], what segment 0 adds, the state in front of segment 1, and so on.  Four
// elements a thread.
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ LinearChunkParams cp) {
    grid_dependency_wait();
    const uint32_t which = blockIdx.x % cp.passes, block = blockIdx.x / cp.passes, segments = cp.segments, seg_chunks = cp.seg_chunks;
    const LinearPass& p = cp.pass[which];
    const uint32_t size = p.D * p.D, blocks = size / 1024, heads = p.P * p.Hl;
    const uint32_t unit = block / blocks, e = (block % blocks * 256 + threadIdx.x) * 4, head = unit % heads, n = unit / heads;
    const LinearSequence seq = linear_sequence(p, n, &g_linear_chunks_status);
    if (!seq.ok) return;
    const uint32_t chunks = (seq.len + kChunk - 1) / kChunk, used = (chunks + seg_chunks - 1) / seg_chunks;
    if (used < 2) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.state) {
        const float* from = p.state + (int64_t(seq.slot) * heads + head) * size;
        const uint32_t row = e / p.D, col = e % p.D;
        s = p.transposed ? make_float4(from[col * p.D + row], from[(col + 1) * p.D + row], from[(col + 2) * p.D + row], from[(col + 3) * p.D + row])
                         : *reinterpret_cast<const float4*>(from + e);
    }
    const float decay = p.decay[head];
    float4* at = reinterpret_cast<float4*>(cp.parts + (int64_t(which) * p.N * heads + unit) * segments * size + e);
    if (p.state) *at = s;
    const uint32_t whole = seg_chunks * kChunk, short_by = chunks * kChunk - seq.len;
    const Fade fade(decay * float(whole)), begin(decay * float(p.reverse ? whole - short_by : whole));
    constexpr uint32_t kAhead = 8;  // loads on their way together
    for (uint32_t x0 = 0; x0 + 1 < used; x0 += kAhead) {
        float4 add[kAhead];
#pragma unroll
        for (uint32_t y = 0; y < kAhead; ++y)
            if (x0 + y + 1 < used) add[y] = at[(x0 + y + 1) * (size / 4)];
#pragma unroll
        for (uint32_t y = 0; y < kAhead; ++y) {
            if (x0 + y + 1 >= used) break;
            const Fade& f = x0 + y == 0 ? begin : fade;
            s = make_float4(f.of(s.x, add[y].x), f.of(s.y, add[y].y), f.of(s.z, add[y].z), f.of(s.w, add[y].w));
            at[(x0 + y + 1) * (size / 4)] = s;
        }
    }
}

template <Fused kF, int kD, bool kOutputs, int kRests>
cudaError_t launch(const LinearChunkParams& p, uint32_t grid, cudaStream_t stream) {
    const size_t smem = Shape<kD, kOutputs, kRests>::kSmem;
    auto kernel = p.passes == 1 ? linear_chunks_kernel<kF, kD, kOutputs, kRests, true> : linear_chunks_kernel<kF, kD, kOutputs, kRests, false>;
    // setting it twice is harmless; the cost is a fraction of a microsecond
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, grid, kThreadsC, smem, stream, p);
}

template <Fused kF, int kD, int kRests>
cudaError_t launch_all(const LinearChunkParams& p, cudaStream_t stream, int* launches) {
    const uint32_t units = p.passes * p.pass[0].N * p.pass[0].P * p.pass[0].Hl;
    cudaError_t e;
    if (p.segments > 1) {
        if ((e = launch<kF, kD, false, kRests>(p, units * (p.segments - 1), stream)) != cudaSuccess) return e;
        if ((e = launch_overlapped(linear_join_kernel, units * (kD * kD / 1024), 256, 0, stream, p)) !=
            cudaSuccess)
            return e;
        *launches += 2;
    }
    if ((e = launch<kF, kD, true, kRests>(p, units * p.segments, stream)) != cudaSuccess) return e;
    *launches += 1;
    return cudaSuccess;
}

// Three bf16 parts of a weighted key where a state is handed out, two where it stays inside the call.
template <int kD>
cudaError_t launch_typed(const LinearChunkParams& p, bool bf16, cudaStream_t stream, int* launches) {
    if (!bf16) return launch_all<Fused::kFP16, kD, 1>(p, stream, launches);
    bool out = false;
    for (uint32_t i = 0; i < p.passes; ++i) out |= p.pass[i].final_state != nullptr;
    return out ? launch_all<Fused::kBF16, kD, 2>(p, stream, launches) : launch_all<Fused::kBF16, kD, 1>(p, stream, launches);
}

cudaError_t read_word(const unsigned& symbol, unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, symbol, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(symbol, &zero, sizeof(unsigned));
}

}  // namespace

cudaError_t launch_linear_chunks(const LinearChunkParams& p, bool bf16, cudaStream_t stream, int* launches) {
    *launches = 0;
    return p.pass[0].D == 64 ? launch_typed<64>(p, bf16, stream, launches) : launch_typed<128>(p, bf16, stream, launches);
}

cudaError_t read_linear_chunks_status(unsigned* out, unsigned* waits, bool clear) {
    const cudaError_t e = read_word(g_linear_chunks_status, out, clear);
    return e != cudaSuccess ? e : read_word(g_linear_chunks_waits, waits, clear);
}

}  // namespace tfu
