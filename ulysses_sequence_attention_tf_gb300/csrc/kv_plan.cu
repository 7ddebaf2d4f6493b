// kv_plan.cu -- pages, starts, positions and slots of a step's requests from their lengths.
//
// Three prefix sums over the requests -- new tokens, pages taken, pages given back -- decide everything: a request is
// served while the sums up to it fit the free pages and the rows, so the served ones are a prefix and a page's rank among
// those taken is its place in the ring.  Every CTA computes the sums for itself (8 bytes a request from the L2) and then
// takes its share of rows and pages, each found by a binary search in the sums: no CTA waits for another, and one
// launch is enough.  Entries that one CTA writes (new table entries, pages given back) none reads: a row on a new page
// takes the page from the ring by its rank.  Bound: latency -- the launch, loads of the lengths, three block-wide steps
// and a page's load: 64 requests 5.4 us, 512 with prompts of 22 thousand rows 7.3.
#include "device_common.cuh"
#include "kv_plan.h"

namespace tfu {

__device__ unsigned g_kv_plan_status;

namespace {

using namespace dev;

constexpr uint32_t kThreadsP = 1024, kWarpsP = kThreadsP / 32;
constexpr uint32_t kMany = 1u << 30;  // sums stop here: above every count that they are compared with

struct Sums {
    uint32_t tokens, pages, back;
};
__device__ __forceinline__ uint32_t capped(uint32_t a, uint32_t b) { return min(a + b, kMany); }
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
    return {capped(a.tokens, b.tokens), capped(a.pages, b.pages), capped(a.back, b.back)};
}
__device__ __forceinline__ Sums shuffled_up(const Sums& a, uint32_t d) {
    return {__shfl_up_sync(0xffffffffu, a.tokens, d), __shfl_up_sync(0xffffffffu, a.pages, d), __shfl_up_sync(0xffffffffu, a.back, d)};
}
__device__ __forceinline__ Sums scanned(Sums a) {  // inclusive over the warp
    for (uint32_t d = 1; d < 32; d *= 2) {
        const Sums b = shuffled_up(a, d);
        if (threadIdx.x % 32 >= d) a = a + b;
    }
    return a;
}

// the last n in [0, count) with first[n] <= x (first ascends, first[0] = 0)
__device__ __forceinline__ uint32_t owner(const uint32_t* first, uint32_t count, uint32_t x) {
    uint32_t lo = 0, hi = count;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct Request {
    int32_t len;
    uint32_t had;  // pages
    Sums asks;     // what it asks for, or gives back
    bool serve;    // may get tokens
    bool bad;
};
__device__ __forceinline__ Request request(const KvPlanParams& p, uint32_t n) {
    const int64_t len = p.lens[n], more = p.new_tokens[n], room = int64_t(p.max_pages) * p.page;
    Request r{int32_t(len), 0, {0, 0, 0}, false, len < 0 || len > room || (more > 0 && len + more > room)};
    if (r.bad) return r;
    r.had = (uint32_t(len) + p.page - 1) >> p.page_bits;
    r.serve = more >= 0;
    if (r.serve)
        r.asks = {uint32_t(more), ((uint32_t(len + more) + p.page - 1) >> p.page_bits) - r.had, 0};
    else
        r.asks.back = r.had;
    return r;
}

__global__ void __launch_bounds__(kThreadsP) kv_plan_kernel(const __grid_constant__ KvPlanParams p) {
    extern __shared__ uint32_t first[];  // [3][N + 1]: of tokens, pages taken, pages given back
    uint32_t* first_page = first + p.N + 1;
    uint32_t* first_back = first_page + p.N + 1;
    uint32_t* lens = first_back + p.N + 1;  // [N]; of no use where a length is out of range
    __shared__ Sums warp_sums[kWarpsP];
    __shared__ uint32_t total_tokens, total_pages;
    grid_dependency_wait();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t head_in = p.free_span[0], count_in = p.free_span[1];
    const bool span = head_in >= 0 && uint32_t(head_in) < p.num_pages && count_in >= 0 && uint32_t(count_in) <= p.num_pages;
    const uint32_t head = span ? uint32_t(head_in) : 0, count = span ? uint32_t(count_in) : 0;
    bool bad = !span;
    if (threadIdx.x == 0) total_tokens = total_pages = 0;

    // each thread sums a run of requests, then the block
    const uint32_t each = (p.N + kThreadsP - 1) / kThreadsP, from = min(threadIdx.x * each, p.N), to = min(from + each, p.N);
    Sums own{0, 0, 0};
    Request held{};  // the run's first: up to 1024 requests, all there is
    for (uint32_t n = from; n < to; ++n) {
        const Request r = request(p, n);
        if (n == from) held = r;
        own = own + r.asks;
    }
    const Sums upto = scanned(own);
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    const Sums warps = scanned(warp_sums[lane]);
    Sums at = shuffled_up(upto, 1);
    if (lane == 0) at = {0, 0, 0};
    const uint32_t before = warp == 0 ? 0 : warp - 1;
    const Sums in_front{__shfl_sync(0xffffffffu, warps.tokens, before), __shfl_sync(0xffffffffu, warps.pages, before),
                        __shfl_sync(0xffffffffu, warps.back, before)};
    if (warp > 0) at = in_front + at;
    // pages given back: those that the ring has room for
    const uint32_t room = span ? p.num_pages - count : 0;
    uint32_t most_tokens = 0, most_pages = 0;
    for (uint32_t n = from; n < to; ++n) {
        const Request r = n == from ? held : request(p, n);
        bad |= r.bad;
        lens[n] = uint32_t(r.len);
        first[n] = at.tokens;
        first_page[n] = at.pages;
        first_back[n] = at.back;
        const Sums next = at + r.asks;
        const bool served = r.serve && next.pages <= count && next.tokens <= p.T;
        if (served) {
            most_tokens = next.tokens;
            most_pages = next.pages;
        }
        if (blockIdx.x == 0)
            p.lens_out[n] = r.bad ? r.len : !r.serve ? 0 : served ? r.len + int32_t(r.asks.tokens) : r.len;
        at = next;
    }
    if (to == p.N && from < to) first_back[p.N] = at.back;
    if (most_tokens) atomicMax(&total_tokens, most_tokens);
    if (most_pages) atomicMax(&total_pages, most_pages);
    __syncthreads();
    const uint32_t tokens = total_tokens, taken = total_pages, asked_back = p.N ? first_back[p.N] : 0, back = min(asked_back, room);
    bad |= back < asked_back;
    if (bad && blockIdx.x == 0) atomicOr(&g_kv_plan_status, 1u);

    const uint32_t stride = gridDim.x * kThreadsP, me = blockIdx.x * kThreadsP + threadIdx.x;
    for (uint32_t n = me; n <= p.N; n += stride) p.starts[n] = int32_t(n < p.N ? min(first[n], tokens) : tokens);
    if (me == 0) {
        p.span_out[0] = int32_t(head + taken < p.num_pages ? head + taken : head + taken - p.num_pages);
        p.span_out[1] = int32_t(count - taken + back);
    }
    auto ring = [&](uint32_t rank) {  // rank <= num_pages
        const uint32_t x = head + rank;
        return x < p.num_pages ? x : x - p.num_pages;
    };
    auto pages_of = [&](uint32_t n) { return (lens[n] + p.page - 1) >> p.page_bits; };
    for (uint32_t r = me; r < taken; r += stride) {
        const uint32_t n = owner(first_page, p.N, r);
        p.table[int64_t(n) * p.table_stride + pages_of(n) + (r - first_page[n])] = p.free_pages[ring(r)];
    }
    for (uint32_t r = me; r < back; r += stride) {
        const uint32_t n = owner(first_back, p.N, r);
        p.free_pages[ring(count + r)] = p.table[int64_t(n) * p.table_stride + (r - first_back[n])];
    }
    for (uint32_t t = me; t < p.T; t += stride) {
        int32_t position = 0, slot = -1;
        if (t < tokens) {
            const uint32_t n = owner(first, p.N, t);
            position = int32_t(lens[n] + (t - first[n]));
            const uint32_t page = uint32_t(position) >> p.page_bits, had = pages_of(n);
            const int32_t id = page < had ? p.table[int64_t(n) * p.table_stride + page] : p.free_pages[ring(first_page[n] + page - had)];
            // a page whose slots no 32-bit number holds (-1 of an entry never filled among them) has none
            if (uint32_t(id) < (1u << 31) >> p.page_bits)
                slot = int32_t(uint32_t(id) * p.page + (uint32_t(position) & (p.page - 1)));
            else
                atomicOr(&g_kv_plan_status, 1u);
        }
        p.positions[t] = position;
        p.slots[t] = slot;
    }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t stream) {
    const size_t smem = (4 * size_t(p.N) + 3) * sizeof(uint32_t);
    // always the largest: with this call's own size, a smaller call of another thread could set it back before the launch
    constexpr int kMostSmem = (4 * kMostRequests + 3) * int(sizeof(uint32_t));
    const cudaError_t e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    const uint32_t most = 152, want = (p.T + kThreadsP - 1) / kThreadsP;
    return launch_overlapped(kv_plan_kernel, want < 1 ? 1 : want > most ? most : want, kThreadsP, smem, stream, p);
}

cudaError_t read_kv_plan_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv_plan_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_kv_plan_status, &zero, sizeof(unsigned));
}

}  // namespace tfu
