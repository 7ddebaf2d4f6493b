// tf_kv_cache.cpp -- host side of the key-value cache entry points of tf_ulysses.h:
// argument checks (all of them before any CUDA call) and the launches.
#include <cmath>

#include "host.h"
#include "kv_cache.h"
#include "kv_plan.h"

using namespace tfu::host;

namespace {

tf_status check_cache(const tf_kv_cache* c, int P, int T, tf_dtype dtype, tfu::KvCache* out) {
    if (!c) return fail(TF_ERR_INVALID, "the cache's description is NULL");
    if (P < 1 || P > TF_ULYSSES_MAX_SHARDS) return fail(TF_ERR_INVALID, "P=%d outside [1, %d]", P, TF_ULYSSES_MAX_SHARDS);
    if (T < 0 || c->N < 0) return fail(TF_ERR_INVALID, "T=%d, N=%d must be >= 0", T, c->N);
    if (c->num_pages < 1 || c->Hkv < 1 || c->max_pages < 1)
        return fail(TF_ERR_INVALID, "num_pages=%d, Hkv=%d, max_pages=%d must be >= 1", c->num_pages, c->Hkv, c->max_pages);
    if (c->Hkv % P != 0) return fail(TF_ERR_DIVISIBILITY, "Hkv=%d is not divisible by P=%d", c->Hkv, P);
    if (dtype != TF_BF16 && dtype != TF_FP16)
        return fail(TF_ERR_UNSUPPORTED, "the cache takes bf16 or fp16 rows (dtype %d)", int(dtype));
    if (c->D != 64 && c->D != 128) return fail(TF_ERR_UNSUPPORTED, "the cache is built for D in {64, 128}, not %d", c->D);
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return fail(TF_ERR_UNSUPPORTED, "the cache is built for pages of 16, 32, 64 or 128 tokens, not %d", c->page_size);
    if (int64_t(c->max_pages) * c->page_size > (int64_t(1) << 30))
        return fail(TF_ERR_UNSUPPORTED, "max_pages * page_size exceeds 2^30 tokens");
    if (c->table_stride < c->max_pages)
        return fail(TF_ERR_INVALID, "table_stride=%lld is below max_pages=%d", (long long)c->table_stride, c->max_pages);
    const void* needed[] = {c->k, c->v, c->k_scale, c->v_scale, c->page_table, c->lens, c->starts};
    const char* names[] = {"k", "v", "k_scale", "v_scale", "page_table", "lens", "starts"};
    for (int i = 0; i < 7; ++i)
        if (!needed[i]) return fail(TF_ERR_INVALID, "the cache's %s is NULL", names[i]);
    if (!aligned16(c->k) || !aligned16(c->v)) return fail(TF_ERR_ALIGNMENT, "the cache's k and v must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(c->k_scale) % 4 || reinterpret_cast<uintptr_t>(c->v_scale) % 4 ||
        reinterpret_cast<uintptr_t>(c->page_table) % 4 || reinterpret_cast<uintptr_t>(c->lens) % 4 ||
        reinterpret_cast<uintptr_t>(c->starts) % 4)
        return fail(TF_ERR_ALIGNMENT, "the cache's scales, table, lengths and starts must be 4-byte aligned");
    out->codes[0] = static_cast<uint8_t*>(c->k);
    out->codes[1] = static_cast<uint8_t*>(c->v);
    out->scales[0] = c->k_scale;
    out->scales[1] = c->v_scale;
    out->table = c->page_table;
    out->lens = c->lens;
    out->starts = c->starts;
    out->table_stride = c->table_stride;
    out->pages = uint32_t(c->num_pages);
    out->Hkv = uint32_t(c->Hkv);
    out->page = uint32_t(c->page_size);
    out->D = uint32_t(c->D);
    out->N = uint32_t(c->N);
    out->max_pages = uint32_t(c->max_pages);
    return TF_OK;
}

tf_status rows_of(const char* name, const void* const* base, const tf_strides* given, int P, int T, int heads, int D,
                  bool written, tfu::RowView* out) {
    const int hl = heads / P;
    if (!base) return fail(TF_ERR_INVALID, "%s is NULL", name);
    tf_status s;
    if (T > 0 && (s = check_ptrs(name, base, P)) != TF_OK) return s;
    const tf_strides st = given ? *given : tf_strides{0, int64_t(hl) * D, D};
    if ((s = check_strides(name, st, 2, 1, T, hl)) != TF_OK) return s;
    if (written && ((T > 1 && st.t == 0) || (hl > 1 && st.h == 0)))
        return fail(TF_ERR_INVALID, "%s is written and has a stride of 0", name);
    for (int g = 0; g < P; ++g) out->base[g] = static_cast<uint8_t*>(const_cast<void*>(base[g]));
    out->t = st.t * 2;
    out->h = st.h * 2;
    return TF_OK;
}

// Up to this many rows (new tokens times query heads) of a key head take the decode kernel,
// which reads each code once for 16 rows; more take the tile kernel, whose cost hardly depends
// on the rows below 256.
constexpr uint32_t kDecodeMost = 64;
constexpr uint32_t kSms = 152;

// How the keys are split.  Decode: about kTargetCtas CTAs when every sequence is as long
// as the longest may be, in chunks of at least kLeastChunk keys (below it the join costs
// more than the parallel chunks give) and at most kMostChunk (so that one long sequence
// among many is spread).  Tiles: one CTA an SM, so the number of chunks that makes the
// rounds of CTAs fullest, a chunk's fixed cost counted as kChunkCost keys.
constexpr uint32_t kTargetCtas = 2432, kLeastChunk = 512, kMostChunk = 8192, kChunkCost = 512;

void plan_chunks(tfu::KvAttendParams* p) {
    const uint32_t rows = p->max_tokens * p->shared;
    p->tiles = rows > kDecodeMost;
    const uint32_t unit = p->tiles ? tfu::kTileRows : rows <= 8 ? 8 : 16;
    p->unit = unit;
    p->row_cap = (rows + unit - 1) / unit * unit;
    const uint64_t ctas = uint64_t(p->c.N) * p->c.Hkv * (p->row_cap / unit);
    uint64_t chunk;
    if (p->tiles) {
        uint64_t best = 1, least = UINT64_MAX;
        for (uint64_t c = 1; c <= 16 && p->max_len / c >= kLeastChunk; ++c) {
            const uint64_t cost = (ctas * c + kSms - 1) / kSms * (p->max_len / c + kChunkCost);
            if (cost < least) {
                least = cost;
                best = c;
            }
        }
        chunk = (p->max_len + best - 1) / best;
    } else {
        const uint64_t want = ctas ? (kTargetCtas + ctas - 1) / ctas : 1;
        chunk = (p->max_len + want - 1) / want;
        chunk = chunk < kLeastChunk ? kLeastChunk : chunk > kMostChunk ? kMostChunk : chunk;
    }
    p->chunk = uint32_t((chunk + 127) / 128 * 128);
    p->chunks = (p->max_len + p->chunk - 1) / p->chunk;
}

tf_status check_kv_attention(const tf_kv_cache* c, const tf_kv_attention* a, tfu::KvAttendParams* p) {
    if (!a) return fail(TF_ERR_INVALID, "the attention's description is NULL");
    tf_status s = check_cache(c, a->P, a->T, a->dtype, &p->c);
    if (s != TF_OK) return s;
    if (a->H < 1) return fail(TF_ERR_INVALID, "H=%d must be >= 1", a->H);
    if (a->H % c->Hkv != 0) return fail(TF_ERR_DIVISIBILITY, "H=%d is not divisible by Hkv=%d", a->H, c->Hkv);
    if ((s = check_scores(a->scale, a->softcap)) != TF_OK) return s;
    if (a->causal != 0 && a->causal != 1) return fail(TF_ERR_INVALID, "causal=%d is neither 0 nor 1", a->causal);
    if (a->T > 0 && (a->max_tokens < 1 || a->max_tokens > a->T))
        return fail(TF_ERR_INVALID, "max_tokens=%d outside [1, T=%d]", a->max_tokens, a->T);
    if (a->max_len < 1 || int64_t(a->max_len) > int64_t(c->max_pages) * c->page_size)
        return fail(TF_ERR_INVALID, "max_len=%d outside [1, max_pages * page_size]", a->max_len);
    if (c->N > 65535 || c->Hkv > 16383 || int64_t(a->max_tokens) * (a->H / c->Hkv) > (int64_t(1) << 30))
        return fail(TF_ERR_UNSUPPORTED, "more than 65535 sequences or 16383 key heads, or 2^30 rows of one key head");
    p->slopes = a->slopes;
    p->scale = a->scale;
    p->cap = a->softcap;
    p->P = uint32_t(a->P);
    p->T = uint32_t(a->T);
    p->Hl = uint32_t(a->H / a->P);
    p->Hkl = uint32_t(c->Hkv / a->P);
    p->shared = uint32_t(a->H / c->Hkv);
    p->max_tokens = uint32_t(a->max_tokens);
    p->max_len = uint32_t(a->max_len);
    p->causal = uint32_t(a->causal);
    plan_chunks(p);
    if (uint64_t(c->N) * c->Hkv * (p->row_cap / p->unit) * p->chunks >= (uint64_t(1) << 31))
        return fail(TF_ERR_UNSUPPORTED, "problem exceeds 2^31 work units");
    return TF_OK;
}

// Bytes of the chunks' sums, then of their statistics.
size_t part_bytes(const tfu::KvAttendParams& p) {
    return p.chunks > 1 ? size_t(p.c.N) * p.c.Hkv * p.row_cap * p.chunks * p.c.D * sizeof(float) : 0;
}
size_t stat_bytes(const tfu::KvAttendParams& p) { return part_bytes(p) / (p.c.D * sizeof(float)) * sizeof(float2); }

}  // namespace

extern "C" {

TF_API tf_status tf_ulysses_kv_append(const tf_kv_cache* c, int P, int T, int H, tf_dtype dtype, const void* const* k,
                                      const void* const* v, const void* const* q, const tf_strides* strides,
                                      void* const* q_out, const tf_strides* q_out_strides, const tf_norm_rope* nr,
                                      tf_rope rope, int table_rows, void* stream) {
    CallRange call_range("tf_ulysses_kv_append");
    tfu::KvAppendParams p{};
    tf_status s = check_cache(c, P, T, dtype, &p.c);
    if (s != TF_OK) return s;
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    if ((s = rows_of("k", k, &strides[0], P, T, c->Hkv, c->D, false, &p.src[0])) != TF_OK) return s;
    if ((s = rows_of("v", v, &strides[1], P, T, c->Hkv, c->D, false, &p.src[1])) != TF_OK) return s;
    if (!q != !q_out) return fail(TF_ERR_INVALID, "q and q_out are given together or not at all");
    if (q) {
        if (H < 1) return fail(TF_ERR_INVALID, "H=%d must be >= 1", H);
        if (H % P != 0) return fail(TF_ERR_DIVISIBILITY, "H=%d is not divisible by P=%d", H, P);
        if ((s = rows_of("q", q, &strides[2], P, T, H, c->D, false, &p.q)) != TF_OK) return s;
        if ((s = rows_of("q_out", q_out, q_out_strides, P, T, H, c->D, true, &p.q_out)) != TF_OK) return s;
    }
    if (rope != TF_ROPE_NONE && rope != TF_ROPE_INTERLEAVED && rope != TF_ROPE_HALF_SPLIT)
        return fail(TF_ERR_INVALID, "unknown rope %d", int(rope));
    if (rope != TF_ROPE_NONE && !nr) return fail(TF_ERR_INVALID, "the rotation needs norm/rope parameters");
    if (nr) {
        if (!aligned16(nr->q_weight) || !aligned16(nr->k_weight))
            return fail(TF_ERR_ALIGNMENT, "q_weight/k_weight are not 16-byte aligned");
        if ((nr->q_weight || nr->k_weight) && (!std::isfinite(nr->eps) || nr->eps < 0))
            return fail(TF_ERR_INVALID, "eps must be finite and >= 0");
        if (rope != TF_ROPE_NONE) {
            if (nr->cos_sin) {
                if (!aligned16(nr->cos_sin)) return fail(TF_ERR_ALIGNMENT, "cos_sin is not 16-byte aligned");
                if (table_rows < 1) return fail(TF_ERR_INVALID, "table_rows=%d must be >= 1", table_rows);
            } else if (!std::isfinite(nr->theta) || nr->theta <= 0) {
                return fail(TF_ERR_INVALID, "theta must be finite and > 0");
            }
        }
        p.weight[0] = nr->k_weight;
        p.weight[1] = nr->q_weight;
        p.eps = nr->eps;
        p.table = rope != TF_ROPE_NONE ? nr->cos_sin : nullptr;
    }
    const int64_t heads = 2 * int64_t(c->Hkv) + (q ? H : 0);
    const int64_t units = int64_t(T) / c->page_size + 2 * int64_t(c->N);
    if (units * heads >= (int64_t(1) << 31)) return fail(TF_ERR_UNSUPPORTED, "too many heads, rows or sequences");
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (T == 0 || c->N == 0) return TF_OK;
    p.rope = tfu::Rope(int(rope));
    p.table_rows = uint32_t(table_rows);
    p.P = uint32_t(P);
    p.T = uint32_t(T);
    p.Hl = q ? uint32_t(H / P) : 1;
    p.Hkl = uint32_t(c->Hkv / P);
    p.units = uint32_t(units);
    const bool bf16 = dtype == TF_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rope != TF_ROPE_NONE && !p.table) {
        const int rows = c->max_pages * c->page_size;
        s = with_rope_table(nr->theta, rows, c->D, st, [&](const float* table) {
            p.table = table;
            p.table_rows = uint32_t(rows);
            return tfu::launch_kv_append(p, bf16, st);
        });
        if (s != TF_OK) return s;
    } else {
        const cudaError_t e = tfu::launch_kv_append(p, bf16, st);
        if (e != cudaSuccess) return cuda_fail(e, "launching the cache append");
    }
    count_launches(1);
    return TF_OK;
}

TF_API tf_status tf_ulysses_kv_attend_workspace(const tf_kv_cache* c, const tf_kv_attention* a, size_t* bytes) {
    if (!bytes) return fail(TF_ERR_INVALID, "bytes is NULL");
    tfu::KvAttendParams p{};
    tf_status s = check_kv_attention(c, a, &p);
    if (s != TF_OK) return s;
    *bytes = part_bytes(p) + stat_bytes(p);
    return TF_OK;
}

TF_API tf_status tf_ulysses_kv_attend(const tf_kv_cache* c, const tf_kv_attention* a, const void* const* q,
                                      const tf_strides* q_strides, void* const* out, const tf_strides* out_strides,
                                      float* const* lse, void* workspace, size_t workspace_bytes, void* stream) {
    CallRange call_range("tf_ulysses_kv_attend");
    tfu::KvAttendParams p{};
    tf_status s = check_kv_attention(c, a, &p);
    if (s != TF_OK) return s;
    if (!q_strides) return fail(TF_ERR_INVALID, "q_strides is NULL");
    if ((s = rows_of("q", q, q_strides, a->P, a->T, a->H, c->D, false, &p.q)) != TF_OK) return s;
    if ((s = rows_of("out", out, out_strides, a->P, a->T, a->H, c->D, true, &p.out)) != TF_OK) return s;
    for (int g = 0; lse && g < a->P; ++g) {
        if (a->T > 0 && !lse[g]) return fail(TF_ERR_INVALID, "lse[%d] is NULL", g);
        p.lse[g] = lse[g];
    }
    const size_t need = part_bytes(p) + stat_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(TF_ERR_INVALID, "the workspace holds %zu bytes of the %zu needed", workspace ? workspace_bytes : size_t(0), need);
    if (need > 0 && !aligned16(workspace)) return fail(TF_ERR_ALIGNMENT, "the workspace is not 16-byte aligned");
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (a->T == 0 || c->N == 0) return TF_OK;
    if (p.chunks > 1) {
        p.part = static_cast<float*>(workspace);
        p.part_stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + part_bytes(p));
    }
    int launches = 0;
    const cudaError_t e = tfu::launch_kv_attend(p, a->dtype == TF_BF16, static_cast<cudaStream_t>(stream), &launches);
    count_launches(launches);
    if (e != cudaSuccess) return cuda_fail(e, "launching the cache attention");
    return TF_OK;
}

TF_API tf_status tf_ulysses_kv_plan(const tf_kv_plan* p, void* stream) {
    CallRange call_range("tf_ulysses_kv_plan");
    if (!p) return fail(TF_ERR_INVALID, "the plan's description is NULL");
    if (p->N < 0 || p->T < 0) return fail(TF_ERR_INVALID, "N=%d, T=%d must be >= 0", p->N, p->T);
    if (p->max_pages < 1 || p->num_pages < 1)
        return fail(TF_ERR_INVALID, "max_pages=%d, num_pages=%d must be >= 1", p->max_pages, p->num_pages);
    if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
        return fail(TF_ERR_UNSUPPORTED, "the cache is built for pages of 16, 32, 64 or 128 tokens, not %d", p->page_size);
    if (p->N > tfu::kMostRequests) return fail(TF_ERR_UNSUPPORTED, "the plan is built for up to %d requests, not %d", tfu::kMostRequests, p->N);
    if (p->T >= 1 << 30) return fail(TF_ERR_UNSUPPORTED, "T=%d exceeds 2^30 - 1 rows", p->T);
    if (int64_t(p->max_pages) * p->page_size > (int64_t(1) << 30))
        return fail(TF_ERR_UNSUPPORTED, "max_pages * page_size exceeds 2^30 tokens");
    if (int64_t(p->num_pages) * p->page_size >= (int64_t(1) << 31))
        return fail(TF_ERR_UNSUPPORTED, "num_pages * page_size exceeds 2^31 - 1 slots");
    if (p->table_stride < p->max_pages)
        return fail(TF_ERR_INVALID, "table_stride=%lld is below max_pages=%d", (long long)p->table_stride, p->max_pages);
    // by size in entries; of size 0 may be NULL
    const int64_t N = p->N, table = N ? (N - 1) * p->table_stride + p->max_pages : 0;
    const struct {
        const char* name;
        const int32_t* at;
        int64_t size;
    } a[] = {{"page_table", p->page_table, table}, {"free_pages", p->free_pages, p->num_pages}, {"lens_out", p->lens_out, N},
             {"starts", p->starts, N + 1}, {"positions", p->positions, p->T}, {"slots", p->slots, p->T},
             {"span_out", p->span_out, 2}, {"lens", p->lens, N}, {"new_tokens", p->new_tokens, N}, {"free_span", p->free_span, 2}};
    constexpr int kWritten = 7;
    for (const auto& x : a) {
        if (x.size > 0 && !x.at) return fail(TF_ERR_INVALID, "%s is NULL", x.name);
        if (reinterpret_cast<uintptr_t>(x.at) % 4) return fail(TF_ERR_ALIGNMENT, "%s must be 4-byte aligned", x.name);
    }
    for (int i = 0; i < kWritten; ++i)
        for (const auto& y : a)
            if (&y != &a[i] && a[i].size > 0 && y.size > 0 && a[i].at < y.at + y.size && y.at < a[i].at + a[i].size)
                return fail(TF_ERR_INVALID, "%s overlaps %s", a[i].name, y.name);
    int device = 0;
    tf_status s = current_device(&device);
    if (s != TF_OK) return s;
    tfu::KvPlanParams k{};
    k.lens = p->lens;
    k.new_tokens = p->new_tokens;
    k.free_span = p->free_span;
    k.table = p->page_table;
    k.free_pages = p->free_pages;
    k.lens_out = p->lens_out;
    k.starts = p->starts;
    k.positions = p->positions;
    k.slots = p->slots;
    k.span_out = p->span_out;
    k.table_stride = p->table_stride;
    k.N = uint32_t(p->N);
    k.max_pages = uint32_t(p->max_pages);
    k.page = uint32_t(p->page_size);
    while ((1u << k.page_bits) < k.page) ++k.page_bits;
    k.num_pages = uint32_t(p->num_pages);
    k.T = uint32_t(p->T);
    const cudaError_t e = tfu::launch_kv_plan(k, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "launching the cache's plan");
    count_launches(1);
    return TF_OK;
}

}  // extern "C"
