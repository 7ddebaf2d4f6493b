// tf_linear.cpp -- host side of the linear attention entry points of tf_ulysses.h:
// argument checks (all of them before any CUDA call) and the launches.
#include <cmath>

#include "host.h"
#include "linear.h"

using namespace tfu::host;

namespace {

tf_status check_linear(const tf_linear* a) {
    if (!a) return fail(TF_ERR_INVALID, "the linear attention's description is NULL");
    if (a->P < 1 || a->P > TF_ULYSSES_MAX_SHARDS)
        return fail(TF_ERR_INVALID, "P=%d outside [1, %d]", a->P, TF_ULYSSES_MAX_SHARDS);
    if (a->B < 0 || a->S < 0) return fail(TF_ERR_INVALID, "B=%d, S=%d must be >= 0", a->B, a->S);
    if (a->H < 1) return fail(TF_ERR_INVALID, "H=%d must be >= 1", a->H);
    if (a->H % a->P != 0) return fail(TF_ERR_DIVISIBILITY, "H=%d is not divisible by P=%d", a->H, a->P);
    if (a->dtype != TF_BF16 && a->dtype != TF_FP16)
        return fail(TF_ERR_UNSUPPORTED, "linear attention needs bf16 or fp16 (dtype %d)", int(a->dtype));
    if (a->D != 64 && a->D != 128) return fail(TF_ERR_UNSUPPORTED, "linear attention is built for D in {64, 128}, not %d", a->D);
    if (!std::isfinite(a->scale)) return fail(TF_ERR_INVALID, "scale must be finite");
    if (!a->decay) return fail(TF_ERR_INVALID, "decay is NULL");
    if (reinterpret_cast<uintptr_t>(a->decay) % 4) return fail(TF_ERR_ALIGNMENT, "decay must be 4-byte aligned");
    if (a->S > 1 << 30) return fail(TF_ERR_UNSUPPORTED, "S exceeds 2^30 tokens");
    // without tokens a state is still copied
    if (int64_t(a->B) * a->H >= (int64_t(1) << 28) || int64_t(a->B) * a->H * ((int64_t(a->S) + 127) / 128) >= (int64_t(1) << 28))
        return fail(TF_ERR_UNSUPPORTED, "problem exceeds 2^28 work units");
    return TF_OK;
}

tf_status view(const char* name, const void* const* base, const tf_strides* given, const tf_linear& a, bool written, tfu::GroupView* out) {
    const int64_t hl = a.H / a.P;
    const bool empty = a.B == 0 || a.S == 0;
    if (!base) return fail(TF_ERR_INVALID, "%s is NULL", name);
    tf_status s;
    if (!empty && (s = check_ptrs(name, base, a.P)) != TF_OK) return s;
    const tf_strides st = given ? *given : tf_strides{a.S * hl * a.D, hl * a.D, a.D};
    if ((s = check_strides(name, st, 2, a.B, a.S, hl)) != TF_OK) return s;
    for (int g = 0; g < a.P; ++g) out->base[g] = static_cast<uint8_t*>(const_cast<void*>(base[g]));
    out->b = st.b * 2;
    out->t = st.t * 2;
    out->h = st.h * 2;
    if (!empty && ((a.B > 1 && st.b == 0) || (a.S > 1 && st.t == 0) || (hl > 1 && st.h == 0)))
        return fail(written ? TF_ERR_INVALID : TF_ERR_UNSUPPORTED, "%s has a stride of 0", name);
    return TF_OK;
}

const void* const* starts(void* const* p) { return const_cast<const void* const*>(p); }

tf_status check_state(const char* name, const float* s) {
    return reinterpret_cast<uintptr_t>(s) % 32 == 0 ? TF_OK : fail(TF_ERR_ALIGNMENT, "%s is not 32-byte aligned", name);
}

// Two states over the same memory, `same` excepted where it is the very same.
tf_status check_apart(const char* written, const float* to, const char* read, const float* from, const tf_linear& a, bool same) {
    const int64_t n = int64_t(a.B) * a.H * a.D * a.D;
    if (!to || !from || (same && to == from)) return TF_OK;
    return to < from + n && from < to + n ? fail(TF_ERR_INVALID, "%s overlaps %s", written, read) : TF_OK;
}

tf_status check_workspace(size_t need, const void* workspace, size_t bytes) {
    if (need == 0) return TF_OK;
    if (!workspace || bytes < need)
        return fail(TF_ERR_INVALID, "the workspace holds %zu bytes of the %zu needed", workspace ? bytes : size_t(0), need);
    if (reinterpret_cast<uintptr_t>(workspace) % 32) return fail(TF_ERR_ALIGNMENT, "the workspace is not 32-byte aligned");
    return TF_OK;
}

tfu::LinearPass pass_of(const tf_linear& a) {
    tfu::LinearPass p{};
    p.decay = a.decay;
    p.P = uint32_t(a.P);
    p.N = uint32_t(a.B);
    p.S = p.most = uint32_t(a.S);
    p.Hl = uint32_t(a.H / a.P);
    p.D = uint32_t(a.D);
    p.kv_scale = 1.f;
    p.out_scale = a.scale;
    return p;
}

// Up to this many tokens of a sequence go token by token; more in chunks.  A chunk costs the same for one token and 128, about 12
// us of a CTA with its state's way in and out at D = 128, a token 0.5 us.  One round of CTAs: 8 tokens 14 against 13 us, 16
// tokens 22 against 13 (8 sequences, 16 heads).  Many, at D = 128 and 64: 8 tokens 99 against 163 us, 26 against 97, 16
// tokens 162 against 163, 44 against 96 (64 sequences, 32 heads), because the steps' CTAs share an SM.
uint32_t steps_most(const tfu::LinearPass& p) { return uint64_t(p.N) * p.P * p.Hl > 2 * tfu::kAttnSms ? 16 : 8; }

// How the sequences are cut.  A CTA runs alone on its SM; `units` sequences and heads of `chunks` chunks each.  In chunks of
// time, a CTA's start costs kStart, the sums of a segment kSums of a chunk each (K and V only), their join kJoin.  64 segments at
// most bound the search and the workspace, so one or two heads leave SMs free from 65 chunks on (one head of 131072 tokens: 104 us).
struct Cut {
    uint32_t segments = 1, seg_chunks = 0;
};
Cut plan_cut(uint64_t units, uint32_t chunks) {
    constexpr double kStart = 3, kSums = 0.6, kJoin = 1.5;
    Cut best;
    double least = 0;
    for (uint32_t want = 1; want <= chunks && want <= 64; ++want) {
        const uint32_t size = (chunks + want - 1) / want, n = (chunks + size - 1) / size;
        if (n != want) continue;
        auto rounds = [&](uint64_t ctas) { return double((ctas + tfu::kAttnSms - 1) / tfu::kAttnSms); };
        const double cost = rounds(units * n) * (size + kStart) + (n > 1 ? rounds(units * (n - 1)) * (kSums * size + kStart) + kJoin : 0);
        if (want == 1 || cost < least) {
            least = cost;
            best.segments = n;
            best.seg_chunks = size;
        }
    }
    return best;
}
Cut cut_of(const tfu::LinearPass& p, uint32_t passes) {
    if (p.most <= steps_most(p)) return {};
    return plan_cut(uint64_t(passes) * p.N * p.P * p.Hl, (p.most + tfu::kLinearChunk - 1) / tfu::kLinearChunk);
}

size_t workspace_of(const tfu::LinearPass& p, uint32_t passes) {
    const uint32_t segments = cut_of(p, passes).segments;
    return segments > 1 ? size_t(passes) * segments * p.N * p.P * p.Hl * p.D * p.D * sizeof(float) : 0;
}

// Passes over the same sequences that depend on one another in nothing: tensor[i] are pass i's q, k, v among `views`.
tf_status run(const tfu::LinearPass* p, uint32_t passes, const tfu::GroupView* views, uint32_t tensors,
              const uint32_t (*tensor)[3], bool bf16, void* workspace, cudaStream_t stream) {
    int launches = 0;
    cudaError_t e = cudaSuccess;
    if (p->most <= steps_most(*p)) {
        for (uint32_t i = 0; i < passes && e == cudaSuccess; ++i, ++launches) e = tfu::launch_linear_steps(p[i], bf16, stream);
    } else {
        tfu::LinearChunkParams c{};
        const uint32_t B = p->starts ? 1 : p->N;
        for (uint32_t i = 0; i < tensors; ++i)
            if (!tfu::encode_group_maps(&c.maps[i], views[i], p->P, B, p->S, p->Hl, p->D, tfu::kLinearChunk, bf16))
                return fail(TF_ERR_UNSUPPORTED, "the driver refuses a tensor map of these views");
        const Cut cut = cut_of(*p, passes);
        c.passes = passes;
        c.segments = cut.segments;
        c.seg_chunks = cut.seg_chunks;
        c.parts = static_cast<float*>(workspace);
        for (uint32_t i = 0; i < passes; ++i) {
            c.pass[i] = p[i];
            for (int x = 0; x < 3; ++x) c.tensor[i][x] = tensor[i][x];
            uintptr_t bits = uintptr_t(p[i].out.b | p[i].out.t | p[i].out.h);
            for (uint32_t g = 0; g < p->P; ++g) bits |= reinterpret_cast<uintptr_t>(p[i].out.base[g]);
            c.wide_out[i] = bits % 32 == 0;
        }
        e = tfu::launch_linear_chunks(c, bf16, stream, &launches);
    }
    if (e != cudaSuccess) return cuda_fail(e, "launching linear attention");
    count_launches(launches);
    return TF_OK;
}
constexpr uint32_t kInOrder[1][3] = {{0, 1, 2}};

tf_status check_pool(const tf_linear* a, const tf_linear_pool* pool, tfu::LinearPass* p) {
    tf_status s = check_linear(a);
    if (s != TF_OK) return s;
    if (!pool) return fail(TF_ERR_INVALID, "the pool's description is NULL");
    if (a->B != 1) return fail(TF_ERR_INVALID, "B=%d must be 1 for rows", a->B);
    if (pool->N < 0 || pool->num_slots < 1)
        return fail(TF_ERR_INVALID, "N=%d must be >= 0 and num_slots=%d >= 1", pool->N, pool->num_slots);
    if (!pool->states || !pool->starts || (pool->N > 0 && !pool->slots))
        return fail(TF_ERR_INVALID, "the pool's states, slots or starts are NULL");
    if ((s = check_state("states", pool->states)) != TF_OK) return s;
    if (reinterpret_cast<uintptr_t>(pool->slots) % 4 || reinterpret_cast<uintptr_t>(pool->starts) % 4)
        return fail(TF_ERR_ALIGNMENT, "slots and starts must be 4-byte aligned");
    if (a->S > 0 && (pool->max_tokens < 1 || pool->max_tokens > a->S))
        return fail(TF_ERR_INVALID, "max_tokens=%d outside [1, T=%d]", pool->max_tokens, a->S);
    if (int64_t(pool->N) * a->H >= (int64_t(1) << 28) ||
        int64_t(pool->N) * a->H * ((int64_t(pool->max_tokens) + 127) / 128) >= (int64_t(1) << 28))
        return fail(TF_ERR_UNSUPPORTED, "problem exceeds 2^28 work units");
    *p = pass_of(*a);
    p->N = uint32_t(pool->N);
    p->most = uint32_t(pool->max_tokens);
    p->starts = pool->starts;
    p->slots = pool->slots;
    p->num_slots = uint32_t(pool->num_slots);
    p->state = p->final_state = pool->states;
    return TF_OK;
}

}  // namespace

extern "C" {

TF_API tf_status tf_ulysses_linear_attention_workspace(const tf_linear* a, int backward, size_t* bytes) {
    if (!bytes) return fail(TF_ERR_INVALID, "bytes is NULL");
    const tf_status s = check_linear(a);
    if (s != TF_OK) return s;
    *bytes = workspace_of(pass_of(*a), backward ? 3 : 1);
    return TF_OK;
}

TF_API tf_status tf_ulysses_linear_attention(const tf_linear* a, const void* const* q, const void* const* k,
                                             const void* const* v, const tf_strides* strides, const float* state,
                                             void* const* out, const tf_strides* out_strides, float* final_state,
                                             void* workspace, size_t workspace_bytes, void* stream) {
    CallRange call_range("tf_ulysses_linear_attention");
    tf_status s = check_linear(a);
    if (s != TF_OK) return s;
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    tfu::LinearPass p = pass_of(*a);
    if ((s = view("q", q, &strides[0], *a, false, &p.q)) != TF_OK || (s = view("k", k, &strides[1], *a, false, &p.k)) != TF_OK ||
        (s = view("v", v, &strides[2], *a, false, &p.v)) != TF_OK || (s = view("out", out, out_strides, *a, true, &p.out)) != TF_OK)
        return s;
    if ((s = check_state("state", state)) != TF_OK || (s = check_state("final_state", final_state)) != TF_OK) return s;
    if ((s = check_apart("final_state", final_state, "state", state, *a, true)) != TF_OK) return s;
    const Named in[3] = {{"q", q}, {"k", k}, {"v", v}}, written{"out", starts(out)};
    if (a->B > 0 && a->S > 0 && (s = check_starts(&written, 1, in, 3, a->P, false)) != TF_OK) return s;
    if ((s = check_workspace(workspace_of(p, 1), workspace, workspace_bytes)) != TF_OK) return s;
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (a->B == 0 || (a->S == 0 && !final_state)) return TF_OK;
    p.state = state;
    p.final_state = final_state;
    const tfu::GroupView views[3] = {p.q, p.k, p.v};
    return run(&p, 1, views, 3, kInOrder, a->dtype == TF_BF16, workspace, static_cast<cudaStream_t>(stream));
}

TF_API tf_status tf_ulysses_linear_attention_backward(const tf_linear* a, const void* const* dout, const void* const* q,
                                                      const void* const* k, const void* const* v,
                                                      const tf_strides* strides, const float* state,
                                                      const float* dfinal_state, void* const* dq, void* const* dk,
                                                      void* const* dv, const tf_strides* grad_strides, float* dstate,
                                                      void* workspace, size_t workspace_bytes, void* stream) {
    CallRange call_range("tf_ulysses_linear_attention_backward");
    tf_status s = check_linear(a);
    if (s != TF_OK) return s;
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    const tf_strides* gs = grad_strides;
    tfu::GroupView vdout, vq, vk, vv, vdq, vdk, vdv;
    if ((s = view("dout", dout, &strides[0], *a, false, &vdout)) != TF_OK || (s = view("q", q, &strides[1], *a, false, &vq)) != TF_OK ||
        (s = view("k", k, &strides[2], *a, false, &vk)) != TF_OK || (s = view("v", v, &strides[3], *a, false, &vv)) != TF_OK ||
        (s = view("dq", dq, gs ? &gs[0] : nullptr, *a, true, &vdq)) != TF_OK ||
        (s = view("dk", dk, gs ? &gs[1] : nullptr, *a, true, &vdk)) != TF_OK ||
        (s = view("dv", dv, gs ? &gs[2] : nullptr, *a, true, &vdv)) != TF_OK)
        return s;
    if ((s = check_state("state", state)) != TF_OK || (s = check_state("dfinal_state", dfinal_state)) != TF_OK ||
        (s = check_state("dstate", dstate)) != TF_OK)
        return s;
    // the passes run together: one reads what another would write
    if ((s = check_apart("dstate", dstate, "dfinal_state", dfinal_state, *a, false)) != TF_OK ||
        (s = check_apart("dstate", dstate, "state", state, *a, false)) != TF_OK)
        return s;
    const Named in[4] = {{"dout", dout}, {"q", q}, {"k", k}, {"v", v}}, written[3] = {{"dq", starts(dq)}, {"dk", starts(dk)}, {"dv", starts(dv)}};
    if (a->B > 0 && a->S > 0 && (s = check_starts(written, 3, in, 4, a->P, false)) != TF_OK) return s;
    const tfu::LinearPass all = pass_of(*a);
    if ((s = check_workspace(workspace_of(all, 3), workspace, workspace_bytes)) != TF_OK) return s;
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (a->B == 0 || (a->S == 0 && !dstate)) return TF_OK;
    const tfu::GroupView views[4] = {vdout, vq, vk, vv};
    constexpr uint32_t kRoles[3][3] = {{0, 3, 2}, {3, 0, 1}, {2, 1, 0}};  // dq: (dout, v, k), dk: (v, dout, q), dv: (k, q, dout)
    tfu::LinearPass p[3] = {all, all, all};
    for (int i = 0; i < 3; ++i) {
        p[i].q = views[kRoles[i][0]], p[i].k = views[kRoles[i][1]], p[i].v = views[kRoles[i][2]];
        p[i].state = i == 0 ? state : dfinal_state;
        p[i].transposed = i < 2;
        p[i].reverse = i > 0;
        if (i > 0) p[i].kv_scale = a->scale, p[i].out_scale = 1.f;
    }
    p[0].out = vdq, p[1].out = vdk, p[2].out = vdv;
    p[2].final_state = dstate;
    const bool bf16 = a->dtype == TF_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->S == 0) return run(&p[2], 1, views, 4, kRoles + 2, bf16, workspace, st);
    return run(p, 3, views, 4, kRoles, bf16, workspace, st);
}

TF_API tf_status tf_ulysses_linear_attend_workspace(const tf_linear* a, const tf_linear_pool* pool, size_t* bytes) {
    if (!bytes) return fail(TF_ERR_INVALID, "bytes is NULL");
    tfu::LinearPass p{};
    const tf_status s = check_pool(a, pool, &p);
    if (s != TF_OK) return s;
    *bytes = workspace_of(p, 1);
    return TF_OK;
}

TF_API tf_status tf_ulysses_linear_attend(const tf_linear* a, const tf_linear_pool* pool, const void* const* q,
                                          const void* const* k, const void* const* v, const tf_strides* strides,
                                          void* const* out, const tf_strides* out_strides, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    CallRange call_range("tf_ulysses_linear_attend");
    tfu::LinearPass p{};
    tf_status s = check_pool(a, pool, &p);
    if (s != TF_OK) return s;
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    if ((s = view("q", q, &strides[0], *a, false, &p.q)) != TF_OK || (s = view("k", k, &strides[1], *a, false, &p.k)) != TF_OK ||
        (s = view("v", v, &strides[2], *a, false, &p.v)) != TF_OK || (s = view("out", out, out_strides, *a, true, &p.out)) != TF_OK)
        return s;
    const Named in[3] = {{"q", q}, {"k", k}, {"v", v}}, written{"out", starts(out)};
    if (a->S > 0 && (s = check_starts(&written, 1, in, 3, a->P, false)) != TF_OK) return s;
    if ((s = check_workspace(workspace_of(p, 1), workspace, workspace_bytes)) != TF_OK) return s;
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (a->S == 0 || pool->N == 0) return TF_OK;
    const tfu::GroupView views[3] = {p.q, p.k, p.v};
    return run(&p, 1, views, 3, kInOrder, a->dtype == TF_BF16, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
