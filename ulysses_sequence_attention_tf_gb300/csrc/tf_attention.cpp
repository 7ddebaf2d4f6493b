// tf_attention.cpp -- host side of the attention entry points of tf_ulysses.h:
// argument checks (all of them before any CUDA call) and the launches.
#include <cmath>

#include "attention.h"
#include "host.h"

using namespace tfu::host;

tf_status tfu::host::check_scores(float scale, float softcap) {
    if (!std::isfinite(scale)) return fail(TF_ERR_INVALID, "scale must be finite");
    if (!std::isfinite(softcap) || softcap < 0) return fail(TF_ERR_INVALID, "softcap must be finite and >= 0");
    if (softcap == 0) return TF_OK;
    const float to_x = scale / softcap;
    if ((to_x != 0 && !std::isnormal(to_x)) || softcap > 0x1p127f)
        return fail(TF_ERR_UNSUPPORTED, "softcap=%g: scale / softcap must be 0 or a normal fp32 number, softcap at most 2^127", double(softcap));
    return TF_OK;
}

namespace {

tf_status check_attention(const tf_attention* a) {
    if (!a) return fail(TF_ERR_INVALID, "the attention's description is NULL");
    if (a->P < 1 || a->P > TF_ULYSSES_MAX_SHARDS)
        return fail(TF_ERR_INVALID, "P=%d outside [1, %d]", a->P, TF_ULYSSES_MAX_SHARDS);
    if (a->B < 0 || a->Sq < 0 || a->Sk < 0)
        return fail(TF_ERR_INVALID, "B=%d, Sq=%d, Sk=%d must be >= 0", a->B, a->Sq, a->Sk);
    if (a->H < 1 || a->Hkv < 1) return fail(TF_ERR_INVALID, "H=%d, Hkv=%d must be >= 1", a->H, a->Hkv);
    if (a->Hkv % a->P != 0 || a->H % a->Hkv != 0)
        return fail(TF_ERR_DIVISIBILITY, "Hkv=%d must be divisible by P=%d and H=%d by Hkv", a->Hkv, a->P, a->H);
    if (a->dtype != TF_BF16 && a->dtype != TF_FP16)
        return fail(TF_ERR_UNSUPPORTED, "attention needs bf16 or fp16 (dtype %d)", int(a->dtype));
    if (a->D != 64 && a->D != 128) return fail(TF_ERR_UNSUPPORTED, "attention is built for D in {64, 128}, not %d", a->D);
    const tf_status s = check_scores(a->scale, a->softcap);
    if (s != TF_OK) return s;
    if (a->causal != 0 && a->causal != 1) return fail(TF_ERR_INVALID, "causal=%d is neither 0 nor 1", a->causal);
    if (a->prefix && !a->causal) return fail(TF_ERR_INVALID, "a prefix needs the causal mask");
    if (!a->q_docs != !a->k_docs) return fail(TF_ERR_INVALID, "q_docs and k_docs are given together or not at all");
    if (int64_t(a->Sq) + a->Sk > (int64_t(1) << 30)) return fail(TF_ERR_UNSUPPORTED, "Sq + Sk exceeds 2^30 tokens");
    if (int64_t(a->B) * a->H * ((int64_t(a->Sq > a->Sk ? a->Sq : a->Sk) + 31) / 32) >= (int64_t(1) << 31))
        return fail(TF_ERR_UNSUPPORTED, "problem exceeds 2^31 work units");
    return TF_OK;
}

tf_status view(const char* name, const void* const* base, const tf_strides* given, const tf_attention& a, int64_t tokens,
               int heads, bool written, tfu::GroupView* out) {
    const int64_t hl = heads / a.P;
    const bool empty = a.B == 0 || tokens == 0;
    if (!base) return fail(TF_ERR_INVALID, "%s is NULL", name);
    tf_status s;
    if (!empty && (s = check_ptrs(name, base, a.P)) != TF_OK) return s;
    const tf_strides st = given ? *given : tf_strides{tokens * hl * a.D, hl * a.D, a.D};
    if ((s = check_strides(name, st, 2, a.B, tokens, hl)) != TF_OK) return s;
    for (int g = 0; g < a.P; ++g) out->base[g] = static_cast<uint8_t*>(const_cast<void*>(base[g]));
    out->b = st.b * 2;
    out->t = st.t * 2;
    out->h = st.h * 2;
    if (empty) return TF_OK;  // no element is read or written
    if (!written && ((a.B > 1 && st.b == 0) || (tokens > 1 && st.t == 0) || (hl > 1 && st.h == 0)))
        return fail(TF_ERR_UNSUPPORTED, "%s has a stride of 0 (key heads are shared through Hkv)", name);
    if (written && ((a.B > 1 && st.b == 0) || (tokens > 1 && st.t == 0) || (hl > 1 && st.h == 0)))
        return fail(TF_ERR_INVALID, "%s is written and has a stride of 0", name);
    return TF_OK;
}

void describe(const tf_attention& a, tfu::AttentionParams* p) {
    p->slopes = a.slopes;
    p->prefix = a.prefix;
    p->q_docs = a.q_docs;
    p->k_docs = a.k_docs;
    p->scale = a.scale;
    p->cap = a.softcap;
    p->P = uint32_t(a.P);
    p->B = uint32_t(a.B);
    p->Sq = uint32_t(a.Sq);
    p->Sk = uint32_t(a.Sk);
    p->Hl = uint32_t(a.H / a.P);
    p->Hkl = uint32_t(a.Hkv / a.P);
    p->shared = uint32_t(a.H / a.Hkv);
    p->D = uint32_t(a.D);
    p->causal = uint32_t(a.causal);
}

uint64_t units_of(const tf_attention& a, int tokens, uint32_t rows, int heads) {
    return (uint64_t(tokens) + rows - 1) / rows * uint64_t(a.B) * uint64_t(heads);
}

// How the units of a pass are cut (Split), and the parts of the workspace, in order, each a
// multiple of 16 bytes.
struct Workspace {
    tfu::Split forward{}, dq{}, dkv{};
    size_t delta = 0, plan = 0, key_plan = 0, sizes = 0, parts = 0;  // bytes
    size_t dq_sums = 0;                                   // of the parts: dQ's sums, the statistics behind them
    Workspace(const tf_attention& a, bool backward) {
        auto up = [](size_t n) { return (n + 15) / 16 * 16; };
        const uint32_t B = uint32_t(a.B), Sq = uint32_t(a.Sq), Sk = uint32_t(a.Sk), D = uint32_t(a.D);
        const bool docs = a.q_docs && Sq > 0 && Sk > 0, even = !a.q_docs && !a.causal;
        const uint32_t q_tiles = (Sq + tfu::kAttnRows - 1) / tfu::kAttnRows, k_tiles = (Sk + tfu::kAttnRows - 1) / tfu::kAttnRows;
        auto cut = [](const tfu::Split& s, uint64_t units) { return s.parts > 1 ? (units - s.whole) * s.parts : 0; };
        if (docs) plan = up(tfu::tile_plan(Sq, backward ? tfu::kAttnRows : tfu::kAttnPair, Sk).bytes(B));
        if (!backward) {
            const uint64_t units = units_of(a, a.Sq, tfu::kAttnPair, a.H);
            forward = tfu::plan_split(units, k_tiles, even);
            parts = cut(forward, units) * tfu::kAttnPair * (D * sizeof(float) + sizeof(float2));
            return;
        }
        if (docs) key_plan = up(tfu::tile_plan(Sk, tfu::kAttnRows, Sq).bytes(B));
        delta = up(size_t(B) * size_t(a.H) * Sq * sizeof(float));
        const uint64_t rows = units_of(a, a.Sq, tfu::kAttnRows, a.H), keys = units_of(a, a.Sk, tfu::kAttnRows, a.Hkv);
        if (a.dtype == TF_FP16 && Sq > 0 && Sk > 0) sizes = up(size_t(rows + keys) * sizeof(float));
        dq = tfu::plan_split(rows, k_tiles, even);
        dkv = tfu::plan_split(keys, q_tiles * uint32_t(a.H / a.Hkv), even);
        // one after the other in the same place
        const size_t sums = tfu::kAttnRows * D * sizeof(float);
        dq_sums = 2 * cut(dq, rows) * sums;
        const size_t first = dq_sums + cut(dq, rows) * tfu::kAttnRows * sizeof(float2), second = 2 * cut(dkv, keys) * sums;
        parts = first > second ? first : second;
    }
    size_t bytes() const { return delta + plan + key_plan + sizes + parts; }
};

size_t workspace_bytes_of(const tf_attention& a, bool backward) { return Workspace(a, backward).bytes(); }

tf_status check_workspace(const tf_attention& a, bool backward, const void* workspace, size_t bytes) {
    const size_t need = workspace_bytes_of(a, backward);
    if (need == 0) return TF_OK;
    if (!workspace || bytes < need)
        return fail(TF_ERR_INVALID, "the workspace holds %zu bytes of the %zu needed", workspace ? bytes : size_t(0), need);
    if (!aligned16(workspace)) return fail(TF_ERR_ALIGNMENT, "the workspace is not 16-byte aligned");
    return TF_OK;
}

}  // namespace

extern "C" {

TF_API tf_status tf_ulysses_attention_workspace(const tf_attention* a, int backward, size_t* bytes) {
    if (!bytes) return fail(TF_ERR_INVALID, "bytes is NULL");
    tf_status s = check_attention(a);
    if (s != TF_OK) return s;
    *bytes = workspace_bytes_of(*a, backward != 0);
    return TF_OK;
}

TF_API tf_status tf_ulysses_attention(const tf_attention* a, const void* const* q, const void* const* k,
                                      const void* const* v, const tf_strides* strides, void* const* out,
                                      const tf_strides* out_strides, float* const* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    CallRange call_range("tf_ulysses_attention");
    tf_status s = check_attention(a);
    if (s != TF_OK) return s;
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    tfu::ForwardParams fp;  // tensor maps of absent groups stay unset
    fp.a = tfu::AttentionParams{};
    tfu::AttentionParams& p = fp.a;
    if ((s = view("q", q, &strides[0], *a, a->Sq, a->H, false, &p.q)) != TF_OK) return s;
    if ((s = view("k", k, &strides[1], *a, a->Sk, a->Hkv, false, &p.k)) != TF_OK) return s;
    if ((s = view("v", v, &strides[2], *a, a->Sk, a->Hkv, false, &p.v)) != TF_OK) return s;
    if ((s = view("out", out, out_strides, *a, a->Sq, a->H, true, &p.out)) != TF_OK) return s;
    const bool empty = a->B == 0 || a->Sq == 0;
    for (int g = 0; lse && g < a->P; ++g) {
        if (!empty && !lse[g]) return fail(TF_ERR_INVALID, "lse[%d] is NULL", g);
        p.lse[g] = lse[g];
    }
    if ((s = check_workspace(*a, false, workspace, workspace_bytes)) != TF_OK) return s;
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (empty) return TF_OK;
    describe(*a, &p);
    const bool bf16 = a->dtype == TF_BF16;
    if (!tfu::encode_group_maps(&fp.q, p.q, p.P, p.B, p.Sq, p.Hl, p.D, tfu::kAttnRows, bf16) ||
        (a->Sk > 0 && (!tfu::encode_group_maps(&fp.k, p.k, p.P, p.B, p.Sk, p.Hkl, p.D, tfu::kAttnRows, bf16) ||
                       !tfu::encode_group_maps(&fp.v, p.v, p.P, p.B, p.Sk, p.Hkl, p.D, tfu::kAttnRows, bf16))))
        return fail(TF_ERR_UNSUPPORTED, "the driver refused a tensor map of q, k or v");
    const Workspace ws(*a, false);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    p.plan = ws.plan > 0 ? reinterpret_cast<uint32_t*>(at) : nullptr;
    fp.split = ws.forward;
    if (ws.parts > 0) {
        const size_t rows = ws.parts / (size_t(a->D) * sizeof(float) + sizeof(float2));
        fp.split.part = reinterpret_cast<float*>(at + ws.plan);
        fp.split.stat = reinterpret_cast<float2*>(fp.split.part + rows * size_t(a->D));
    }
    fp.q_tiles = (p.Sq + tfu::kAttnPair - 1) / tfu::kAttnPair;
    fp.ranked = p.plan && tfu::rank_units(uint64_t(p.B) * fp.q_tiles, tfu::tile_plan(p.Sq, tfu::kAttnPair, p.Sk).words,
                                          uint64_t(a->B) * a->Hkv, p.Sk, p.D);
    fp.head_block = tfu::head_block(a->causal, uint64_t(a->B) * a->H, p.Sk, p.D);
    int launches = 0;
    const cudaError_t e = tfu::launch_attention(fp, bf16, static_cast<cudaStream_t>(stream), &launches);
    count_launches(launches);
    if (e != cudaSuccess) return cuda_fail(e, "launching the attention kernel");
    return TF_OK;
}

TF_API tf_status tf_ulysses_attention_backward(const tf_attention* a, const void* const* dout, const void* const* q,
                                               const void* const* k, const void* const* v, const void* const* out,
                                               const float* const* lse, const tf_strides* strides, void* const* dq,
                                               void* const* dk, void* const* dv, const tf_strides* grad_strides,
                                               void* workspace, size_t workspace_bytes, void* stream) {
    CallRange call_range("tf_ulysses_attention_backward");
    tf_status s = check_attention(a);
    if (s != TF_OK) return s;
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    tfu::BackwardParams bp;  // tensor maps of absent groups stay unset
    bp.a = tfu::AttentionParams{};
    tfu::AttentionParams& p = bp.a;
    if ((s = view("dout", dout, &strides[0], *a, a->Sq, a->H, false, &p.dout)) != TF_OK) return s;
    if ((s = view("q", q, &strides[1], *a, a->Sq, a->H, false, &p.q)) != TF_OK) return s;
    if ((s = view("k", k, &strides[2], *a, a->Sk, a->Hkv, false, &p.k)) != TF_OK) return s;
    if ((s = view("v", v, &strides[3], *a, a->Sk, a->Hkv, false, &p.v)) != TF_OK) return s;
    if ((s = view("out", out, &strides[4], *a, a->Sq, a->H, false, &p.out)) != TF_OK) return s;
    const tf_strides* gs = grad_strides;
    if ((s = view("dq", dq, gs ? &gs[0] : nullptr, *a, a->Sq, a->H, true, &p.dq)) != TF_OK) return s;
    if ((s = view("dk", dk, gs ? &gs[1] : nullptr, *a, a->Sk, a->Hkv, true, &p.dk)) != TF_OK) return s;
    if ((s = view("dv", dv, gs ? &gs[2] : nullptr, *a, a->Sk, a->Hkv, true, &p.dv)) != TF_OK) return s;
    if (!lse) return fail(TF_ERR_INVALID, "lse is NULL");
    for (int g = 0; g < a->P; ++g) {
        if (a->B > 0 && a->Sq > 0 && !lse[g]) return fail(TF_ERR_INVALID, "lse[%d] is NULL", g);
        p.lse[g] = const_cast<float*>(lse[g]);
    }
    if ((s = check_workspace(*a, true, workspace, workspace_bytes)) != TF_OK) return s;
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (a->B == 0 || (a->Sq == 0 && a->Sk == 0)) return TF_OK;
    describe(*a, &p);
    const bool bf16 = a->dtype == TF_BF16;
    auto query_maps = [&](tfu::GroupMaps* m, const tfu::GroupView& v, uint32_t box) {
        return a->Sq == 0 || tfu::encode_group_maps(m, v, p.P, p.B, p.Sq, p.Hl, p.D, box, bf16);
    };
    auto key_maps = [&](tfu::GroupMaps* m, const tfu::GroupView& v) {
        return a->Sk == 0 || tfu::encode_group_maps(m, v, p.P, p.B, p.Sk, p.Hkl, p.D, tfu::kAttnRows, bf16);
    };
    if (!query_maps(&bp.q, p.q, tfu::kAttnRows) || !query_maps(&bp.dout, p.dout, tfu::kAttnRows) ||
        !query_maps(&bp.q_half, p.q, tfu::kAttnRows / 2) || !query_maps(&bp.dout_half, p.dout, tfu::kAttnRows / 2) ||
        !key_maps(&bp.k, p.k) || !key_maps(&bp.v, p.v))
        return fail(TF_ERR_UNSUPPORTED, "the driver refused a tensor map of dout, q, k or v");
    const Workspace ws(*a, true);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    p.delta = reinterpret_cast<float*>(at);
    p.plan = ws.plan > 0 ? reinterpret_cast<uint32_t*>(at + ws.delta) : nullptr;
    bp.key_plan = ws.plan > 0 ? reinterpret_cast<uint32_t*>(at + ws.delta + ws.plan) : nullptr;
    bp.sizes = reinterpret_cast<float*>(at + ws.delta + ws.plan + ws.key_plan);
    bp.dq_split = ws.dq;
    bp.dkv_split = ws.dkv;
    bp.dq_split.part = bp.dkv_split.part = reinterpret_cast<float*>(at + ws.delta + ws.plan + ws.key_plan + ws.sizes);
    if (bp.dq_split.parts > 1) bp.dq_split.stat = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(bp.dq_split.part) + ws.dq_sums);
    bp.q_tiles = (p.Sq + tfu::kAttnRows - 1) / tfu::kAttnRows;
    bp.k_tiles = (p.Sk + tfu::kAttnRows - 1) / tfu::kAttnRows;
    bp.head_block = tfu::head_block(a->causal, uint64_t(a->B) * a->H, p.Sk, p.D);
    bp.key_head_block = tfu::head_block(a->causal, uint64_t(a->B) * a->Hkv, uint64_t(p.Sq) * p.shared, p.D);
    int launches = 0;
    const cudaError_t e = tfu::launch_attention_backward(bp, bf16, static_cast<cudaStream_t>(stream), &launches);
    count_launches(launches);
    if (e != cudaSuccess) return cuda_fail(e, "launching the attention's gradient kernels");
    return TF_OK;
}

}  // extern "C"
