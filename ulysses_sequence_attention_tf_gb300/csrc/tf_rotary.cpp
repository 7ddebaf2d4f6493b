// tf_rotary.cpp -- host side of the rotary positions of tf_ulysses.h: argument checks (all of
// them before any CUDA call), the frequencies, and the launch.
#include <cmath>

#include "host.h"
#include "rotary.h"
#include "rotary_turns.h"

using namespace tfu::host;

namespace {

constexpr double kTurn = 6.283185307179586476925286766559;  // 2 pi

// Heads that one thread takes: as many as leave kRotaryThreads threads, an SM's worth of resident ones twice over (four times
// as many: 24 heads of 12002 tokens, half of D = 64, 14 -> 26 us, for the sines and cosines are computed again), at most
// kRotaryMost -- then these no longer show (8: 80 heads of 32760 tokens 197 -> 217 us).
constexpr uint64_t kRotaryThreads = 2 * 152 * 1024;
constexpr uint32_t kRotaryMost = 16;

tf_status tensor(const char* name, const void* const* in, void* const* out, const tf_strides* in_st, const tf_strides* out_st,
                 const tf_rotary& r, int heads, tfu::RotaryTensor* x) {
    const int hl = heads / r.P;
    const bool empty = r.B == 0 || r.T == 0;
    if (!in || !out) return fail(TF_ERR_INVALID, "%s or %s_out is NULL", name, name);
    tf_status s;
    if (!empty && ((s = check_ptrs(name, in, r.P)) != TF_OK || (s = check_ptrs(name, const_cast<const void* const*>(out), r.P)) != TF_OK))
        return s;
    const tf_strides ost = out_st ? *out_st : tf_strides{int64_t(r.T) * hl * r.D, int64_t(hl) * r.D, r.D};
    if ((s = check_strides(name, *in_st, 2, r.B, r.T, hl)) != TF_OK) return s;
    if ((s = check_strides(name, ost, 2, r.B, r.T, hl)) != TF_OK) return s;
    if (!empty && ((r.B > 1 && ost.b == 0) || (r.T > 1 && ost.t == 0) || (hl > 1 && ost.h == 0)))
        return fail(TF_ERR_INVALID, "%s_out is written and has a stride of 0", name);
    auto same = [](int n, int64_t a, int64_t b) { return n <= 1 || a == b; };
    const bool same_strides = same(r.B, in_st->b, ost.b) && same(r.T, in_st->t, ost.t) && same(hl, in_st->h, ost.h);
    uint32_t in_place = 0;
    for (int g = 0; g < r.P; ++g) {
        x->in[g] = static_cast<const uint8_t*>(in[g]);
        x->out[g] = static_cast<uint8_t*>(out[g]);
        if (in[g] && in[g] == out[g]) ++in_place;
    }
    if (!empty && in_place && !same_strides) return fail(TF_ERR_INVALID, "%s_out is %s with other strides", name, name);
    if (!empty && in_place && in_place != uint32_t(r.P)) return fail(TF_ERR_INVALID, "%s_out is %s in some head groups only", name, name);
    x->ib = in_st->b * 2, x->it = in_st->t * 2, x->ih = in_st->h * 2;
    x->ob = ost.b * 2, x->ot = ost.t * 2, x->oh = ost.h * 2;
    x->Hl = uint32_t(hl);
    x->in_place = in_place != 0;
    return TF_OK;
}

}  // namespace

extern "C" {

TF_API tf_status tf_ulysses_rope_frequencies(int rotary_dim, double theta, tf_rope_scale scale, double factor, double original,
                                             double low, double high, double* out) {
    if (!out) return fail(TF_ERR_INVALID, "out is NULL");
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 256)
        return fail(TF_ERR_INVALID, "rotary_dim=%d is not an even number in [2, 256]", rotary_dim);
    if (!std::isfinite(theta) || theta <= 0) return fail(TF_ERR_INVALID, "theta must be finite and > 0");
    if (scale != TF_ROPE_SCALE_NONE && scale != TF_ROPE_SCALE_LINEAR && scale != TF_ROPE_SCALE_BASE && scale != TF_ROPE_SCALE_PARTS)
        return fail(TF_ERR_INVALID, "unknown scale %d", int(scale));
    if (scale != TF_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor <= 0))
        return fail(TF_ERR_INVALID, "factor must be finite and > 0");
    if (scale == TF_ROPE_SCALE_BASE) {
        if (rotary_dim == 2) return fail(TF_ERR_INVALID, "a scaled base needs rotary_dim > 2");
        theta *= std::pow(factor, double(rotary_dim) / (rotary_dim - 2));
        if (!std::isfinite(theta) || theta <= 0) return fail(TF_ERR_INVALID, "the scaled base is not finite and > 0");
    }
    if (scale == TF_ROPE_SCALE_PARTS &&
        (!std::isfinite(original) || original <= 0 || !std::isfinite(low) || !std::isfinite(high) || !(low < high)))
        return fail(TF_ERR_INVALID, "scaling by parts needs original > 0 and low < high");
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rotary_dim);
        if (scale == TF_ROPE_SCALE_LINEAR) f /= factor;
        if (scale == TF_ROPE_SCALE_PARTS) {
            double keep = (original * f / kTurn - low) / (high - low);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f *= keep + (1 - keep) / factor;
        }
        out[i] = f;
    }
    return TF_OK;
}

TF_API tf_status tf_ulysses_rope(const tf_rotary* r, const void* const* q, const void* const* k, const tf_strides* strides,
                                 void* const* q_out, void* const* k_out, const tf_strides* out_strides, void* stream) {
    CallRange call_range("tf_ulysses_rope");
    if (!r) return fail(TF_ERR_INVALID, "the rotation's description is NULL");
    if (r->P < 1 || r->P > TF_ULYSSES_MAX_SHARDS) return fail(TF_ERR_INVALID, "P=%d outside [1, %d]", r->P, TF_ULYSSES_MAX_SHARDS);
    if (r->B < 0 || r->T < 0) return fail(TF_ERR_INVALID, "B=%d, T=%d must be >= 0", r->B, r->T);
    if (r->H < 1 || (k && r->Hk < 1)) return fail(TF_ERR_INVALID, "H=%d, Hk=%d must be >= 1", r->H, r->Hk);
    if (r->H % r->P != 0 || (k && r->Hk % r->P != 0))
        return fail(TF_ERR_DIVISIBILITY, "H=%d, Hk=%d must be divisible by P=%d", r->H, r->Hk, r->P);
    if (r->D < 8 || r->D > 256 || r->D % 8 != 0)
        return fail(TF_ERR_UNSUPPORTED, "the rotation is built for D a multiple of 8 up to 256, not %d", r->D);
    if (r->rotary_dim < 2 || r->rotary_dim > r->D || r->rotary_dim % 2 != 0)
        return fail(TF_ERR_INVALID, "rotary_dim=%d is not an even number in [2, D=%d]", r->rotary_dim, r->D);
    if (r->dtype != TF_BF16 && r->dtype != TF_FP16)
        return fail(TF_ERR_UNSUPPORTED, "the rotation needs bf16 or fp16 (dtype %d)", int(r->dtype));
    if (r->rope != TF_ROPE_INTERLEAVED && r->rope != TF_ROPE_HALF_SPLIT) return fail(TF_ERR_INVALID, "unknown rope %d", int(r->rope));
    if (r->inverse != 0 && r->inverse != 1) return fail(TF_ERR_INVALID, "inverse=%d is neither 0 nor 1", r->inverse);
    if (!std::isfinite(r->magnitude)) return fail(TF_ERR_INVALID, "magnitude must be finite");
    if (!r->frequencies) return fail(TF_ERR_INVALID, "frequencies is NULL");
    if (!strides) return fail(TF_ERR_INVALID, "strides is NULL");
    if (!k != !k_out) return fail(TF_ERR_INVALID, "k and k_out are given together or not at all");
    tfu::RotaryParams p{};
    for (int i = 0; i < r->rotary_dim / 2; ++i) {
        if (!std::isfinite(r->frequencies[i])) return fail(TF_ERR_INVALID, "frequencies[%d] is not finite", i);
        if (std::fabs(r->frequencies[i]) > tfu::kMostFrequency)
            return fail(TF_ERR_UNSUPPORTED, "frequencies[%d] exceeds 2^60 radians a position", i);
        p.turn[i] = tfu::turn_fraction(r->frequencies[i]);
    }
    if (reinterpret_cast<uintptr_t>(r->positions) % 4) return fail(TF_ERR_ALIGNMENT, "positions must be 4-byte aligned");
    tf_status s = tensor("q", q, q_out, &strides[0], out_strides ? &out_strides[0] : nullptr, *r, r->H, &p.x[0]);
    if (s != TF_OK) return s;
    if (k && (s = tensor("k", k, k_out, &strides[1], out_strides ? &out_strides[1] : nullptr, *r, r->Hk, &p.x[1])) != TF_OK) return s;
    const int64_t heads = int64_t(r->H) + (k ? r->Hk : 0), rows = int64_t(r->B) * r->T;
    if (rows * heads >= (int64_t(1) << 31)) return fail(TF_ERR_UNSUPPORTED, "problem exceeds 2^31 head rows");
    const Named in[2] = {{"q", q}, {"k", k}}, out[2] = {{"q_out", const_cast<const void* const*>(q_out)}, {"k_out", const_cast<const void* const*>(k_out)}};
    if (rows > 0 && (s = check_starts(out, k ? 2 : 1, in, k ? 2 : 1, r->P, true)) != TF_OK) return s;
    int device = 0;
    if ((s = current_device(&device)) != TF_OK) return s;
    if (rows == 0) return TF_OK;
    const bool half_split = r->rope == TF_ROPE_HALF_SPLIT;
    // vectors hold whole pairs' halves: the widest that divides R/2
    uint32_t width = 8;
    while (half_split && (r->rotary_dim / 2) % int(width) != 0) width /= 2;
    p.positions = r->positions;
    p.first = r->first;
    p.B = uint32_t(r->B);
    p.T = uint32_t(r->T);
    p.D = uint32_t(r->D);
    p.R = uint32_t(r->rotary_dim);
    p.q_heads = uint32_t(r->H);
    p.heads = uint32_t(heads);
    p.magnitude = r->magnitude;
    p.sign = r->inverse ? -1.f : 1.f;
    p.items = half_split ? p.R / 2 / width + (p.D - p.R + 2 * width - 1) / (2 * width) : p.D / 8;
    const uint64_t fit = uint64_t(rows) * p.items * p.heads / kRotaryThreads;
    const uint32_t most = fit < 1 ? 1 : fit < kRotaryMost ? uint32_t(fit) : kRotaryMost;
    p.chunks = (p.heads + most - 1) / most;
    p.chunk = (p.heads + p.chunks - 1) / p.chunks;
    p.chunks = (p.heads + p.chunk - 1) / p.chunk;
    const cudaError_t e = tfu::launch_rotary(p, r->dtype == TF_BF16, half_split, width, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "launching the rotation");
    count_launches(1);
    return TF_OK;
}

}  // extern "C"
