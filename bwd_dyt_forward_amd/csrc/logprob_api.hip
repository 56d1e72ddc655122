// logprob_api.hip - C ABI of the token log probabilities (include/dyt_lm.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "block_host.hpp"
#include "dyt_lm.h"
#include "logprob_launch.hpp"

namespace dytb {
namespace {

static_assert(kLpMaxTop == DYT_LOGPROB_MAX_TOP, "the kernels' limit is the header's");
constexpr int64_t kMaxV = (int64_t)1 << 26;
constexpr int64_t kPastCache = (int64_t)256 << 20;   // the last-level cache
// With alternatives: lines of a part and parts of a row, for what of both is in
// LDS (51 KB of maxima and candidates of a part, 32 KB of candidates of a row),
// and the longest row that they leave.
constexpr int64_t kMaxLines = 4096, kMaxTopParts = 64;
constexpr int64_t kMaxTopV = (int64_t)1 << 23;
static_assert(kMaxTopV <= kMaxTopParts * kMaxLines * 8 * 4, "float32 lines have 32 elements");

int lp_shape(int64_t T, int64_t V, int top, int dt) {
    if (T < 0 || V < 0 || T > 0x7fffffff || V > kMaxV || top < 0 || top > kLpMaxTop || top > V ||
        (top > 0 && V > kMaxTopV))
        return DYT_ERR_INVALID_ARG;
    return dtype_ok(dt) ? DYT_OK : DYT_ERR_UNSUPPORTED_DTYPE;
}

// Lanes of a row, parts of a row and their columns. Rows of up to 128 vectors
// take a power of two of lanes up to a wave; longer ones, and any with
// alternatives, a workgroup. Fewer than 512 such rows would leave most of the
// card idle: they are cut into parts, as many as make 1,024 workgroups, of four
// vectors a thread at least.
struct LpPlan {
    int tpr, parts;
    int64_t part_len;
    size_t shared, join_shared, part_bytes, bytes;
};

LpPlan lp_plan(int64_t T, int64_t V, int top, int dt, bool backward = false) {
    LpPlan p{};
    const int64_t vec = 16 / dtype_size(dt), nv = (V + vec - 1) / vec;
    p.tpr = 256;
    if (!top && nv <= 128) {
        p.tpr = 1;
        while (p.tpr < nv && p.tpr < 64) p.tpr *= 2;
    }
    int64_t parts = 1;
    const int64_t step = 256 * vec;   // one vector of every thread
    if (p.tpr == 256 && T < 512) parts = std::min((1024 + T - 1) / T, (nv + 1023) / 1024);
    if (top) parts = std::min(std::max(parts, (V + kMaxLines * 8 * vec - 1) / (kMaxLines * 8 * vec)), kMaxTopParts);
    parts = std::min<int64_t>(parts, 256);
    if (backward && p.tpr == 256) {
        // tiles that follow each other in memory: 290 us for 320 of a workgroup for each row
        p.part_len = kLpBwdVecs * step;
        p.parts = (int)((V + vec - 1 + p.part_len - 1) / p.part_len);
        return p;
    }
    // a row may begin up to vec - 1 places after the 16-byte grid
    const int64_t places = V + vec - 1;
    p.part_len = p.tpr == 256 ? ((places + parts - 1) / parts + step - 1) / step * step : places;
    p.parts = (int)((places + p.part_len - 1) / p.part_len);
    if (top) {
        const int64_t lines = p.part_len / (8 * vec);
        p.shared = (size_t)((lines + 1) / 2 + top * 4 * std::max((lines + 255) / 256, 2 * vec)) * 8;
        p.join_shared = (size_t)(top * 4 * ((p.parts * top + 255) / 256)) * 8;
    }
    if (p.parts > 1) {
        p.part_bytes = (size_t)T * p.parts * 16;
        p.bytes = p.part_bytes + (size_t)T * p.parts * top * 8;
    }
    return p;
}

// A launch has fewer than 2^32 threads, 2^24 workgroups: more rows than that take
// several, launch(arguments, workgroups) for each run of rows.
template <typename Launch>
void in_launches(LpArgs a, const LpPlan& p, int64_t elem_bytes, Launch&& launch) {
    const int64_t per = 256 / p.tpr, most = (((int64_t)1 << 24) - 1) * per / p.parts, T = a.T;
    for (int64_t done = 0; done < T; done += a.T) {
        a.T = std::min(most, T - done);
        launch(a, (a.T * p.parts + per - 1) / per);
        const int64_t n = a.T;
        const auto on = [n](auto*& q, int64_t of_row) {
            using Q = std::remove_reference_t<decltype(q)>;
            if (q) q = (Q)((uintptr_t)q + (uintptr_t)(n * of_row));
        };
        on(a.logits, a.ld * elem_bytes);
        on(a.dlogits, a.ldd * elem_bytes);
        on(a.tokens, a.token_bits / 8);
        for (float** q : {&a.logp, &a.entropy, &a.lse}) on(*q, 4);
        for (const float** q : {&a.dlogp, &a.dentropy}) on(*q, 4);
        on(a.norm, 12);
        on(a.top_logp, 4 * (int64_t)a.top);
        on(a.top_tokens, 8 * (int64_t)a.top);
        on(a.part, 16 * (int64_t)p.parts);
        on(a.part_top, 8 * (int64_t)p.parts * a.top);
    }
}

template <typename F>
void with_type(int dt, F&& f) {
    if (dt == DYT_F32) f((float*)nullptr);
    else if (dt == DYT_BF16) f((bf16_t*)nullptr);
    else f((f16_t*)nullptr);
}

int lp_forward(const void* logits, int64_t ld, const void* tokens, float* logp, float* entropy, float* lse,
               float* norm, float* top_logp, int64_t* top_tokens, void* ws, size_t ws_bytes, int64_t T, int64_t V, float scale,
               int top, int dt, int bits, void* stream) {
    if (int e = lp_shape(T, V, top, dt)) return e;
    if (ld == 0) ld = V;
    if ((bits != 32 && bits != 64) || !(scale > 0.0f) || std::isinf(scale) || !pitch_ok(T, V, ld)) return DYT_ERR_INVALID_ARG;
    if (T == 0) return DYT_OK;
    if (V == 0 || !logits || !tokens || !logp || !entropy || !lse || (top > 0) != (top_logp != nullptr) ||
        (top > 0) != (top_tokens != nullptr))
        return DYT_ERR_INVALID_ARG;
    const int64_t s = dtype_size(dt);
    if (!aligned({logits}, s) || !aligned({tokens}, bits / 8) || !aligned({logp, entropy, lse, norm, top_logp}, 4) ||
        !aligned({top_tokens}, 8))
        return DYT_ERR_MISALIGNED;
    const LpPlan p = lp_plan(T, V, top, dt);
    if (p.bytes && (ws_bytes < p.bytes || !ws)) return DYT_ERR_WORKSPACE_TOO_SMALL;
    if (p.bytes && !aligned({ws}, 16)) return DYT_ERR_MISALIGNED;
    const Range in[] = {{logits, ((T - 1) * ld + V) * s}, {tokens, T * (bits / 8)}};
    const Range out[] = {{logp, T * 4}, {entropy, T * 4}, {lse, T * 4}, {norm, T * 12}, {top_logp, T * top * 4},
                         {top_tokens, T * top * 8}, {ws, (int64_t)p.bytes}};
    if (!disjoint(in, 2, out, 7)) return DYT_ERR_INVALID_ARG;
    LpArgs a{};
    a.logits = logits; a.tokens = tokens; a.logp = logp; a.entropy = entropy; a.lse = lse; a.norm = norm;
    a.top_logp = top_logp; a.top_tokens = top_tokens; a.part = (float*)ws;
    a.part_top = p.bytes ? (uint64_t*)((uint8_t*)ws + p.part_bytes) : nullptr;
    a.ld = ld; a.T = T; a.V = V; a.part_len = p.part_len; a.parts = p.parts; a.top = top; a.token_bits = bits;
    a.tpr = p.tpr; a.scale = scale;
    const float k = scale * kLog2e;   // as the kernels round it
    a.to_ln = (double)scale / (double)k;
    // Logits past the last-level cache (256 MB) leave it to what was written before
    // them: nontemporal loads (8,192 x 50,257 bfloat16: 182 -> 140 us; 8,192 x 4,096,
    // which fit, 17.8 -> 18.4). The backward, whose reads and writes both pass through
    // it, is slower with such loads or stores (289 -> 305).
    a.stream = T * V * s >= kPastCache;
    with_type(dt, [&](auto* t) {
        in_launches(a, p, s, [&](const LpArgs& b, int64_t grid) {
            lp_launch_forward<std::remove_pointer_t<decltype(t)>>(b, grid, p.shared, p.join_shared, (hipStream_t)stream);
        });
    });
    return hip_status();
}

// The sums of the rows: entropy and lse, or norm in their place.
int lp_backward(const void* logits, int64_t ld, const void* tokens, const float* entropy, const float* lse,
                const float* norm, const float* dlogp, const float* dentropy, void* dlogits, int64_t ldd, int64_t T, int64_t V, float scale,
                int dt, int bits, void* stream) {
    if (int e = lp_shape(T, V, 0, dt)) return e;
    if (ld == 0) ld = V;
    if (ldd == 0) ldd = V;
    if ((bits != 32 && bits != 64) || !(scale > 0.0f) || std::isinf(scale) || !pitch_ok(T, V, ld) || !pitch_ok(T, V, ldd))
        return DYT_ERR_INVALID_ARG;
    if (T == 0) return DYT_OK;
    if (V == 0 || !logits || !tokens || (!norm && (!entropy || !lse)) || !dlogits) return DYT_ERR_INVALID_ARG;
    const int64_t s = dtype_size(dt);
    if (!aligned({logits, dlogits}, s) || !aligned({tokens}, bits / 8) || !aligned({entropy, lse, norm, dlogp, dentropy}, 4))
        return DYT_ERR_MISALIGNED;
    const LpPlan p = lp_plan(T, V, 0, dt, true);
    const bool same = dlogits == logits && ldd == ld;   // in place
    const Range in[] = {{same ? nullptr : logits, ((T - 1) * ld + V) * s}, {tokens, T * (bits / 8)}, {entropy, T * 4},
                        {lse, T * 4}, {norm, T * 12}, {dlogp, T * 4}, {dentropy, T * 4}};
    const Range out[] = {{dlogits, ((T - 1) * ldd + V) * s}};
    if (!disjoint(in, 7, out, 1)) return DYT_ERR_INVALID_ARG;
    LpArgs a{};
    a.logits = logits; a.tokens = tokens; a.entropy = const_cast<float*>(entropy); a.lse = const_cast<float*>(lse); a.norm = const_cast<float*>(norm);
    a.dlogp = dlogp; a.dentropy = dentropy; a.dlogits = dlogits; a.ld = ld; a.ldd = ldd; a.T = T; a.V = V;
    a.part_len = p.part_len; a.parts = p.parts; a.token_bits = bits; a.tpr = p.tpr;
    a.scale = scale;
    a.stream = T * V * s >= kPastCache;
    with_type(dt, [&](auto* t) {
        in_launches(a, p, s, [&](const LpArgs& b, int64_t grid) {
            lp_launch_backward<std::remove_pointer_t<decltype(t)>>(b, grid, (hipStream_t)stream);
        });
    });
    return hip_status();
}

}  // namespace
}  // namespace dytb

using namespace dytb;

extern "C" {

size_t dyt_logprob_forward_workspace_size(int64_t T, int64_t V, int top, int dtype) {
    if (lp_shape(T, V, top, dtype) || T == 0 || V == 0) return 0;
    return lp_plan(T, V, top, dtype).bytes;
}

int dyt_logprob_forward(const void* logits, int64_t ld, const void* tokens, float* logp, float* entropy, float* lse,
                        float* top_logp, int64_t* top_tokens, void* workspace, size_t workspace_bytes, int64_t T,
                        int64_t V, float scale, int top, int dtype, int token_bits, void* stream) {
    return lp_forward(logits, ld, tokens, logp, entropy, lse, nullptr, top_logp, top_tokens, workspace,
                      workspace_bytes, T, V, scale, top, dtype, token_bits, stream);
}

int dyt_logprob_forward_norm(const void* logits, int64_t ld, const void* tokens, float* logp, float* entropy, float* lse,
                             float* norm, float* top_logp, int64_t* top_tokens, void* workspace,
                             size_t workspace_bytes, int64_t T, int64_t V, float scale, int top, int dtype,
                             int token_bits, void* stream) {
    if (T > 0 && !norm) return DYT_ERR_INVALID_ARG;
    return lp_forward(logits, ld, tokens, logp, entropy, lse, norm, top_logp, top_tokens, workspace, workspace_bytes,
                      T, V, scale, top, dtype, token_bits, stream);
}

int dyt_logprob_backward(const void* logits, int64_t ld, const void* tokens, const float* entropy, const float* lse,
                         const float* dlogp, const float* dentropy, void* dlogits, int64_t ldd, int64_t T, int64_t V,
                         float scale, int dtype, int token_bits, void* stream) {
    return lp_backward(logits, ld, tokens, entropy, lse, nullptr, dlogp, dentropy, dlogits, ldd, T, V, scale, dtype,
                       token_bits, stream);
}

int dyt_logprob_backward_norm(const void* logits, int64_t ld, const void* tokens, const float* norm,
                              const float* dlogp, const float* dentropy, void* dlogits, int64_t ldd, int64_t T, int64_t V,
                              float scale, int dtype, int token_bits, void* stream) {
    if (T > 0 && !norm) return DYT_ERR_INVALID_ARG;
    return lp_backward(logits, ld, tokens, nullptr, nullptr, norm, dlogp, dentropy, dlogits, ldd, T, V, scale, dtype,
                       token_bits, stream);
}

}  // extern "C"
