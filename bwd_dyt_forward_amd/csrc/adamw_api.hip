// adamw_api.hip - C ABI of the AdamW step (include/dyt_lm.h): argument checks
// and the cut of a list of tensors into launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "adamw_launch.hpp"
#include "dyt_lm.h"

namespace dytb {
namespace {

constexpr int64_t kMaxN = (int64_t)1 << 34;
constexpr int64_t kMaxGrid = (int64_t)1 << 22;

struct Span {
    uintptr_t lo, hi;
    bool written;
};

// Whether nothing that is written shares memory with anything else.
bool apart(std::vector<Span>& spans) {
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;   // where what came before ends
    for (const Span& s : spans) {
        if (s.lo < written || (s.written && s.lo < any)) return false;
        any = std::max(any, s.hi);
        if (s.written) written = std::max(written, s.hi);
    }
    return true;
}

void add(std::vector<Span>& spans, const void* p, int64_t bytes, bool written) {
    if (p && bytes > 0) spans.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written});
}

// Launches in batches of kAdamTensors tensors that `pick` takes; returns
// whether there were any.
template <typename Pick, typename Launch>
bool in_batches(AdamArgs& a, int64_t count, int64_t chunk, Pick&& pick, Launch&& launch) {
    uint32_t grid = 0;
    bool any = false;
    a.count = 0;
    const auto flush = [&] {
        if (a.count) {
            launch(grid);
            any = true;
        }
        a.count = 0;
        grid = 0;
    };
    for (int64_t i = 0; i < count; ++i) {
        AdamTensor t{};
        if (!pick(i, t) || t.n == 0) continue;
        const int64_t need = (t.n + chunk - 1) / chunk;
        if (a.count == kAdamTensors || grid + need > kMaxGrid) flush();
        t.first = grid;
        a.t[a.count++] = t;
        grid += (uint32_t)need;
    }
    flush();
    return any;
}

// What a step refuses; `bytes`: of all its tensors.
int adamw_check(const dyt_adamw_tensor* list, int64_t count, const dyt_adamw_options* o, int64_t& bytes) {
    if (count < 0 || count > 0x7fffffff || !o || (count > 0 && !list)) return DYT_ERR_INVALID_ARG;
    for (double v : {o->lr, o->beta1, o->beta2, o->eps, o->weight_decay})
        if (!(v >= 0.0) || std::isinf(v)) return DYT_ERR_INVALID_ARG;
    if (o->beta1 >= 1.0 || o->beta2 >= 1.0 || (!o->step_dev && o->step < 1) || (o->seeded != 0 && o->seeded != 1) ||
        (o->state_bits != 8 && o->state_bits != 32) || o->reserved != 0)
        return DYT_ERR_INVALID_ARG;
    if (!aligned({o->lr_dev, o->grad_scale}, 4) || !aligned({o->step_dev}, 8)) return DYT_ERR_MISALIGNED;
    const bool bits8 = o->state_bits == 8;
    std::vector<Span> spans;
    spans.reserve((size_t)count * 7 + 3);
    add(spans, o->lr_dev, 4, false);
    add(spans, o->step_dev, 8, false);
    add(spans, o->grad_scale, 4, false);
    for (int64_t i = 0; i < count; ++i) {
        const dyt_adamw_tensor& t = list[i];
        if (t.n < 0 || t.n > kMaxN) return DYT_ERR_INVALID_ARG;
        if (!dtype_ok(t.param_dtype) || (t.grad_dtype != t.param_dtype && t.grad_dtype != DYT_F32))
            return DYT_ERR_UNSUPPORTED_DTYPE;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || bits8 != (t.avg_scale != nullptr) ||
            bits8 != (t.sq_scale != nullptr) || (t.master && t.param_dtype == DYT_F32))
            return DYT_ERR_INVALID_ARG;
        const int64_t sp = dtype_size(t.param_dtype), ss = bits8 ? 1 : 4, blocks = (t.n + kAdamBlock - 1) / kAdamBlock;
        if (!aligned({t.param}, sp) || !aligned({t.grad}, dtype_size(t.grad_dtype)) ||
            !aligned({t.exp_avg, t.exp_avg_sq}, ss) || !aligned({t.avg_scale, t.sq_scale, t.master}, 4))
            return DYT_ERR_MISALIGNED;
        add(spans, t.param, t.n * sp, true);
        add(spans, t.grad, t.n * dtype_size(t.grad_dtype), false);
        add(spans, t.exp_avg, t.n * ss, true);
        add(spans, t.exp_avg_sq, t.n * ss, true);
        add(spans, t.avg_scale, blocks * 4, true);
        add(spans, t.sq_scale, blocks * 4, true);
        add(spans, t.master, t.n * 4, true);
    }
    bytes = 0;
    for (const Span& t : spans) bytes += (int64_t)(t.hi - t.lo);
    return apart(spans) ? DYT_OK : DYT_ERR_INVALID_ARG;
}

int adamw_step(const dyt_adamw_tensor* list, int64_t count, const dyt_adamw_options* o, void* stream) {
    int64_t bytes = 0;
    if (int e = adamw_check(list, count, o, bytes)) return e;
    const bool bits8 = o->state_bits == 8;
    AdamArgs a{};
    const bool stream_past = bytes >= ((int64_t)256 << 20);   // the last-level cache
    a.seeded = o->seeded; a.seed = o->seed;
    a.beta1 = (float)o->beta1; a.one_beta1 = (float)(1.0 - o->beta1);
    a.beta2 = (float)o->beta2; a.one_beta2 = (float)(1.0 - o->beta2);
    a.eps = (float)o->eps; a.lr = o->lr; a.weight_decay = o->weight_decay;
    a.log_beta1 = std::log(o->beta1); a.log_beta2 = std::log(o->beta2);
    a.step = o->step; a.lr_dev = o->lr_dev; a.step_dev = o->step_dev; a.grad_scale = o->grad_scale;
    a.keep = (float)(1.0 - o->lr * o->weight_decay);
    a.rate = (float)(o->lr / -std::expm1((double)o->step * a.log_beta1));
    a.root_corr2 = (float)(1.0 / std::sqrt(-std::expm1((double)o->step * a.log_beta2)));
    // the types of a parameter, its gradient and whether it has a master: a kernel each
    bool any = false;
    for (int pdt : {DYT_F32, DYT_BF16, DYT_F16})
        for (int own = 0; own < (pdt == DYT_F32 ? 1 : 2); ++own)
            for (int master = 0; master < (pdt == DYT_F32 ? 1 : 2); ++master) {
                const int gdt = own ? pdt : DYT_F32;
                any |= in_batches(
                    a, count, bits8 ? kAdamChunk8 : kAdamChunk,
                    [&](int64_t i, AdamTensor& t) {
                        const dyt_adamw_tensor& x = list[i];
                        if (x.param_dtype != pdt || x.grad_dtype != gdt || (x.master != nullptr) != (master != 0)) return false;
                        t = {x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.avg_scale, x.sq_scale, x.master, x.n, (uint32_t)i, 0};
                        return true;
                    },
                    [&](unsigned grid) {
                        if (bits8) adamw_launch8(a, pdt, gdt, master != 0, grid, (hipStream_t)stream);
                        else adamw_launch32(a, pdt, gdt, master != 0, stream_past, grid, (hipStream_t)stream);
                    });
            }
    return any ? hip_status() : DYT_OK;
}

int adamw_values(const dyt_adamw_codes* list, int64_t count, int vdt, void* stream) {
    if (count < 0 || count > 0x7fffffff || (count > 0 && !list)) return DYT_ERR_INVALID_ARG;
    if (!dtype_ok(vdt)) return DYT_ERR_UNSUPPORTED_DTYPE;
    std::vector<Span> spans;
    spans.reserve((size_t)count * 3);
    for (int64_t i = 0; i < count; ++i) {
        const dyt_adamw_codes& t = list[i];
        if (t.n < 0 || t.n > kMaxN || (t.second != 0 && t.second != 1) || t.reserved != 0) return DYT_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (!t.codes || !t.scale || !t.values) return DYT_ERR_INVALID_ARG;
        if (!aligned({t.scale}, 4) || !aligned({t.values}, dtype_size(vdt))) return DYT_ERR_MISALIGNED;
        add(spans, t.codes, t.n, false);
        add(spans, t.scale, (t.n + kAdamBlock - 1) / kAdamBlock * 4, false);
        add(spans, t.values, t.n * dtype_size(vdt), true);
    }
    if (!apart(spans)) return DYT_ERR_INVALID_ARG;
    AdamArgs a{};
    const bool any = in_batches(
        a, count, kAdamChunk8,
        [&](int64_t i, AdamTensor& t) {
            const dyt_adamw_codes& x = list[i];
            t.param = x.values;
            t.avg = const_cast<void*>(x.codes);
            t.avg_scale = const_cast<float*>(x.scale);
            t.n = x.n;
            t.number = (uint32_t)x.second;
            return true;
        },
        [&](unsigned grid) {
            const hipStream_t s = (hipStream_t)stream;
            if (vdt == DYT_F32) adamw_values_kernel<float><<<grid, kAdamThreads, 0, s>>>(a);
            else if (vdt == DYT_BF16) adamw_values_kernel<bf16_t><<<grid, kAdamThreads, 0, s>>>(a);
            else adamw_values_kernel<f16_t><<<grid, kAdamThreads, 0, s>>>(a);
        });
    return any ? hip_status() : DYT_OK;
}

}  // namespace
}  // namespace dytb

using namespace dytb;

extern "C" {

// The lists of spans are the only memory these calls ask the host for.
int dyt_adamw_check(const dyt_adamw_tensor* tensors, int64_t count, const dyt_adamw_options* options) {
    try {
        int64_t bytes = 0;
        return adamw_check(tensors, count, options, bytes);
    } catch (const std::bad_alloc&) {
        return DYT_ERR_INVALID_ARG;
    }
}

int dyt_adamw_step(const dyt_adamw_tensor* tensors, int64_t count, const dyt_adamw_options* options, void* stream) {
    try {
        return adamw_step(tensors, count, options, stream);
    } catch (const std::bad_alloc&) {
        return DYT_ERR_INVALID_ARG;
    }
}

int dyt_adamw_values(const dyt_adamw_codes* list, int64_t count, int values_dtype, void* stream) {
    try {
        return adamw_values(list, count, values_dtype, stream);
    } catch (const std::bad_alloc&) {
        return DYT_ERR_INVALID_ARG;
    }
}

}  // extern "C"
