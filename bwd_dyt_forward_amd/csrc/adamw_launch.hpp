// adamw_launch.hpp - the AdamW step's launches (adamw32.hip, adamw8.hip),
// called by adamw_api.hip.
#pragma once

#include "adamw_kernels.hpp"
#include "block_host.hpp"

namespace dytb {

// One launch of `grid` workgroups over tensors of the same types; stream_past:
// the call's tensors do not fit the last-level cache.
void adamw_launch32(const AdamArgs&, int param_dtype, int grad_dtype, bool master, bool stream_past, unsigned grid, hipStream_t);
void adamw_launch8(const AdamArgs&, int param_dtype, int grad_dtype, bool master, unsigned grid, hipStream_t);

// Calls f with the types of a parameter and its gradient (the parameter's or
// float32).
template <typename F>
void adamw_types(int pdt, int gdt, F&& f) {
    const auto with = [&](auto* p) {
        if (gdt == pdt) f(p, p);
        else f(p, (float*)nullptr);
    };
    if (pdt == DYT_F32) f((float*)nullptr, (float*)nullptr);
    else if (pdt == DYT_BF16) with((bf16_t*)nullptr);
    else with((f16_t*)nullptr);
}

}  // namespace dytb
