// rms_launch.hpp - the root-mean-square norm's launches per activation type
// (rms_fwd_, rms_q8_ and rms_bwd_<type>.hip), called by lm_api.hip.
#pragma once

#include "ln_launch.hpp"
#include "rms_kernels.hpp"

namespace dytb {

// The layer norm's shapes, and wider rows: without a mean and its second sum
// 1,024 threads hold 8 vectors each in the forward and 4 in the backward.
inline LnConfig rms_config(int64_t M, int64_t N, int elem_bytes, bool backward) {
    LnConfig c = ln_config(M, N, elem_bytes, backward);
    const int vec = 16 / elem_bytes;
    const int64_t nv = (N + vec - 1) / vec;
    if (c.threads == 0 && M * N >= vec) {
        if (nv <= 4096) return {1024, 4, 1024};
        if (!backward && nv <= 8192) return {1024, 8, 1024};
    }
    return c;
}

template <typename T> void rms_launch_forward(const LnConfig&, const RmsArgs&, hipStream_t);
template <typename T> void rms_launch_forward_q8(const LnConfig&, const RmsArgs&, hipStream_t);
template <typename T> void rms_launch_backward(const LnConfig&, int grid, const RmsArgs&, hipStream_t);

}  // namespace dytb
