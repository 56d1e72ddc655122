// logprob_launch_impl.hpp - instances of the log probabilities' kernels for
// one type.
#pragma once

#include "logprob_launch.hpp"

namespace dytb {

template <typename T>
void lp_launch_forward(const LpArgs& a, int64_t grid, size_t shared, size_t join_shared, hipStream_t s) {
    if (a.top) lp_fwd_kernel<T, true><<<(unsigned)grid, kLpThreads, shared, s>>>(a);
    else lp_fwd_kernel<T, false><<<(unsigned)grid, kLpThreads, 0, s>>>(a);
    if (a.parts == 1) return;
    if (a.top) lp_join_kernel<T, true><<<(unsigned)a.T, kLpThreads, join_shared, s>>>(a);
    else lp_join_kernel<T, false><<<(unsigned)a.T, kLpThreads, 0, s>>>(a);
}

template <typename T>
void lp_launch_backward(const LpArgs& a, int64_t grid, hipStream_t s) {
    lp_bwd_kernel<T><<<(unsigned)grid, kLpThreads, 0, s>>>(a);
}

}  // namespace dytb
