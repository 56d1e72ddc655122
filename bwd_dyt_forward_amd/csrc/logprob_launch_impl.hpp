// logprob_launch_impl.hpp - instances of the log probabilities' kernels for
// one type.
#pragma once

#include "logprob_launch.hpp"

namespace dytb {

// Two vectors of a thread at a time with two more on their way leave the
// registers to eight waves per SIMD (four and four to half of them: 175 us for
// 162 at 8,192 x 50,257 bfloat16).
template <typename T, bool TOP, bool ROW>
void lp_fwd_pick(const LpArgs& a, int64_t grid, size_t shared, hipStream_t s) {
    if (a.stream) lp_fwd_kernel<T, TOP, ROW, true><<<(unsigned)grid, kLpThreads, shared, s>>>(a);
    else lp_fwd_kernel<T, TOP, ROW, false><<<(unsigned)grid, kLpThreads, shared, s>>>(a);
}

template <typename T>
void lp_launch_forward(const LpArgs& a, int64_t grid, size_t shared, size_t join_shared, hipStream_t s) {
    if (a.top) lp_fwd_pick<T, true, true>(a, grid, shared, s);
    else if (a.tpr == kLpThreads) lp_fwd_pick<T, false, true>(a, grid, 0, s);
    else lp_fwd_pick<T, false, false>(a, grid, 0, s);
    if (a.parts == 1) return;
    if (a.top) lp_join_kernel<T, true><<<(unsigned)a.T, kLpThreads, join_shared, s>>>(a);
    else lp_join_kernel<T, false><<<(unsigned)a.T, kLpThreads, 0, s>>>(a);
}

// Past the last-level cache the backward asks for LDS that it does not use, so that
// four workgroups and no more share a CU: fewer rows of memory are open at a time
// (8,192 x 50,257 bfloat16 299 us for 321 of eight, 317 of three; 50,304 291, 320 and
// 300; 32,000 198, 208 and 200; 4,096 x 50,257 float32 316, 337 and 311).
constexpr size_t kLpBwdApart = 40000;

template <typename T>
void lp_launch_backward(const LpArgs& a, int64_t grid, hipStream_t s) {
    const size_t apart = a.stream ? kLpBwdApart : 0;
    if (a.norm) lp_bwd_kernel<T, true><<<(unsigned)grid, kLpThreads, apart, s>>>(a);
    else lp_bwd_kernel<T, false><<<(unsigned)grid, kLpThreads, apart, s>>>(a);
}

}  // namespace dytb
