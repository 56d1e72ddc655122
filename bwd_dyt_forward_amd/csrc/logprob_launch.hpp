// logprob_launch.hpp - the launches of the token log probabilities per type
// (logprob_<type>.hip), called by logprob_api.hip.
#pragma once

#include "logprob_kernels.hpp"

namespace dytb {

// `grid` workgroups, `shared` bytes of LDS for the alternatives; `join`: the
// same of the kernel that joins a row's parts.
template <typename T> void lp_launch_forward(const LpArgs&, int64_t grid, size_t shared, size_t join_shared, hipStream_t);
template <typename T> void lp_launch_backward(const LpArgs&, int64_t grid, hipStream_t);

}  // namespace dytb
