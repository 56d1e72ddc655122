// logprob_bf16.hip - the log probabilities' kernel instances for bf16 logits.
#include "logprob_launch_impl.hpp"

namespace dytb {
template void lp_launch_forward<bf16_t>(const LpArgs&, int64_t, size_t, size_t, hipStream_t);
template void lp_launch_backward<bf16_t>(const LpArgs&, int64_t, hipStream_t);
}  // namespace dytb
