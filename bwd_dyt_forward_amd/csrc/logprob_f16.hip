// logprob_f16.hip - the log probabilities' kernel instances for f16 logits.
#include "logprob_launch_impl.hpp"

namespace dytb {
template void lp_launch_forward<f16_t>(const LpArgs&, int64_t, size_t, size_t, hipStream_t);
template void lp_launch_backward<f16_t>(const LpArgs&, int64_t, hipStream_t);
}  // namespace dytb
