// logprob_f32.hip - the log probabilities' kernel instances for f32 logits.
#include "logprob_launch_impl.hpp"

namespace dytb {
template void lp_launch_forward<float>(const LpArgs&, int64_t, size_t, size_t, hipStream_t);
template void lp_launch_backward<float>(const LpArgs&, int64_t, hipStream_t);
}  // namespace dytb
