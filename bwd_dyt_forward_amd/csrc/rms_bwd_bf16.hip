// rms_bwd_bf16.hip - the root-mean-square norm's backward instances for bf16 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_backward_few<bf16_t>(const RmsArgs&, hipStream_t);
template int rms_launch_backward<bf16_t>(const LnConfig&, int, const RmsArgs&, hipStream_t);
}  // namespace dytb
