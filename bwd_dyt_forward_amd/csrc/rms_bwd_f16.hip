// rms_bwd_f16.hip - the root-mean-square norm's backward instances for f16 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_backward_few<f16_t>(const RmsArgs&, hipStream_t);
template int rms_launch_backward<f16_t>(const LnConfig&, int, const RmsArgs&, hipStream_t);
}  // namespace dytb
