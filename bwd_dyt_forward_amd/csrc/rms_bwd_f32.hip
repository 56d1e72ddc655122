// rms_bwd_f32.hip - the root-mean-square norm's backward instances for f32 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_backward_few<float>(const RmsArgs&, hipStream_t);
template int rms_launch_backward<float>(const LnConfig&, int, const RmsArgs&, hipStream_t);
}  // namespace dytb
