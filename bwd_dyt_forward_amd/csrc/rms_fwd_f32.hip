// rms_fwd_f32.hip - the root-mean-square norm's forward instances for f32 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_forward<float>(const LnConfig&, const RmsArgs&, hipStream_t);
}  // namespace dytb
