// rms_fwd_f16.hip - the root-mean-square norm's forward instances for f16 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_forward<f16_t>(const LnConfig&, const RmsArgs&, hipStream_t);
}  // namespace dytb
