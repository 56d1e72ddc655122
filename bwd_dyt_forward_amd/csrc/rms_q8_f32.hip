// rms_q8_f32.hip - the root-mean-square norm's 8-bit forward instances for f32 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_forward_q8<float>(const LnConfig&, const RmsArgs&, hipStream_t);
}  // namespace dytb
