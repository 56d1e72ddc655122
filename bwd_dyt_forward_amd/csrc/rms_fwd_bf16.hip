// rms_fwd_bf16.hip - the root-mean-square norm's forward instances for bf16 activations.
#include "rms_launch_impl.hpp"

namespace dytb {
template void rms_launch_forward<bf16_t>(const LnConfig&, const RmsArgs&, hipStream_t);
}  // namespace dytb
