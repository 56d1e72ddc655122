// ln_launch_f32.hip - the layer norm kernel instances for f32 activations.
#include "ln_launch_impl.hpp"

namespace dytb {
template void ln_launch_forward<float>(const LnConfig&, const LnArgs&, hipStream_t);
template void ln_launch_backward<float>(const LnConfig&, int, const LnArgs&, hipStream_t);
}  // namespace dytb
