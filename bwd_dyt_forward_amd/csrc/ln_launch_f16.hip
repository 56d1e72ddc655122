// ln_launch_f16.hip - the layer norm kernel instances for f16 activations.
#include "ln_launch_impl.hpp"

namespace dytb {
template void ln_launch_forward<f16_t>(const LnConfig&, const LnArgs&, hipStream_t);
template void ln_launch_backward<f16_t>(const LnConfig&, int, const LnArgs&, hipStream_t);
}  // namespace dytb
