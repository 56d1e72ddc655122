// ln_launch_bf16.hip - the layer norm kernel instances for bf16 activations.
#include "ln_launch_impl.hpp"

namespace dytb {
template void ln_launch_forward<bf16_t>(const LnConfig&, const LnArgs&, hipStream_t);
template void ln_launch_backward<bf16_t>(const LnConfig&, int, const LnArgs&, hipStream_t);
}  // namespace dytb
