// attn_fwd_f16.hip - the attention forward's kernel instances for f16.
#include "attn_launch_fwd.hpp"

namespace dytb {
template int attn_launch_fwd<f16_t>(const AttnPick&, const AttnArgs&, hipStream_t);
}  // namespace dytb
