// attn_fwd_f32.hip - the attention forward's kernel instances for f32.
#include "attn_launch_fwd.hpp"

namespace dytb {
template int attn_launch_fwd<float>(const AttnPick&, const AttnArgs&, hipStream_t);
}  // namespace dytb
