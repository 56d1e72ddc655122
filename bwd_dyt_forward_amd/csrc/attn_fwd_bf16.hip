// attn_fwd_bf16.hip - the attention forward's kernel instances for bf16.
#include "attn_launch_fwd.hpp"

namespace dytb {
template int attn_launch_fwd<bf16_t>(const AttnPick&, const AttnArgs&, hipStream_t);
}  // namespace dytb
