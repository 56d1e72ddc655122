// attn_dq_bf16.hip - the attention backward's dq kernel instances for bf16.
#include "attn_launch_dq.hpp"

namespace dytb {
template int attn_launch_dq<bf16_t>(const AttnPick&, const AttnArgs&, hipStream_t);
}  // namespace dytb
