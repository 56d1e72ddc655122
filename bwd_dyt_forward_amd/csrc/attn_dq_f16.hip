// attn_dq_f16.hip - the attention backward's dq kernel instances for f16.
#include "attn_launch_dq.hpp"

namespace dytb {
template int attn_launch_dq<f16_t>(const AttnPick&, const AttnArgs&, hipStream_t);
}  // namespace dytb
