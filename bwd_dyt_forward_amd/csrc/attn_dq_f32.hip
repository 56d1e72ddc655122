// attn_dq_f32.hip - the attention backward's dq kernel instances for f32.
#include "attn_launch_dq.hpp"

namespace dytb {
template int attn_launch_dq<float>(const AttnPick&, const AttnArgs&, hipStream_t);
}  // namespace dytb
