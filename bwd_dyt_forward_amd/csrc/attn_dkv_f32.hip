// attn_dkv_f32.hip - the attention backward's dk and dv kernel instances for f32.
#include "attn_launch_dkv.hpp"

namespace dytb {
template int attn_launch_dkv<float>(const AttnPick&, const AttnArgs&, hipStream_t);
template void attn_launch_sum<float>(int, const SumArgs&, hipStream_t);
}  // namespace dytb
