// attn_dkv_f16.hip - the attention backward's dk and dv kernel instances for f16.
#include "attn_launch_dkv.hpp"

namespace dytb {
template int attn_launch_dkv<f16_t>(const AttnPick&, const AttnArgs&, hipStream_t);
template void attn_launch_sum<f16_t>(int, const SumArgs&, hipStream_t);
}  // namespace dytb
