// attn_dkv_bf16.hip - the attention backward's dk and dv kernel instances for bf16.
#include "attn_launch_dkv.hpp"

namespace dytb {
template int attn_launch_dkv<bf16_t>(const AttnPick&, const AttnArgs&, hipStream_t);
template void attn_launch_sum<bf16_t>(int, const SumArgs&, hipStream_t);
}  // namespace dytb
