// attn_launch_dq.hpp - launch of the attention backward's dq kernel.
#pragma once

#include "attn_bwd.hpp"
#include "attn_launch.hpp"

namespace dytb {

template <typename T>
int attn_launch_dq(const AttnPick& p, const AttnArgs& a, hipStream_t s) {
    int st = DYT_OK;
    with_pick<(int)sizeof(T), false>(p, [&](auto dp, auto nw, auto sl, auto bias, auto vec) {
        constexpr int DP = decltype(dp)::value, NW = decltype(nw)::value, SL = decltype(sl)::value;
        constexpr bool BIAS = decltype(bias)::value != 0, VEC = decltype(vec)::value != 0;
        const int lds = attn_lds_bytes((int)sizeof(T), DP, NW, SL) + (BIAS ? bias_lds_bytes(a.borders) : 0);
        st = launch_lds<attn_dq_kernel<T, DP, NW, SL, BIAS, VEC>>(attn_grid(a), NW * SL * 64, lds, a, s);
    });
    return st;
}

}  // namespace dytb
