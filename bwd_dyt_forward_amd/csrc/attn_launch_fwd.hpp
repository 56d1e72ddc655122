// attn_launch_fwd.hpp - launch of the attention forward for one type.
#pragma once

#include "attn_fwd.hpp"
#include "attn_launch.hpp"

namespace dytb {

template <typename T>
int attn_launch_fwd(const AttnPick& p, const AttnArgs& a, hipStream_t s) {
    int st = DYT_OK;
    with_pick<(int)sizeof(T), false>(p, [&](auto dp, auto nw, auto sl, auto bias, auto vec) {
        constexpr int DP = decltype(dp)::value, NW = decltype(nw)::value, SL = decltype(sl)::value;
        constexpr bool BIAS = decltype(bias)::value != 0, VEC = decltype(vec)::value != 0;
        const int lds = attn_lds_bytes((int)sizeof(T), DP, NW, SL) + (BIAS ? bias_lds_bytes(a.borders) : 0);
        st = launch_lds<attn_fwd_kernel<T, DP, NW, SL, BIAS, VEC>>(attn_grid(a), NW * SL * 64, lds, a, s);
    });
    if (st || a.nsplit == 1) return st;
    with_dp(p.dp, [&](auto dp) {
        constexpr int DP = decltype(dp)::value, TPR = DP / 4;
        const int64_t rows = (int64_t)a.units * a.Sq * a.pack;
        if (a.nsplit >= 8) {
            constexpr int JG = 256 / TPR < 8 ? 256 / TPR : 8, PER = 256 / (TPR * JG);
            attn_join_kernel<T, DP, JG><<<(unsigned)((rows + PER - 1) / PER), 256, 0, s>>>(a);
        } else {
            constexpr int PER = 256 / TPR;
            attn_join_kernel<T, DP, 1><<<(unsigned)((rows + PER - 1) / PER), 256, 0, s>>>(a);
        }
    });
    return hipGetLastError() == hipSuccess ? DYT_OK : DYT_ERR_HIP;
}

}  // namespace dytb
