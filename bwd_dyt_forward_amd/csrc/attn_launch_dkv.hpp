// attn_launch_dkv.hpp - launches of the attention backward's dk and dv kernel
// and of the sums of float32 parts.
#pragma once

#include <algorithm>

#include "attn_bwd.hpp"
#include "attn_launch.hpp"

namespace dytb {

template <typename T>
int attn_launch_dkv(const AttnPick& p, const AttnArgs& a, hipStream_t s) {
    int st = DYT_OK;
    with_pick<(int)sizeof(T), true>(p, [&](auto dp, auto nw, auto sl, auto bias, auto vec) {
        constexpr int DP = decltype(dp)::value, NW = decltype(nw)::value, SL = decltype(sl)::value;
        constexpr bool BIAS = decltype(bias)::value != 0, VEC = decltype(vec)::value != 0;
        int lds = attn_dkv_lds_bytes((int)sizeof(T), DP, NW, SL);
        if (BIAS) lds += bias_lds_bytes(a.borders) + dbias_lds_bytes(a.borders, NW * SL);
        st = launch_lds<attn_dkv_kernel<T, DP, NW, SL, BIAS, VEC>>(attn_grid(a), NW * SL * 64, lds, a, s);
    });
    return st;
}

// From here on a sum's workgroups walk: far above what fills the card, and
// below the 2^32 threads of a launch.
constexpr int64_t kSumGrid = 1 << 22;

template <typename T>
void attn_launch_sum(int dp, const SumArgs& x, hipStream_t s) {
    with_dp(dp, [&](auto d) {
        constexpr int DP = decltype(d)::value, PER = 256 / (DP / 4);
        const int64_t groups = (x.total + PER - 1) / PER * (x.out2 ? 2 : 1);
        attn_sum_kernel<T, DP><<<(unsigned)std::min(groups, kSumGrid), 256, 0, s>>>(x);
    });
}

}  // namespace dytb
