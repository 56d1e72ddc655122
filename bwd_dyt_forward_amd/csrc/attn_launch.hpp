// attn_launch.hpp - the attention's launches per type (attn_*_<type>.hip),
// called by attn_api.hip, and the picking of instances.
#pragma once

#include "attn_tile.hpp"

namespace dytb {

// The rounded-up head dimension and waves per workgroup of an instance.
struct AttnPick {
    int dp, nw;
    bool bias;
};

inline int attn_dp(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : D <= 96 ? 96 : 128; }

inline unsigned attn_grid(const AttnArgs& a) {
    const int64_t total = (int64_t)a.units * a.blocks * a.nsplit;
    return (unsigned)((total + 7) / 8 * 8);
}

template <typename T> int attn_launch_fwd(const AttnPick&, const AttnArgs&, hipStream_t);
template <typename T> int attn_launch_dq(const AttnPick&, const AttnArgs&, hipStream_t);
template <typename T> int attn_launch_dkv(const AttnPick&, const AttnArgs&, hipStream_t);

template <typename T> void attn_launch_sum(int dp, const SumArgs&, hipStream_t);

// Calls f with the compile-time (DP, NW, BIAS) of the pick.
template <int V> struct Int { static constexpr int value = V; };

template <int DP, typename F>
void with_nw_bias(const AttnPick& p, F&& f) {
    if (p.nw == 4) {
        if (p.bias) f(Int<DP>{}, Int<4>{}, Int<1>{});
        else f(Int<DP>{}, Int<4>{}, Int<0>{});
    } else {
        if (p.bias) f(Int<DP>{}, Int<1>{}, Int<1>{});
        else f(Int<DP>{}, Int<1>{}, Int<0>{});
    }
}

template <typename F>
void with_pick(const AttnPick& p, F&& f) {
    switch (p.dp) {
        case 32: return with_nw_bias<32>(p, f);
        case 64: return with_nw_bias<64>(p, f);
        case 96: return with_nw_bias<96>(p, f);
        default: return with_nw_bias<128>(p, f);
    }
}

template <typename F>
void with_dp(int dp, F&& f) {
    switch (dp) {
        case 32: return f(Int<32>{});
        case 64: return f(Int<64>{});
        case 96: return f(Int<96>{});
        default: return f(Int<128>{});
    }
}

// Launches with dynamic LDS; more than the default 64 KB is asked for.
inline int launch_lds(const void* kernel, unsigned grid, unsigned threads, size_t lds, AttnArgs a, hipStream_t s) {
    if (lds > 64 * 1024 &&
        hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return DYT_ERR_HIP;
    void* args[] = {&a};
    return hipLaunchKernel(kernel, dim3(grid), dim3(threads), args, lds, s) == hipSuccess ? DYT_OK : DYT_ERR_HIP;
}

inline size_t bias_lds_bytes(const AttnArgs& a) { return kColBytes + (size_t)2 * (a.borders.reach + kPad) * sizeof(float); }

}  // namespace dytb
