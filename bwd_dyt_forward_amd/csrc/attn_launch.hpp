// attn_launch.hpp - the attention's launches per type (attn_*_<type>.hip),
// called by attn_api.hip, and the picking of instances.
#pragma once

#include "attn_tile.hpp"

namespace dytb {

// The rounded-up head dimension and waves per workgroup of an instance.
struct AttnPick {
    int dp, nw;
    bool bias, vec;
};

inline int attn_dp(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : D <= 96 ? 96 : 128; }

// Rows to a tile of the dk/dv kernel's workgroups of four waves (DkvTile).
inline int attn_dkv_tile(int dtype, int dp) { return dtype == DYT_F32 || dp > 64 ? 32 : 64; }

inline unsigned attn_grid(const AttnArgs& a) { return (unsigned)((int64_t)a.units * a.blocks * a.nsplit); }

template <typename T> int attn_launch_fwd(const AttnPick&, const AttnArgs&, hipStream_t);
template <typename T> int attn_launch_dq(const AttnPick&, const AttnArgs&, hipStream_t);
template <typename T> int attn_launch_dkv(const AttnPick&, const AttnArgs&, hipStream_t);

template <typename T> void attn_launch_sum(int dp, const SumArgs&, hipStream_t);

// Calls f with the compile-time (DP, NW, BIAS, VEC) of the pick. Tensors that
// do not take 16-byte loads go element by element, in single waves.
template <int DP, int NW, int VEC, typename F>
void with_bias(const AttnPick& p, F&& f) {
    if (p.bias) f(Int<DP>{}, Int<NW>{}, Int<1>{}, Int<VEC>{});
    else f(Int<DP>{}, Int<NW>{}, Int<0>{}, Int<VEC>{});
}

template <int DP, typename F>
void with_waves(const AttnPick& p, F&& f) {
    if (!p.vec) with_bias<DP, 1, 0>(p, f);
    else if (p.nw == 4) with_bias<DP, 4, 1>(p, f);
    else with_bias<DP, 1, 1>(p, f);
}

template <typename F>
void with_pick(const AttnPick& p, F&& f) {
    switch (p.dp) {
        case 32: return with_waves<32>(p, f);
        case 64: return with_waves<64>(p, f);
        case 96: return with_waves<96>(p, f);
        default: return with_waves<128>(p, f);
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

inline size_t bias_lds_bytes(const AttnArgs& a) { return (size_t)2 * (a.borders.reach + kPad) * sizeof(float); }

}  // namespace dytb
