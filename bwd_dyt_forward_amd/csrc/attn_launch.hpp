// attn_launch.hpp - the attention's launches per type (attn_*_<type>.hip),
// called by attn_api.hip, and the picking of instances.
#pragma once

#include <atomic>

#include "attn_tile.hpp"

namespace dytb {

// The rounded-up head dimension, row groups and slices of an instance.
struct AttnPick {
    int dp, nw, sl;
    bool bias, vec;
};

inline int attn_dp(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : D <= 96 ? 96 : 128; }

inline unsigned attn_grid(const AttnArgs& a) { return (unsigned)((int64_t)a.units * a.blocks * a.nsplit); }

template <typename T> int attn_launch_fwd(const AttnPick&, const AttnArgs&, hipStream_t);
template <typename T> int attn_launch_dq(const AttnPick&, const AttnArgs&, hipStream_t);
template <typename T> int attn_launch_dkv(const AttnPick&, const AttnArgs&, hipStream_t);

template <typename T> void attn_launch_sum(int dp, const SumArgs&, hipStream_t);

// Calls f with the compile-time (DP, NW, SL, BIAS, VEC) of the pick. Tensors
// that do not take 16-byte loads go element by element, in single waves.
// PAIRS: the workgroups of four row groups come with two slices above dp = 64.
template <int DP, int NW, int SL, int VEC, typename F>
void with_bias(const AttnPick& p, F&& f) {
    if (p.bias) f(Int<DP>{}, Int<NW>{}, Int<SL>{}, Int<1>{}, Int<VEC>{});
    else f(Int<DP>{}, Int<NW>{}, Int<SL>{}, Int<0>{}, Int<VEC>{});
}

template <int ES, bool PAIRS, int DP, typename F>
void with_waves(const AttnPick& p, F&& f) {
    if (!p.vec) return with_bias<DP, 1, 1, 0>(p, f);
    if (p.nw == 4) {
        if constexpr (PAIRS && dkv_vals_in_lds(ES, DP)) {
            // (one slice only where a wide table's sums leave no LDS for two)
            static_assert(attn_dkv_lds_bytes(ES, DP, 4, 2) <= kMaxLds);
            if (p.sl == 2) return with_bias<DP, 4, 2, 1>(p, f);
            return f(Int<DP>{}, Int<4>{}, Int<1>{}, Int<1>{}, Int<1>{});
        } else {
            return with_bias<DP, 4, 1, 1>(p, f);
        }
    }
    if constexpr (attn_lds_bytes(ES, DP, 1, 4) <= kMaxLds) {
        if (p.sl == 4) return with_bias<DP, 1, 4, 1>(p, f);
    }
    if (p.sl == 2) return with_bias<DP, 1, 2, 1>(p, f);
    with_bias<DP, 1, 1, 1>(p, f);
}

template <int ES, bool PAIRS, typename F>
void with_pick(const AttnPick& p, F&& f) {
    switch (p.dp) {
        case 32: return with_waves<ES, PAIRS, 32>(p, f);
        case 64: return with_waves<ES, PAIRS, 64>(p, f);
        case 96: return with_waves<ES, PAIRS, 96>(p, f);
        default: return with_waves<ES, PAIRS, 128>(p, f);
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

// Launches with dynamic LDS. An instance that may need more than the default 64
// KB is given all of it, once per device (a microsecond of a small call
// otherwise).
template <auto Kernel>
int launch_lds(unsigned grid, unsigned threads, size_t lds, const AttnArgs& a, hipStream_t s) {
    if (lds > 64 * 1024) {
        static std::atomic<uint64_t> raised{0};
        int device = 0;
        if (hipGetDevice(&device) != hipSuccess) return DYT_ERR_HIP;
        const uint64_t bit = (uint64_t)1 << (device & 63);
        if (device > 63 || !(raised.load(std::memory_order_acquire) & bit)) {
            if (hipFuncSetAttribute((const void*)Kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds) != hipSuccess)
                return DYT_ERR_HIP;
            if (device <= 63) raised.fetch_or(bit, std::memory_order_release);
        }
    }
    Kernel<<<grid, threads, lds, s>>>(a);
    return hipGetLastError() == hipSuccess ? DYT_OK : DYT_ERR_HIP;
}

// LDS of the bias by relative position, and of its gradient's sums.
inline int bias_lds_bytes(const Borders& o) { return 2 * (o.reach + kPad) * (int)sizeof(float); }
inline int dbias_lds_bytes(const Borders& o, int waves) {
    return dbias_floats(2 * (o.reach + kPad), waves) * (int)sizeof(float);
}

}  // namespace dytb
