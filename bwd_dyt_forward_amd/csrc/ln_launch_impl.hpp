// ln_launch_impl.hpp - instances of the layer norm kernels for one type.
#pragma once

#include <algorithm>
#include <type_traits>

#include "ln_launch.hpp"

namespace dytb {

// Workgroups of a forward launch: enough to fill 256 CUs several times over
// and no more, since each loads gamma and beta once for all its rows. Where
// loads and stores are nontemporal and a row takes whole workgroups, two of 256
// threads per CU, or one of 512, or half of 1,024 (32,768 x 4,096 bfloat16 with the residual: 203 -> 185 us; at half the
// rows, where the tensors fit the last-level cache, the other way round: 84
// against 92).
constexpr int kFwdGridThreads = 256 * 2048, kFwdGridThreadsFew = 256 * 512;

template <typename T, int TPR, int V, int U>
void ln_fwd_one(const LnArgs& a, hipStream_t s) {
    using S = LnShape<TPR>;
    const int64_t per = (int64_t)S::groups * U;
    const int64_t need = (a.M + per - 1) / per;
    const auto with = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        const int grid = (int)std::min<int64_t>(need, kFwdGridThreads / S::threads);
        if (a.r) ln_fwd_kernel<T, TPR, V, U, true, NT><<<grid, S::threads, 0, s>>>(a);
        else ln_fwd_kernel<T, TPR, V, U, false, NT><<<grid, S::threads, 0, s>>>(a);
    };
    if constexpr (TPR >= 256) {
        if (a.traffic == 2) {
            const int grid = (int)std::min<int64_t>(need, kFwdGridThreadsFew / S::threads);
            ln_fwd_kernel<T, TPR, V, U, true, 2><<<grid, S::threads, 0, s>>>(a);
            return;
        }
    }
    if (a.traffic) with(std::integral_constant<int, 1>{});
    else with(std::integral_constant<int, 0>{});
}

// U rows per thread at a time keep enough loads in flight where a row is few
// vectors; with few rows (under one round of the grid) one row per thread
// spreads them over more CUs.
template <typename T, int TPR, int V, int U>
void ln_fwd_pick(const LnArgs& a, hipStream_t s) {
    if constexpr (U > 1) {
        if (a.M > (int64_t)LnShape<TPR>::groups * U * 512) return ln_fwd_one<T, TPR, V, U>(a, s);
    }
    ln_fwd_one<T, TPR, V, 1>(a, s);
}

template <typename T>
void ln_launch_forward(const LnConfig& c, const LnArgs& a, hipStream_t s) {
    switch (c.threads * 8 + c.vecs) {
        case 1 * 8 + 1: return ln_fwd_pick<T, 1, 1, 4>(a, s);
        case 2 * 8 + 1: return ln_fwd_pick<T, 2, 1, 4>(a, s);
        case 4 * 8 + 1: return ln_fwd_pick<T, 4, 1, 4>(a, s);
        case 8 * 8 + 1: return ln_fwd_pick<T, 8, 1, 4>(a, s);
        case 16 * 8 + 1: return ln_fwd_pick<T, 16, 1, 4>(a, s);
        case 32 * 8 + 1: return ln_fwd_pick<T, 32, 1, 4>(a, s);
        case 64 * 8 + 1: return ln_fwd_pick<T, 64, 1, 4>(a, s);
        case 64 * 8 + 2: return ln_fwd_pick<T, 64, 2, 2>(a, s);
        case 64 * 8 + 4: return ln_fwd_pick<T, 64, 4, 1>(a, s);
        case 256 * 8 + 2: return ln_fwd_pick<T, 256, 2, 1>(a, s);
        case 256 * 8 + 4: return ln_fwd_pick<T, 256, 4, 1>(a, s);
        case 512 * 8 + 4: return ln_fwd_pick<T, 512, 4, 1>(a, s);
        default: break;
    }
    if constexpr (sizeof(T) == 4) {
        if (c.threads == 1024) return ln_fwd_pick<T, 1024, 4, 1>(a, s);
    }
    const int grid = (int)std::min<int64_t>(a.M, 512);
    if (a.r) ln_fwd_long_kernel<T, true><<<grid, kLongThreads, 0, s>>>(a);
    else ln_fwd_long_kernel<T, false><<<grid, kLongThreads, 0, s>>>(a);
}

template <typename T, int TPR, int TH, int V, int U>
void ln_bwd_one(int grid, const LnArgs& a, hipStream_t s) {
    const auto with = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (a.dres) ln_bwd_kernel<T, TPR, TH, V, U, true, NT><<<grid, TH, 0, s>>>(a);
        else ln_bwd_kernel<T, TPR, TH, V, U, false, NT><<<grid, TH, 0, s>>>(a);
    };
    if (a.traffic == 2) with(std::integral_constant<int, 2>{});
    else if (a.traffic == 1) with(std::integral_constant<int, 1>{});
    else with(std::integral_constant<int, 0>{});
}

// Several waves to a row: four or eight to a workgroup.
template <typename T, int TPR>
void ln_bwd_wide(const LnConfig& c, int grid, const LnArgs& a, hipStream_t s) {
    if (c.wg == 512) ln_bwd_one<T, TPR, 512, 2, 1>(grid, a, s);
    else ln_bwd_one<T, TPR, 256, 2, 1>(grid, a, s);
}

// U rows per thread at a time where a row is one vector and every workgroup
// has several rounds of them.
template <typename T, int TPR>
void ln_bwd_pick(int grid, const LnArgs& a, hipStream_t s) {
    if (a.M >= (int64_t)grid * LnShape<TPR>::groups * 4) return ln_bwd_one<T, TPR, 256, 1, 2>(grid, a, s);
    ln_bwd_one<T, TPR, 256, 1, 1>(grid, a, s);
}

template <typename T>
void ln_launch_backward(const LnConfig& c, int grid, const LnArgs& a, hipStream_t s) {
    switch (c.threads * 8 + c.vecs) {
        case 1 * 8 + 1: return ln_bwd_pick<T, 1>(grid, a, s);
        case 2 * 8 + 1: return ln_bwd_pick<T, 2>(grid, a, s);
        case 4 * 8 + 1: return ln_bwd_pick<T, 4>(grid, a, s);
        case 8 * 8 + 1: return ln_bwd_pick<T, 8>(grid, a, s);
        case 16 * 8 + 1: return ln_bwd_pick<T, 16>(grid, a, s);
        case 32 * 8 + 1: return ln_bwd_pick<T, 32>(grid, a, s);
        case 64 * 8 + 1: return ln_bwd_pick<T, 64>(grid, a, s);
        case 64 * 8 + 2: return ln_bwd_one<T, 64, 256, 2, 1>(grid, a, s);
        case 128 * 8 + 2: return ln_bwd_wide<T, 128>(c, grid, a, s);
        case 256 * 8 + 2: return ln_bwd_wide<T, 256>(c, grid, a, s);
        case 512 * 8 + 2: return ln_bwd_one<T, 512, 512, 2, 1>(grid, a, s);
        case 1024 * 8 + 2: return ln_bwd_one<T, 1024, 1024, 2, 1>(grid, a, s);
        default: break;
    }
    if constexpr (sizeof(T) == 4) {
        if (c.threads == 1024) return ln_bwd_one<T, 1024, 1024, 4, 1>(grid, a, s);
    }
    if (a.dres) ln_bwd_long_kernel<T, true><<<grid, kLongThreads, 0, s>>>(a);
    else ln_bwd_long_kernel<T, false><<<grid, kLongThreads, 0, s>>>(a);
}

}  // namespace dytb
