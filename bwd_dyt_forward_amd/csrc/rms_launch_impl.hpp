// rms_launch_impl.hpp - instances of the root-mean-square norm's kernels for
// one type.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "rms_launch.hpp"

namespace dytb {

// Workgroups of a forward launch: enough to fill 256 CUs several times over
// and no more, since each loads gamma once for all its rows; two of 256 threads
// per CU where the tensors do not stay in the caches (32,768 x 4,096 bfloat16: 92
// us for 103; 131,072 x 1,024 with the residual 192 for 200).
constexpr int kRmsGridThreads = 256 * 2048, kRmsGridThreadsFew = 256 * 512;

template <typename T, bool Q8, int TPR, int V, int U>
void rms_fwd_one(const RmsArgs& a, hipStream_t s) {
    using S = LnShape<TPR>;
    const int64_t per = (int64_t)S::groups * U;
    const int64_t need = (a.M + per - 1) / per;
    const auto with = [&](auto nt, int threads) {
        constexpr int NT = decltype(nt)::value;
        const int grid = (int)std::min<int64_t>(need, threads / S::threads);
        if (a.r) rms_fwd_kernel<T, TPR, V, U, true, Q8, NT><<<grid, S::threads, 0, s>>>(a);
        else rms_fwd_kernel<T, TPR, V, U, false, Q8, NT><<<grid, S::threads, 0, s>>>(a);
    };
    if constexpr (Q8) {
        // The codes are half a 16-bit row, left to the caches for what reads them next; the
        // other tensors pass them by (16,384 x 4,096 bfloat16 with the residual 80 us for 95),
        // and the second reduction wants all the workgroups (83).
        if (a.traffic == 2) with(std::integral_constant<int, 2>{}, kRmsGridThreads);
        else with(std::integral_constant<int, 0>{}, kRmsGridThreads);
        return;
    }
    if (a.traffic == 2) with(std::integral_constant<int, 2>{}, kRmsGridThreadsFew);
    else if (a.traffic) with(std::integral_constant<int, 1>{}, kRmsGridThreadsFew);
    else with(std::integral_constant<int, 0>{}, kRmsGridThreads);
}

// U rows per thread at a time keep enough loads in flight where a row is few
// vectors; with few rows (under one round of the grid) one row per thread
// spreads them over more CUs.
template <typename T, bool Q8, int TPR, int V, int U>
void rms_fwd_pick(const RmsArgs& a, hipStream_t s) {
    if constexpr (U > 1) {
        if (a.M > (int64_t)LnShape<TPR>::groups * U * 512) return rms_fwd_one<T, Q8, TPR, V, U>(a, s);
    }
    rms_fwd_one<T, Q8, TPR, V, 1>(a, s);
}

template <typename T, bool Q8>
void rms_fwd_any(const LnConfig& c, const RmsArgs& a, hipStream_t s) {
    switch (c.threads * 16 + c.vecs) {
        case 1 * 16 + 1: return rms_fwd_pick<T, Q8, 1, 1, 4>(a, s);
        case 2 * 16 + 1: return rms_fwd_pick<T, Q8, 2, 1, 4>(a, s);
        case 4 * 16 + 1: return rms_fwd_pick<T, Q8, 4, 1, 4>(a, s);
        case 8 * 16 + 1: return rms_fwd_pick<T, Q8, 8, 1, 4>(a, s);
        case 16 * 16 + 1: return rms_fwd_pick<T, Q8, 16, 1, 4>(a, s);
        case 32 * 16 + 1: return rms_fwd_pick<T, Q8, 32, 1, 4>(a, s);
        case 64 * 16 + 1: return rms_fwd_pick<T, Q8, 64, 1, 4>(a, s);
        case 64 * 16 + 2: return rms_fwd_pick<T, Q8, 64, 2, 2>(a, s);
        case 64 * 16 + 4: return rms_fwd_pick<T, Q8, 64, 4, 1>(a, s);
        case 256 * 16 + 2: return rms_fwd_pick<T, Q8, 256, 2, 1>(a, s);
        case 256 * 16 + 4: return rms_fwd_pick<T, Q8, 256, 4, 1>(a, s);
        case 512 * 16 + 4: return rms_fwd_pick<T, Q8, 512, 4, 1>(a, s);
        case 1024 * 16 + 4: return rms_fwd_pick<T, Q8, 1024, 4, 1>(a, s);
        case 1024 * 16 + 8: return rms_fwd_pick<T, Q8, 1024, 8, 1>(a, s);
        default: break;
    }
    const int grid = (int)std::min<int64_t>(a.M, 512);
    if (a.r) rms_fwd_long_kernel<T, true, Q8><<<grid, kLongThreads, 0, s>>>(a);
    else rms_fwd_long_kernel<T, false, Q8><<<grid, kLongThreads, 0, s>>>(a);
}

template <typename T>
void rms_launch_forward(const LnConfig& c, const RmsArgs& a, hipStream_t s) { rms_fwd_any<T, false>(c, a, s); }

template <typename T>
void rms_launch_forward_q8(const LnConfig& c, const RmsArgs& a, hipStream_t s) { rms_fwd_any<T, true>(c, a, s); }

template <typename T, int TPR, int TH, int V, int U>
void rms_bwd_one(int grid, const RmsArgs& a, hipStream_t s) {
    const auto with = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (a.dres) rms_bwd_kernel<T, TPR, TH, V, U, true, NT><<<grid, TH, 0, s>>>(a);
        else rms_bwd_kernel<T, TPR, TH, V, U, false, NT><<<grid, TH, 0, s>>>(a);
    };
    if (a.traffic == 2) with(std::integral_constant<int, 2>{});
    else if (a.traffic == 1) with(std::integral_constant<int, 1>{});
    else with(std::integral_constant<int, 0>{});
}

// Several waves to a row: four or eight to a workgroup.
template <typename T, int TPR>
void rms_bwd_wide(const LnConfig& c, int grid, const RmsArgs& a, hipStream_t s) {
    if (c.wg == 512) rms_bwd_one<T, TPR, 512, 2, 1>(grid, a, s);
    else rms_bwd_one<T, TPR, 256, 2, 1>(grid, a, s);
}

// U rows per thread at a time where a row is one vector and every workgroup
// has several rounds of them.
template <typename T, int TPR>
void rms_bwd_pick(int grid, const RmsArgs& a, hipStream_t s) {
    if (a.M >= (int64_t)grid * LnShape<TPR>::groups * 4) return rms_bwd_one<T, TPR, 256, 1, 2>(grid, a, s);
    rms_bwd_one<T, TPR, 256, 1, 1>(grid, a, s);
}

template <typename T>
void rms_bwd_any(const LnConfig& c, int grid, const RmsArgs& a, hipStream_t s) {
    switch (c.threads * 16 + c.vecs) {
        case 1 * 16 + 1: return rms_bwd_pick<T, 1>(grid, a, s);
        case 2 * 16 + 1: return rms_bwd_pick<T, 2>(grid, a, s);
        case 4 * 16 + 1: return rms_bwd_pick<T, 4>(grid, a, s);
        case 8 * 16 + 1: return rms_bwd_pick<T, 8>(grid, a, s);
        case 16 * 16 + 1: return rms_bwd_pick<T, 16>(grid, a, s);
        case 32 * 16 + 1: return rms_bwd_pick<T, 32>(grid, a, s);
        case 64 * 16 + 1: return rms_bwd_pick<T, 64>(grid, a, s);
        case 64 * 16 + 2: return rms_bwd_one<T, 64, 256, 2, 1>(grid, a, s);
        case 128 * 16 + 2: return rms_bwd_wide<T, 128>(c, grid, a, s);
        case 256 * 16 + 2: return rms_bwd_wide<T, 256>(c, grid, a, s);
        case 512 * 16 + 2: return rms_bwd_one<T, 512, 512, 2, 1>(grid, a, s);
        case 512 * 16 + 4: return rms_bwd_one<T, 512, 512, 4, 1>(grid, a, s);
        default: break;
    }
    if (a.dres) rms_bwd_long_kernel<T, true><<<grid, kLongThreads, 0, s>>>(a);
    else rms_bwd_long_kernel<T, false><<<grid, kLongThreads, 0, s>>>(a);
}

// The wide rows' kernel, with more than the default 64 KB of dynamic LDS: an
// instance is given it once per device (a microsecond of a small call otherwise).
template <auto Kernel>
int launch_wide(int grid, size_t lds, const RmsArgs& a, hipStream_t s) {
    static std::atomic<uint64_t> raised{0};
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess) return DYT_ERR_HIP;
    const uint64_t bit = (uint64_t)1 << (device & 63);
    if (device > 63 || !(raised.load(std::memory_order_acquire) & bit)) {
        if (hipFuncSetAttribute((const void*)Kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                kWideColumns * sizeof(float)) != hipSuccess)
            return DYT_ERR_HIP;
        if (device <= 63) raised.fetch_or(bit, std::memory_order_release);
    }
    Kernel<<<grid, kLongThreads, lds, s>>>(a);
    return DYT_OK;
}

template <typename T, int V>
int rms_bwd_wide_rows(int grid, const RmsArgs& a, hipStream_t s) {
    constexpr size_t lds = (size_t)V * VecOf<T>::n * kLongThreads * sizeof(float);
    const bool past = a.traffic == 2;
    if (a.dres) return past ? launch_wide<rms_bwd_wide_kernel<T, V, true, 2>>(grid, lds, a, s)
                            : launch_wide<rms_bwd_wide_kernel<T, V, true, 0>>(grid, lds, a, s);
    return past ? launch_wide<rms_bwd_wide_kernel<T, V, false, 2>>(grid, lds, a, s)
                : launch_wide<rms_bwd_wide_kernel<T, V, false, 0>>(grid, lds, a, s);
}

template <typename T>
void rms_launch_backward_few(const RmsArgs& a, hipStream_t s) {
    constexpr int cols = 4 * VecOf<T>::n;
    const auto with = [&](auto tpr) {
        constexpr int TPR = decltype(tpr)::value;
        const int rows = (int)((a.M + 256 / TPR - 1) / (256 / TPR)), grid = rows + (a.N + cols - 1) / cols;
        if (a.dres) rms_bwd_few_kernel<T, TPR, true><<<grid, 256, 0, s>>>(a, rows);
        else rms_bwd_few_kernel<T, TPR, false><<<grid, 256, 0, s>>>(a, rows);
    };
    if (a.N <= 64 * 4 * VecOf<T>::n) with(std::integral_constant<int, 64>{});
    else with(std::integral_constant<int, 256>{});
}

template <typename T>
int rms_launch_backward(const LnConfig& c, int grid, const RmsArgs& a, hipStream_t s) {
    if (c.threads == 1024) {
        if constexpr (sizeof(T) == 4) {
            if (c.vecs == 8) return rms_bwd_wide_rows<T, 8>(grid, a, s);
        }
        return rms_bwd_wide_rows<T, 4>(grid, a, s);
    }
    rms_bwd_any<T>(c, grid, a, s);
    return DYT_OK;
}

}  // namespace dytb
