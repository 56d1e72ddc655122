// ln_launch.hpp - the layer norm's launches per activation type
// (ln_launch_<type>.hip), called by block_api.hip.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

// Threads per row and vectors per thread; threads == 0: the long-row kernels
// (also for a tensor of fewer elements than a vector).
struct LnConfig {
    int threads, vecs;
};

inline LnConfig ln_config(int64_t M, int64_t N, int elem_bytes, bool backward) {
    const int vec = 16 / elem_bytes;
    const int64_t nv = (N + vec - 1) / vec;
    if (M * N < vec) return {0, 0};
    if (nv <= 64) {
        int t = 1;
        while (t < nv) t *= 2;
        return {t, 1};
    }
    if (nv <= 128) return {64, 2};
    // the backward holds two sums per column besides the row: half the vectors
    if (nv <= 256) return backward ? LnConfig{128, 2} : LnConfig{64, 4};
    if (nv <= 512) return {256, 2};
    if (nv <= 1024) return backward ? LnConfig{512, 2} : LnConfig{256, 4};
    if (nv <= 2048) return backward ? LnConfig{1024, 2} : LnConfig{512, 4};
    // 16-bit vectors hold twice the columns: they would not fit the registers
    if (nv <= 4096 && elem_bytes == 4) return {1024, 4};
    return {0, 0};
}

inline int ln_groups(const LnConfig& c) { return c.threads && c.threads < 256 ? 256 / c.threads : 1; }

int ln_bwd_grid(const LnConfig& c, int64_t M, int64_t elem_bytes);

template <typename T> void ln_launch_forward(const LnConfig&, const LnArgs&, hipStream_t);
template <typename T> void ln_launch_backward(const LnConfig&, int grid, const LnArgs&, hipStream_t);

}  // namespace dytb
