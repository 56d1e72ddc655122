// ln_launch.hpp - the layer norm's launches per activation type
// (ln_launch_<type>.hip), called by block_api.hip.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

// Threads per row, vectors per thread and threads per workgroup; threads == 0:
// the long-row kernels (also for a tensor of fewer elements than a vector).
struct LnConfig {
    int threads, vecs, wg;
};

inline LnConfig ln_row(int64_t M, int64_t N, int elem_bytes, bool backward) {
    const int vec = 16 / elem_bytes;
    const int64_t nv = (N + vec - 1) / vec;
    if (M * N < vec) return {0, 0, 0};
    if (nv <= 64) {
        int t = 1;
        while (t < nv) t *= 2;
        return {t, 1, 0};
    }
    if (nv <= 128) return {64, 2, 0};
    // the backward holds two sums per column besides the row: half the vectors
    if (nv <= 256) return backward ? LnConfig{128, 2, 0} : LnConfig{64, 4, 0};
    if (nv <= 512) return {256, 2, 0};
    if (nv <= 1024) return backward ? LnConfig{512, 2, 0} : LnConfig{256, 4, 0};
    if (nv <= 2048) return backward ? LnConfig{1024, 2, 0} : LnConfig{512, 4, 0};
    // 16-bit vectors hold twice the columns: they would not fit the registers
    if (nv <= 4096 && elem_bytes == 4) return {1024, 4, 0};
    return {0, 0, 0};
}

// Rows of 128 and 256 threads come four waves to a workgroup, and in the
// backward, where every workgroup has a partial row of sums to write and
// more workgroups mean more of them, eight: at 32,768 x 4,096 bfloat16 with
// the residual 200 -> 176 us (6.1 TB/s). Workgroups of sixteen waves, which get 128
// registers a lane and spill, are left to rows that need them. With fewer than four rounds of rows the smaller
// workgroups spread better.
inline LnConfig ln_config(int64_t M, int64_t N, int elem_bytes, bool backward) {
    LnConfig c = ln_row(M, N, elem_bytes, backward);
    c.wg = c.threads ? ln_threads(c.threads) : 0;
    if (backward && (c.threads == 128 || c.threads == 256) && M >= 256 * 4 * (512 / c.threads)) c.wg = 512;
    return c;
}

// Cache hints by the bytes of one activation tensor (the last-level cache
// holds 256 MB). From a quarter of that, what a kernel writes would only push
// out what it reads: nontemporal stores (100,003 x 255 float32, forward and
// backward 103 -> 93 us; 16,384 x 4,096 bfloat16 forward with the residual
// 105 -> 84 us; a kernel that reads y straight afterwards loses 6 us of
// that). Beyond the whole of it what the backward or the residual's four
// tensors bring in does not survive either: nontemporal loads there (32,768 x
// 4,096 bfloat16, backward 209 -> 200 us; in the plain forward, and for
// tensors that do fit, they cost up to a tenth).
inline int ln_traffic(int64_t M, int64_t N, int elem_bytes, bool many) {
    const int64_t bytes = M * N * elem_bytes;
    if (many && bytes >= ((int64_t)256 << 20)) return 2;
    return bytes >= ((int64_t)64 << 20) ? 1 : 0;
}

inline int ln_groups(const LnConfig& c) { return c.threads ? c.wg / c.threads : 1; }

int ln_bwd_grid(const LnConfig& c, int64_t M, int64_t elem_bytes);

template <typename T> void ln_launch_forward(const LnConfig&, const LnArgs&, hipStream_t);
template <typename T> void ln_launch_backward(const LnConfig&, int grid, const LnArgs&, hipStream_t);

}  // namespace dytb
