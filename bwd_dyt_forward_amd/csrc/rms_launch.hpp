// rms_launch.hpp - the root-mean-square norm's launches per activation type
// (rms_fwd_, rms_q8_ and rms_bwd_<type>.hip), called by lm_api.hip.
#pragma once

#include "ln_launch.hpp"
#include "rms_kernels.hpp"

namespace dytb {

// The layer norm's shapes, and wider rows. Without a mean and its second sum
// 1,024 threads hold 8 vectors each in the forward, and 512 threads, which may
// have twice the registers of 1,024, hold 4 in the backward (8,192 x 16,384
// bfloat16 172 us, with the residual 196; of 1,024 threads that spill 289 and 422).
// Beyond, the backward keeps the columns' sums in LDS up to kWideColumns.
inline LnConfig rms_config(int64_t M, int64_t N, int elem_bytes, bool backward) {
    const LnConfig c = ln_config(M, N, elem_bytes, backward);
    const int vec = 16 / elem_bytes;
    const int64_t nv = (N + vec - 1) / vec;
    if (M * N < vec || nv <= 1024 || (!backward && nv <= 2048)) return c;
    if (!backward) return nv <= 4096 ? LnConfig{1024, 4, 1024} : nv <= 8192 ? LnConfig{1024, 8, 1024} : LnConfig{0, 0, 0};
    if (nv <= 2048) return {512, 4, 512};
    if (nv <= 4096) return {1024, 4, 1024};
    return N <= kWideColumns ? LnConfig{1024, 8, 1024} : LnConfig{0, 0, 0};
}

// Cache hints of the forward: nontemporal stores from 64 MB tensors on, and
// nontemporal loads where its two or four tensors together pass the last-level
// cache (8,192 x 4,096 bfloat16 with the residual: 48 us for 50 with such stores
// only; 100,003 x 255 float32, which stays under it, 44 us with and 40 without).
inline int rms_traffic(int64_t M, int64_t N, int elem_bytes, int tensors) {
    const int64_t bytes = M * N * elem_bytes;
    if (bytes * tensors >= ((int64_t)256 << 20)) return 2;
    return bytes >= ((int64_t)64 << 20) ? 1 : 0;
}

// Whether the backward takes one launch (rms_bwd_few_kernel). On the device, in one
// and in two launches: 1,024 x 64 float32 5.3 and 7.8 us, 512 x 1,024 5.7 and 8.8,
// 64 x 8,192 10.0 and 10.9, 16 x 4,096 4.7 and 8.6, but 2,048 x 64 9.7 and 8.2,
// 1,024 x 1,024 10.4 and 9.6, 512 x 4,096 13.8 and 12.1; the launch itself is some
// 3 us of the calling thread.
inline bool rms_few(int64_t M, int64_t N, int elem_bytes) {
    return M <= 1024 && M * N <= (1 << 19) && M * N * elem_bytes >= 16;
}

template <typename T> void rms_launch_forward(const LnConfig&, const RmsArgs&, hipStream_t);
template <typename T> void rms_launch_forward_q8(const LnConfig&, const RmsArgs&, hipStream_t);
template <typename T> void rms_launch_backward_few(const RmsArgs&, hipStream_t);
template <typename T> int rms_launch_backward(const LnConfig&, int grid, const RmsArgs&, hipStream_t);   // dyt_status

}  // namespace dytb
