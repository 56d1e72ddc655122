// lm_api.hip - C ABI of the root-mean-square norm (include/dyt_lm.h): argument
// checks, the choice of kernel, and the second pass of the backward.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "block_host.hpp"
#include "dyt_lm.h"
#include "rms_launch.hpp"

namespace dytb {
namespace {

// dgamma: column sums of the `rows` partial rows, 64 columns per workgroup,
// slices of rows side by side, each summed in row order, then the slices in
// slice order. A grid may have 2^32 threads: workgroups walk.
constexpr int kFinSlices = 16;
constexpr int64_t kFinGrid = 1 << 15;

__global__ __launch_bounds__(64 * kFinSlices) void rms_finish_kernel(const float* part, int64_t pitch, int rows,
                                                                     int64_t N, void* dgamma, int pdt) {
    __shared__ float red[kFinSlices][64];
    const int lane = (int)threadIdx.x & 63, slice = (int)threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < N; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float s = 0.0f;
        if (c < N) {
            const int per = (rows + kFinSlices - 1) / kFinSlices;
            const int lo = slice * per, hi = min(lo + per, rows);
#pragma unroll 8
            for (int r = lo; r < hi; ++r) s += part[r * pitch + c];
        }
        __syncthreads();   // the columns before have been read
        red[slice][lane] = s;
        __syncthreads();
        if (slice == 0 && c < N) {
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < kFinSlices; ++k) s += red[k][lane];
            store_param(dgamma, c, pdt, s);
        }
    }
}

void rms_finish(const float* part, int64_t pitch, int rows, int64_t N, void* dgamma, int pdt, hipStream_t s) {
    const int64_t need = (N + 63) / 64;
    rms_finish_kernel<<<(unsigned)std::min(need, kFinGrid), 64 * kFinSlices, 0, s>>>(part, pitch, rows, N, dgamma, pdt);
}

constexpr int64_t kMaxN = (int64_t)1 << 30;

struct RmsPlan {
    LnConfig cfg;
    int grid;
    int64_t pitch;
    size_t bytes;
};

int rms_shape(int64_t M, int64_t N, int xdt, int pdt) {
    if (M < 0 || N < 0 || N > kMaxN || (N > 0 && M > (INT64_MAX / 8) / N)) return DYT_ERR_INVALID_ARG;
    if (!dtype_ok(xdt) || !dtype_ok(pdt)) return DYT_ERR_UNSUPPORTED_DTYPE;
    return DYT_OK;
}

// Workgroups of the backward, each with a partial row of N floats to write and
// read again: two of 256 threads or one of 512 a CU, which resident workgroups walk
// without a last round of a few (32,768 x 4,096 bfloat16 with the residual: 171 us for
// 193 of 640 workgroups, 262,144 x 512 175 for 186, 1,000,000 x 100 136 for 145), while
// those rows stay near 3% of the activations' traffic (three tensors of M N
// elements of s bytes: 8 N grid <= 0.03 * 3 M N s).
RmsPlan rms_plan(int64_t M, int64_t N, int xdt) {
    RmsPlan p{};
    const int64_t bytes = dtype_size(xdt);
    p.cfg = rms_config(M, N, (int)bytes, true);
    const int64_t need = (M + ln_groups(p.cfg) - 1) / ln_groups(p.cfg);
    const int64_t most = p.cfg.threads > 512 || p.cfg.threads == 0 ? 256 : 131072 / p.cfg.wg;
    const int64_t cap = std::min(most, std::max<int64_t>(256, M * bytes / 89 / 128 * 128));
    p.grid = (int)std::min(need, cap);
    p.pitch = (N + 31) / 32 * 32;
    p.bytes = (size_t)p.grid * p.pitch * sizeof(float);
    return p;
}

template <typename F>
void with_type(int xdt, F&& f) {
    if (xdt == DYT_F32) f((float*)nullptr);
    else if (xdt == DYT_BF16) f((bf16_t*)nullptr);
    else f((f16_t*)nullptr);
}

// q8: y holds the codes and `stats` the scales, else y and rstd.
int rms_forward(const void* x, int64_t ldx, const void* r, const void* gamma, void* h, void* y, int64_t ldy,
                float* stats, int64_t M, int64_t N, float eps, int xdt, int pdt, bool res, bool q8, int group,
                void* stream) {
    if (int e = rms_shape(M, N, xdt, pdt)) return e;
    if (ldx == 0) ldx = N;
    if (ldy == 0) ldy = N;
    if (!(eps >= 0.0f) || std::isinf(eps) || !pitch_ok(M, N, ldx) || !pitch_ok(M, N, ldy)) return DYT_ERR_INVALID_ARG;
    if (res && ldx != N && M > 1) return DYT_ERR_INVALID_ARG;
    if (group != 0 && group != 32 && group != 64 && group != 128) return DYT_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return DYT_OK;
    if (!x || !gamma || !y || !stats || (res && (!r || !h))) return DYT_ERR_INVALID_ARG;
    const int64_t sx = dtype_size(xdt), sp = dtype_size(pdt);
    if (!aligned({x, r, h}, sx) || !aligned({y}, q8 ? 1 : sx) || !aligned({gamma}, sp) || !aligned({stats}, 4))
        return DYT_ERR_MISALIGNED;
    const int64_t bx = ((M - 1) * ldx + N) * sx, by = q8 ? M * N : ((M - 1) * ldy + N) * sx;
    const int64_t n_stats = M * (group ? (N + group - 1) / group : 1);
    const Range in[] = {{x, bx}, {r, res ? bx : 0}, {gamma, N * sp}};
    const Range out[] = {{y, by}, {h, res ? bx : 0}, {stats, n_stats * 4}};
    if (!disjoint(in, 3, out, 3)) return DYT_ERR_INVALID_ARG;
    RmsArgs a{};
    a.x = x; a.r = res ? r : nullptr; a.h = h; a.y = y; a.gamma = gamma; a.rstd = stats; a.scales = stats;
    a.ldx = ldx; a.ldy = ldy; a.M = M; a.N = (int32_t)N; a.pdt = pdt; a.eps = eps; a.group = group;
    a.traffic = rms_traffic(M, N, (int)sx, res ? 4 : 2);
    const LnConfig cfg = rms_config(M, N, (int)sx, false);
    with_type(xdt, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (q8) rms_launch_forward_q8<T>(cfg, a, (hipStream_t)stream);
        else rms_launch_forward<T>(cfg, a, (hipStream_t)stream);
    });
    return hip_status();
}

int rms_backward(const void* x, int64_t ldx, const void* dy, int64_t lddy, const void* dres, const float* rstd,
                 const void* gamma, void* dx, int64_t lddx, void* dgamma, void* ws, size_t ws_bytes, int64_t M,
                 int64_t N, int xdt, int pdt, bool res, void* stream) {
    if (int e = rms_shape(M, N, xdt, pdt)) return e;
    if (ldx == 0) ldx = N;
    if (lddy == 0) lddy = N;
    if (lddx == 0) lddx = N;
    if (!pitch_ok(M, N, ldx) || !pitch_ok(M, N, lddy) || !pitch_ok(M, N, lddx)) return DYT_ERR_INVALID_ARG;
    if (N == 0) return DYT_OK;
    if (!dgamma) return DYT_ERR_INVALID_ARG;
    const int64_t sx = dtype_size(xdt), sp = dtype_size(pdt);
    const hipStream_t s = (hipStream_t)stream;
    if (M == 0) {
        if (!aligned({dgamma}, sp)) return DYT_ERR_MISALIGNED;
        rms_finish(nullptr, 0, 0, N, dgamma, pdt, s);
        return hip_status();
    }
    if (!x || !dy || !rstd || !gamma || !dx || (res && !dres)) return DYT_ERR_INVALID_ARG;
    if (!aligned({x, dy, dres, dx}, sx) || !aligned({gamma, dgamma}, sp) || !aligned({rstd}, 4)) return DYT_ERR_MISALIGNED;
    const RmsPlan p = rms_plan(M, N, xdt);
    if (ws_bytes < p.bytes || !ws) return DYT_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned({ws}, 16)) return DYT_ERR_MISALIGNED;
    const int64_t bx = ((M - 1) * ldx + N) * sx, bdy = ((M - 1) * lddy + N) * sx, bdx = ((M - 1) * lddx + N) * sx;
    const Range in[] = {{x, bx}, {dy, bdy}, {dres, dres ? bx : 0}, {gamma, N * sp}, {rstd, M * 4}};
    const Range out[] = {{dx, bdx}, {dgamma, N * sp}, {ws, (int64_t)p.bytes}};
    if (!disjoint(in, 5, out, 3)) return DYT_ERR_INVALID_ARG;
    RmsArgs a{};
    a.x = x; a.dy = dy; a.dres = res ? dres : nullptr; a.y = dx; a.gamma = gamma;
    a.rstd = const_cast<float*>(rstd); a.part = (float*)ws;
    a.ldx = ldx; a.lddy = lddy; a.ldy = lddx; a.M = M; a.N = (int32_t)N; a.pdt = pdt; a.pitch = p.pitch;
    a.traffic = ln_traffic(M, N, (int)sx, true);
    a.dgamma = dgamma;
    if (rms_few(M, N, (int)sx)) {
        with_type(xdt, [&](auto* t) { rms_launch_backward_few<std::remove_pointer_t<decltype(t)>>(a, s); });
        return hip_status();
    }
    int e = DYT_OK;
    with_type(xdt, [&](auto* t) {
        e = rms_launch_backward<std::remove_pointer_t<decltype(t)>>(p.cfg, p.grid, a, s);
    });
    if (e) return e;
    rms_finish(a.part, a.pitch, p.grid, N, dgamma, pdt, s);
    return hip_status();
}

#ifndef DYT_BUILD_ID
#define DYT_BUILD_ID "unset"
#endif
__attribute__((used)) const char kBuildId[] = "DYT_BUILD_ID=" DYT_BUILD_ID;
constexpr int kBuildIdSkip = sizeof("DYT_BUILD_ID=") - 1;

}  // namespace
}  // namespace dytb

using namespace dytb;

extern "C" {

int dyt_lm_abi_version(void) { return DYT_LM_ABI_VERSION; }

const char* dyt_lm_build_id(void) { return kBuildId + kBuildIdSkip; }

int dyt_rms_forward(const void* x, int64_t ldx, const void* gamma, void* y, int64_t ldy, float* rstd, int64_t M,
                    int64_t N, float eps, int x_dtype, int param_dtype, void* stream) {
    return rms_forward(x, ldx, nullptr, gamma, nullptr, y, ldy, rstd, M, N, eps, x_dtype, param_dtype, false, false,
                       0, stream);
}

int dyt_rms_forward_residual(const void* x, const void* r, const void* gamma, void* h, void* y, float* rstd,
                             int64_t M, int64_t N, float eps, int x_dtype, int param_dtype, void* stream) {
    return rms_forward(x, 0, r, gamma, h, y, 0, rstd, M, N, eps, x_dtype, param_dtype, true, false, 0, stream);
}

int dyt_rms_forward_q8(const void* x, int64_t ldx, const void* r, const void* gamma, void* h, void* q, float* scales,
                       int64_t M, int64_t N, int group, float eps, int x_dtype, int param_dtype, void* stream) {
    return rms_forward(x, ldx, r, gamma, h, q, 0, scales, M, N, eps, x_dtype, param_dtype, r != nullptr || h != nullptr,
                       true, group, stream);
}

size_t dyt_rms_backward_workspace_size(int64_t M, int64_t N, int x_dtype, int param_dtype) {
    if (rms_shape(M, N, x_dtype, param_dtype) || M == 0 || N == 0) return 0;
    return rms_plan(M, N, x_dtype).bytes;
}

int dyt_rms_backward(const void* x, int64_t ldx, const void* dy, int64_t lddy, const float* rstd, const void* gamma,
                     void* dx, int64_t lddx, void* dgamma, void* workspace, size_t workspace_bytes, int64_t M,
                     int64_t N, int x_dtype, int param_dtype, void* stream) {
    return rms_backward(x, ldx, dy, lddy, nullptr, rstd, gamma, dx, lddx, dgamma, workspace, workspace_bytes, M, N,
                        x_dtype, param_dtype, false, stream);
}

int dyt_rms_backward_residual(const void* h, const void* dy, const void* dres, const float* rstd, const void* gamma,
                              void* dx, void* dgamma, void* workspace, size_t workspace_bytes, int64_t M, int64_t N,
                              int x_dtype, int param_dtype, void* stream) {
    return rms_backward(h, 0, dy, 0, dres, rstd, gamma, dx, 0, dgamma, workspace, workspace_bytes, M, N, x_dtype,
                        param_dtype, true, stream);
}

}  // extern "C"
