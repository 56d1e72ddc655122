// block_api.hip - C ABI of the layer norm (include/dyt_block.h): argument
// checks, the choice of kernel, and the second pass of the backward.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "block_host.hpp"
#include "dyt_block.h"
#include "ln_launch.hpp"

namespace dytb {

// dgamma and dbeta: column sums of the `rows` partial rows. 64 columns per
// workgroup, kFinSlices slices of rows side by side, each summed in row
// order, then the slices in slice order. The loads of a slice do not depend
// on each other; 16 slices of up to 64 rows each take 3-7 us up to 16,384 columns, 12
// at 33,000.
// A grid may have 2^32 threads: from 2^15 workgroups on (over a million columns)
// they walk (WALK).
constexpr int kFinSlices = 16;
constexpr int64_t kFinGrid = 1 << 15;

template <bool WALK>
__global__ __launch_bounds__(64 * kFinSlices) void ln_finish_kernel(const float* part, int64_t pitch,
                                                                    int rows, int64_t N, void* dgamma,
                                                                    void* dbeta, int pdt) {
    __shared__ float red[kFinSlices][64];
    const int lane = (int)threadIdx.x & 63, slice = (int)threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < 2 * N; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float s = 0.0f;
        if (c < 2 * N) {
            const int per = (rows + kFinSlices - 1) / kFinSlices;
            const int lo = slice * per, hi = min(lo + per, rows);
#pragma unroll 8
            for (int r = lo; r < hi; ++r) s += part[r * pitch + c];
        }
        if constexpr (WALK) __syncthreads();   // the columns before have been read
        red[slice][lane] = s;
        __syncthreads();
        if (slice == 0 && c < 2 * N) {
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < kFinSlices; ++k) s += red[k][lane];
            if (c < N) store_param(dgamma, c, pdt, s);
            else store_param(dbeta, c - N, pdt, s);
        }
        if constexpr (!WALK) return;
    }
}

void ln_finish(const float* part, int64_t pitch, int rows, int64_t N, void* dgamma, void* dbeta, int pdt, hipStream_t s) {
    const int64_t need = (2 * N + 63) / 64;
    if (need <= kFinGrid) ln_finish_kernel<false><<<(unsigned)need, 64 * kFinSlices, 0, s>>>(part, pitch, rows, N, dgamma, dbeta, pdt);
    else ln_finish_kernel<true><<<(unsigned)kFinGrid, 64 * kFinSlices, 0, s>>>(part, pitch, rows, N, dgamma, dbeta, pdt);
}

// Workgroups of the backward, each with a partial row of 2 N floats to write
// and read again: as many as fill the card, while those rows stay near 3% of
// the activations' traffic (three tensors of M N elements of s bytes:
// 16 N grid <= 0.03 * 3 M N s).
int ln_bwd_grid(const LnConfig& c, int64_t M, int64_t elem_bytes) {
    const int64_t need = (M + ln_groups(c) - 1) / ln_groups(c);
    const int64_t most = c.threads > 512 || c.threads == 0 ? 256 : 1024;
    const int64_t cap = std::min(most, std::max<int64_t>(256, M * elem_bytes / 178 / 128 * 128));
    return (int)std::min(need, cap);
}

namespace {

constexpr int64_t kMaxN = (int64_t)1 << 30;

struct LnPlan {
    LnConfig cfg;
    int grid;
    int64_t pitch;
    size_t bytes;
};

int ln_shape(int64_t M, int64_t N, int xdt, int pdt) {
    if (M < 0 || N < 0 || N > kMaxN || (N > 0 && M > (INT64_MAX / 8) / N)) return DYT_ERR_INVALID_ARG;
    if (!dtype_ok(xdt) || !dtype_ok(pdt)) return DYT_ERR_UNSUPPORTED_DTYPE;
    return DYT_OK;
}

LnPlan ln_plan(int64_t M, int64_t N, int xdt) {
    LnPlan p{};
    const int bytes = (int)dtype_size(xdt);
    p.cfg = ln_config(M, N, bytes, true);
    p.grid = ln_bwd_grid(p.cfg, M, bytes);
    p.pitch = (2 * N + 31) / 32 * 32;
    p.bytes = (size_t)p.grid * p.pitch * sizeof(float);
    return p;
}

template <typename F>
void with_type(int xdt, F&& f) {
    if (xdt == DYT_F32) f((float*)nullptr);
    else if (xdt == DYT_BF16) f((bf16_t*)nullptr);
    else f((f16_t*)nullptr);
}

int ln_forward(const void* x, int64_t ldx, const void* r, const void* gamma, const void* beta, void* h,
               void* y, int64_t ldy, float* mean, float* rstd, int64_t M, int64_t N, float eps, int xdt,
               int pdt, bool res, void* stream) {
    if (int e = ln_shape(M, N, xdt, pdt)) return e;
    if (ldx == 0) ldx = N;
    if (ldy == 0) ldy = N;
    if (!(eps >= 0.0f) || std::isinf(eps) || !pitch_ok(M, N, ldx) || !pitch_ok(M, N, ldy)) return DYT_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return DYT_OK;
    if (!x || !gamma || !beta || !y || !mean || !rstd || (res && (!r || !h))) return DYT_ERR_INVALID_ARG;
    const int64_t sx = dtype_size(xdt), sp = dtype_size(pdt);
    if (!aligned({x, r, h, y}, sx) || !aligned({gamma, beta}, sp) || !aligned({mean, rstd}, 4)) return DYT_ERR_MISALIGNED;
    const int64_t bx = ((M - 1) * ldx + N) * sx, by = ((M - 1) * ldy + N) * sx;
    const Range in[] = {{x, bx}, {r, r ? bx : 0}, {gamma, N * sp}, {beta, N * sp}};
    const Range out[] = {{y, by}, {h, h ? bx : 0}, {mean, M * 4}, {rstd, M * 4}};
    if (!disjoint(in, 4, out, 4)) return DYT_ERR_INVALID_ARG;
    LnArgs a{};
    a.x = x; a.r = res ? r : nullptr; a.h = h; a.y = y; a.gamma = gamma; a.beta = beta;
    a.mean = mean; a.rstd = rstd; a.ldx = ldx; a.ldy = ldy; a.M = M; a.N = (int32_t)N; a.pdt = pdt; a.eps = eps;
    a.traffic = ln_traffic(M, N, (int)sx, res);
    const LnConfig cfg = ln_config(M, N, (int)sx, false);
    with_type(xdt, [&](auto* t) {
        ln_launch_forward<std::remove_pointer_t<decltype(t)>>(cfg, a, (hipStream_t)stream);
    });
    return hip_status();
}

int ln_backward(const void* x, int64_t ldx, const void* dy, int64_t lddy, const void* dres, const float* mean,
                const float* rstd, const void* gamma, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                void* ws, size_t ws_bytes, int64_t M, int64_t N, int xdt, int pdt, bool res, void* stream) {
    if (int e = ln_shape(M, N, xdt, pdt)) return e;
    if (ldx == 0) ldx = N;
    if (lddy == 0) lddy = N;
    if (lddx == 0) lddx = N;
    if (!pitch_ok(M, N, ldx) || !pitch_ok(M, N, lddy) || !pitch_ok(M, N, lddx)) return DYT_ERR_INVALID_ARG;
    if (N == 0) return DYT_OK;
    if (!dgamma || !dbeta) return DYT_ERR_INVALID_ARG;
    const int64_t sx = dtype_size(xdt), sp = dtype_size(pdt);
    const hipStream_t s = (hipStream_t)stream;
    if (M == 0) {
        if (!aligned({dgamma, dbeta}, sp)) return DYT_ERR_MISALIGNED;
        ln_finish(nullptr, 0, 0, N, dgamma, dbeta, pdt, s);
        return hip_status();
    }
    if (!x || !dy || !mean || !rstd || !gamma || !dx || (res && !dres)) return DYT_ERR_INVALID_ARG;
    if (!aligned({x, dy, dres, dx}, sx) || !aligned({gamma, dgamma, dbeta}, sp) || !aligned({mean, rstd}, 4))
        return DYT_ERR_MISALIGNED;
    const LnPlan p = ln_plan(M, N, xdt);
    if (ws_bytes < p.bytes || !ws) return DYT_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned({ws}, 16)) return DYT_ERR_MISALIGNED;
    const int64_t bx = ((M - 1) * ldx + N) * sx, bdy = ((M - 1) * lddy + N) * sx, bdx = ((M - 1) * lddx + N) * sx;
    const Range in[] = {{x, bx}, {dy, bdy}, {dres, dres ? bx : 0}, {gamma, N * sp}, {mean, M * 4}, {rstd, M * 4}};
    const Range out[] = {{dx, bdx}, {dgamma, N * sp}, {dbeta, N * sp}, {ws, (int64_t)p.bytes}};
    if (!disjoint(in, 6, out, 4)) return DYT_ERR_INVALID_ARG;
    LnArgs a{};
    a.x = x; a.dy = dy; a.dres = res ? dres : nullptr; a.y = dx; a.gamma = gamma;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd); a.part = (float*)ws;
    a.ldx = ldx; a.lddy = lddy; a.ldy = lddx; a.M = M; a.N = (int32_t)N; a.pdt = pdt; a.pitch = p.pitch;
    a.traffic = ln_traffic(M, N, (int)sx, true);
    with_type(xdt, [&](auto* t) {
        ln_launch_backward<std::remove_pointer_t<decltype(t)>>(p.cfg, p.grid, a, s);
    });
    ln_finish(a.part, a.pitch, p.grid, N, dgamma, dbeta, pdt, s);
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

int dyt_block_abi_version(void) { return DYT_BLOCK_ABI_VERSION; }

const char* dyt_block_build_id(void) { return kBuildId + kBuildIdSkip; }

int dyt_ln_forward(const void* x, int64_t ldx, const void* gamma, const void* beta, void* y, int64_t ldy,
                   float* mean, float* rstd, int64_t M, int64_t N, float eps, int x_dtype, int param_dtype,
                   void* stream) {
    return ln_forward(x, ldx, nullptr, gamma, beta, nullptr, y, ldy, mean, rstd, M, N, eps, x_dtype,
                      param_dtype, false, stream);
}

int dyt_ln_forward_residual(const void* x, const void* r, const void* gamma, const void* beta, void* h,
                            void* y, float* mean, float* rstd, int64_t M, int64_t N, float eps, int x_dtype,
                            int param_dtype, void* stream) {
    return ln_forward(x, 0, r, gamma, beta, h, y, 0, mean, rstd, M, N, eps, x_dtype, param_dtype, true, stream);
}

size_t dyt_ln_backward_workspace_size(int64_t M, int64_t N, int x_dtype, int param_dtype) {
    if (ln_shape(M, N, x_dtype, param_dtype) || M == 0 || N == 0) return 0;
    return ln_plan(M, N, x_dtype).bytes;
}

int dyt_ln_backward(const void* x, int64_t ldx, const void* dy, int64_t lddy, const float* mean,
                    const float* rstd, const void* gamma, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                    void* workspace, size_t workspace_bytes, int64_t M, int64_t N, int x_dtype,
                    int param_dtype, void* stream) {
    return ln_backward(x, ldx, dy, lddy, nullptr, mean, rstd, gamma, dx, lddx, dgamma, dbeta, workspace,
                       workspace_bytes, M, N, x_dtype, param_dtype, false, stream);
}

int dyt_ln_backward_residual(const void* h, const void* dy, const void* dres, const float* mean,
                             const float* rstd, const void* gamma, void* dx, void* dgamma, void* dbeta,
                             void* workspace, size_t workspace_bytes, int64_t M, int64_t N, int x_dtype,
                             int param_dtype, void* stream) {
    return ln_backward(h, 0, dy, 0, dres, mean, rstd, gamma, dx, 0, dgamma, dbeta, workspace, workspace_bytes,
                       M, N, x_dtype, param_dtype, true, stream);
}

}  // extern "C"
