// rms_kernels.hpp - root-mean-square norm, forward and backward (gfx950).
//
//   rstd_i = 1 / sqrt(sum_j x[i,j]^2 / N + eps)    n[i,j] = x[i,j] rstd_i
//   y[i,j] = gamma[j] n[i,j]                       d[i,j] = dy[i,j] gamma[j]
//   dx[i,j] = rstd_i (d[i,j] - n[i,j] sum_j (d n)[i,j] / N)
//   dgamma[j] = sum_i dy[i,j] n[i,j]
//
// Bound by HBM traffic like the layer norm, and laid out like it: TPR threads
// hold a row as V vectors of 16 bytes between its one sum and its use, U rows
// side by side where a row is few vectors. There is no mean to take out first,
// so each direction needs a single reduction. The 8-bit output adds one more,
// of the largest |y| of a row or of a group of neighbouring columns; a group of
// 32, 64 or 128 lies in neighbouring lanes of one wave, so its maximum takes
// lane exchanges only.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

constexpr float kE4m3Most = 448.0f;       // largest finite e4m3 value
constexpr float kScaleLeast = 0x1p-126f;  // so that 1 / scale is finite

struct RmsArgs {
    const void* x;        // forward: x; backward: x or h
    const void* r;        // forward: residual or null
    void* h;              // forward: x + r, or null
    void* y;              // forward: y or the 8-bit codes; backward: dx
    const void* dy;       // backward
    const void* dres;     // backward: residual gradient or null
    const void* gamma;
    float* rstd;
    float* scales;        // 8-bit output: [M, groups]
    float* part;          // backward: partial rows
    void* dgamma;         // backward of few elements
    int64_t ldx, ldy, lddy;
    int64_t M;
    int32_t N;
    int32_t pdt;
    float eps;
    int32_t group;        // 8-bit output: columns of a scale, 0: the row
    int64_t pitch;        // backward: floats between partial rows
    int32_t traffic;      // cache hints, see ln_traffic
};

// Parameters of the VEC columns from c on (0 past N).
template <int VEC>
__device__ __forceinline__ void load_params(const void* p, int dt, int c, int N, float* out) {
    load_columns<1, VEC, 1>(p, dt, c / VEC, N, out);
}

__device__ __forceinline__ float lanes_max(float v, int lanes) {
    if (lanes >= 2) v = fmaxf(v, dpp_mov<0xB1>(v));     // lane ^ 1
    if (lanes >= 4) v = fmaxf(v, dpp_mov<0x4E>(v));     // lane ^ 2
    if (lanes >= 8) v = fmaxf(v, dpp_mov<0x141>(v));    // mirrored within 8
    if (lanes >= 16) v = fmaxf(v, dpp_mov<0x140>(v));   // mirrored within 16
    if (lanes >= 32) {
        const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(
            __float_as_uint(v), __float_as_uint(v), false, false));
        v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    }
    if (lanes >= 64) v = swap32_max(v);
    return v;
}

// Scale of a maximum. NaN elements are left out of it (fmaxf drops them) and
// become NaN codes.
__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax / kE4m3Most, kScaleLeast); }

// Division by a scale: the product with the reciprocal and one correction by
// what is left of y, which is the float32 quotient. The product alone may be one
// step off, and of 16-bit elements, whose quotients often lie in the middle between
// two codes, 35 in a million got the other code. (No correction for an infinite
// scale, whose finite elements get 0.)
struct ByScale {
    float inv, scale;

    __device__ __forceinline__ explicit ByScale(float s) : inv(1.0f / s), scale(s < INFINITY ? s : 0.0f) {}

    __device__ __forceinline__ float operator()(float y) const {
        const float q = y * inv;
        return __builtin_fmaf(-__builtin_fmaf(q, scale, -y), inv, q);   // (so written a -0 keeps its sign)
    }
};

// VEC codes of y / scale, rounded to nearest even, at element c of a row.
template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int N, const float* y, ByScale by) {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(by(y[4 * i]), by(y[4 * i + 1]), 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(by(y[4 * i + 2]), by(y[4 * i + 3]), v, true);
    }
    if (c + VEC <= N) {
        __builtin_memcpy(row + c, w, VEC);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < N) row[c + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// Q8: codes and scales in place of y and rstd. Rows of more than 32 elements a
// thread do not fit gamma into the registers beside them and read it at its use.
template <typename T, int TPR, int V, int U, bool RES, bool Q8, int NT>
__global__ __launch_bounds__(LnShape<TPR>::threads) void rms_fwd_kernel(RmsArgs a) {
    using S = LnShape<TPR>;
    constexpr int VEC = VecOf<T>::n;
    constexpr int E = V * VEC;
    constexpr bool HOLD = E <= 32, AHEAD = TPR >= 256 && V <= 2;
    const int t = (int)threadIdx.x % TPR;
    const int g = (int)threadIdx.x / TPR;
    const int N = a.N;
    float gm[HOLD ? E : VEC];
    if constexpr (HOLD) load_columns<V, VEC, TPR>(a.gamma, a.pdt, t, N, gm);
    const float inv_n = 1.0f / (float)N;
    const int64_t limit = (a.M - 1) * a.ldx + N;
    const int64_t step = (int64_t)gridDim.x * S::groups * U;
    const T* xp = (const T*)a.x;
    struct Raw {
        u32x4 x[V], r[RES ? V : 1];
    };
    const auto load = [&](int64_t m, Raw& w) {
        const bool on = m < a.M;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (t + v * TPR) * VEC;
            w.x[v] = load_raw<T, NT>(xp, m * a.ldx, c, N, limit, on);
            if constexpr (RES) w.r[v] = load_raw<T, NT>((const T*)a.r, m * a.ldx, c, N, limit, on);
        }
    };
    Raw next[AHEAD ? U : 1];
    int64_t base = (int64_t)blockIdx.x * S::groups * U;
    if constexpr (AHEAD) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(base + u * S::groups + g, next[u]);
    }
    for (int buf = 0; base < a.M; base += step, buf ^= 1) {
        float x[U][E], ss[U];
        Raw now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (AHEAD) now[u] = next[u];
            else load(base + u * S::groups + g, now[u]);
        }
        if constexpr (AHEAD) {
#pragma unroll
            for (int u = 0; u < U; ++u) load(base + step + u * S::groups + g, next[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
            ss[u] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (t + v * TPR) * VEC;
                float* xv = &x[u][v * VEC];
                unpack_raw<T>(now[u].x[v], xp, m * a.ldx, c, N, limit, m < a.M, xv);
                if constexpr (RES) {
                    float r[VEC];
                    unpack_raw<T>(now[u].r[v], (const T*)a.r, m * a.ldx, c, N, limit, m < a.M, r);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) r[i] += xv[i];
                    if (m < a.M) store_vec<T, NT>((T*)a.h, m * a.ldx, c, N, r);
                    // the layer's input is h as stored
                    unpack16<T>(pack16<T>(r), xv);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss[u] = __builtin_fmaf(xv[i], xv[i], ss[u]);
            }
            ss[u] = lanes_sum<S::L>(ss[u]);
        }
        if constexpr (S::waves > 1) {
            static_assert(S::groups == 1, "a row of several waves has the workgroup to itself");
            __shared__ float red[2][U][S::waves];   // the next rows' sums go to the other half
            if ((t & 63) == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) red[buf][u][t >> 6] = ss[u];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ss[u] = 0.0f;
#pragma unroll
                for (int k = 0; k < S::waves; ++k) ss[u] += red[buf][u][k];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
            const float rs = inv_sqrt(__builtin_fmaf(ss[u], inv_n, a.eps));
            float most = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (t + v * TPR) * VEC;
                if constexpr (!HOLD) load_params<VEC>(a.gamma, a.pdt, c, N, gm);
                float* xv = &x[u][v * VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    xv[i] = xv[i] * rs * gm[(HOLD ? v * VEC : 0) + i];
                    if constexpr (Q8) most = fmaxf(most, __builtin_fabsf(xv[i]));
                }
                if constexpr (!Q8) {
                    if (m < a.M) store_vec<T, NT>((T*)a.y, m * a.ldy, c, N, xv);
                } else if (a.group) {
                    // a group's lanes are neighbours; a row narrower than it has TPR of them
                    const float sc = scale_of(lanes_max(most, min(a.group / VEC, TPR)));
                    most = 0.0f;
                    if (m < a.M && c < N) {
                        store_codes<VEC>((uint8_t*)a.y + m * N, c, N, xv, ByScale(sc));
                        if (c % a.group == 0) a.scales[m * ((N + a.group - 1) / a.group) + c / a.group] = sc;
                    }
                }
            }
            if constexpr (!Q8) {
                if (t == 0 && m < a.M) a.rstd[m] = rs;
            } else if (!a.group) {
                most = lanes_max(most, S::L);
                if constexpr (S::waves > 1) {
                    __shared__ float top[2][U][S::waves];
                    if ((t & 63) == 0) top[buf][u][t >> 6] = most;
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < S::waves; ++k) most = fmaxf(most, top[buf][u][k]);
                }
                const float sc = scale_of(most);
                const ByScale by(sc);
                if (m < a.M) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        store_codes<VEC>((uint8_t*)a.y + m * N, (t + v * TPR) * VEC, N, &x[u][v * VEC], by);
                    if (t == 0) a.scales[m] = sc;
                }
            }
        }
    }
}

// Rows longer than 1,024 threads hold: a workgroup per row, walked again from
// the last-level caches for each use.
template <typename T, bool RES, bool Q8>
__global__ __launch_bounds__(kLongThreads) void rms_fwd_long_kernel(RmsArgs a) {
    constexpr int VEC = VecOf<T>::n;
    __shared__ float red[kLongThreads / 64];
    const int N = a.N, first = (int)threadIdx.x * VEC;
    // every lane takes part in the lane exchanges of a group
    const int end = (N + kLongThreads * VEC - 1) / (kLongThreads * VEC) * (kLongThreads * VEC);
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const T* src = (const T*)a.x;
        float s = 0.0f;
        for (int c = first; c < N; c += kLongThreads * VEC) {
            float x[VEC];
            load_vec<T>(src, m * a.ldx, c, N, x);
            if constexpr (RES) {
                float r[VEC];
                load_vec<T>((const T*)a.r, m * a.ldx, c, N, r);
#pragma unroll
                for (int i = 0; i < VEC; ++i) r[i] += x[i];
                store_vec<T>((T*)a.h, m * a.ldx, c, N, r);
                unpack16<T>(pack16<T>(r), x);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) s = __builtin_fmaf(x[i], x[i], s);
        }
        if constexpr (RES) src = (const T*)a.h;   // each thread reads back its own stores
        const float rs = inv_sqrt(block_sum(s, red) / (float)N + a.eps);
        const auto value = [&](int c, float* y) {
            float gm[VEC];
            load_vec<T>(src, m * a.ldx, c, N, y);
            load_params<VEC>(a.gamma, a.pdt, c, N, gm);
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = y[i] * rs * gm[i];
        };
        float most = 0.0f;
        if (Q8 && !a.group) {
            for (int c = first; c < N; c += kLongThreads * VEC) {
                float y[VEC];
                value(c, y);
#pragma unroll
                for (int i = 0; i < VEC; ++i) most = fmaxf(most, __builtin_fabsf(y[i]));
            }
            most = lanes_max(most, 64);
            __syncthreads();   // the sum has been read
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = most;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kLongThreads / 64; ++k) most = fmaxf(most, red[k]);
        }
        const float sc = scale_of(most);
        const ByScale by(sc);
        for (int c = first; c < (Q8 ? end : N); c += kLongThreads * VEC) {
            float y[VEC];
            if constexpr (!Q8) {
                value(c, y);
                store_vec<T>((T*)a.y, m * a.ldy, c, N, y);
            } else if (!a.group) {
                if (c < N) {
                    value(c, y);
                    store_codes<VEC>((uint8_t*)a.y + m * N, c, N, y, by);
                }
            } else {
                float top = 0.0f;
                if (c < N) {
                    value(c, y);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) top = fmaxf(top, __builtin_fabsf(y[i]));
                }
                const float gsc = scale_of(lanes_max(top, a.group / VEC));
                if (c < N) {
                    store_codes<VEC>((uint8_t*)a.y + m * N, c, N, y, ByScale(gsc));
                    if (c % a.group == 0) a.scales[m * ((N + a.group - 1) / a.group) + c / a.group] = gsc;
                }
            }
        }
        if (threadIdx.x == 0) {
            if constexpr (!Q8) a.rstd[m] = rs;
            else if (!a.group) a.scales[m] = sc;
        }
    }
}

// As the layer norm's backward: U row groups at a time, the next rows' vectors
// loaded before the current ones are reduced (AHEAD; four vectors a thread would
// spill for it), a thread's columns of dgamma summed in
// registers over the rows its workgroup walks, one float32 row of sums per
// workgroup.
template <typename T, int TPR, int TH, int V, int U, bool RES, int NT>
__global__ __launch_bounds__(TH) void rms_bwd_kernel(RmsArgs a) {
    using S = LnShape<TPR, TH>;
    constexpr int VEC = VecOf<T>::n;
    constexpr int E = V * VEC;
    constexpr bool AHEAD = E < 32;
    const int t = (int)threadIdx.x % TPR;
    const int g = (int)threadIdx.x / TPR;
    const int N = a.N;
    float gm[E], ag[E];
    load_columns<V, VEC, TPR>(a.gamma, a.pdt, t, N, gm);
#pragma unroll
    for (int e = 0; e < E; ++e) ag[e] = 0.0f;
    const float inv_n = 1.0f / (float)N;
    const int64_t limit = (a.M - 1) * a.ldx + N;
    const int64_t limit_dy = (a.M - 1) * a.lddy + N;
    const int64_t step = (int64_t)gridDim.x * S::groups * U;
    struct Raw {
        u32x4 x[V], dy[V], res[RES ? V : 1];
        float rs;
    };
    const auto load = [&](int64_t m, Raw& w) {
        const bool on = m < a.M;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (t + v * TPR) * VEC;
            w.x[v] = load_raw<T, NT>((const T*)a.x, m * a.ldx, c, N, limit, on);
            w.dy[v] = load_raw<T, NT>((const T*)a.dy, m * a.lddy, c, N, limit_dy, on);
            if constexpr (RES) w.res[v] = load_raw<T, NT>((const T*)a.dres, m * a.ldx, c, N, limit, on);
        }
        w.rs = a.rstd[on ? m : 0];
    };
    Raw next[AHEAD ? U : 1];
    int64_t base = (int64_t)blockIdx.x * S::groups * U;
    if constexpr (AHEAD) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(base + u * S::groups + g, next[u]);
    }
    for (int buf = 0; base < a.M; base += step, buf ^= 1) {
        Raw now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (AHEAD) now[u] = next[u];
            else load(base + u * S::groups + g, now[u]);
        }
        if constexpr (AHEAD) {
#pragma unroll
            for (int u = 0; u < U; ++u) load(base + step + u * S::groups + g, next[u]);
        }
        float n[U][E], dy[U][E], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
            s[u] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (t + v * TPR) * VEC;
                unpack_raw<T>(now[u].x[v], (const T*)a.x, m * a.ldx, c, N, limit, m < a.M, &n[u][v * VEC]);
                unpack_raw<T>(now[u].dy[v], (const T*)a.dy, m * a.lddy, c, N, limit_dy, m < a.M, &dy[u][v * VEC]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    n[u][e] *= now[u].rs;
                    const float dn = dy[u][e] * n[u][e];
                    ag[e] += dn;
                    s[u] = __builtin_fmaf(dn, gm[e], s[u]);
                }
            }
            s[u] = lanes_sum<S::L>(s[u]);
        }
        if constexpr (S::waves > 1) {
            __shared__ float red[2][U][S::groups][S::waves];
            if ((t & 63) == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) red[buf][u][g][t >> 6] = s[u];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] = 0.0f;
#pragma unroll
                for (int k = 0; k < S::waves; ++k) s[u] += red[buf][u][g][k];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
            if (m >= a.M) continue;
            const float c2 = s[u] * inv_n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float o[VEC], res[VEC];
                const int c = (t + v * TPR) * VEC;
                if constexpr (RES) unpack_raw<T>(now[u].res[v], (const T*)a.dres, m * a.ldx, c, N, limit, true, res);
                if constexpr (!AHEAD && VEC > 4 && !RES) {
                    // The compiler spills 132 bytes for the floats kept over the reduction (with
                    // the residual it keeps them, and spills 100 for this): unpacked again.
                    asm volatile("" : "+v"(now[u].x[v]), "+v"(now[u].dy[v]));
                    unpack_raw<T>(now[u].x[v], (const T*)a.x, m * a.ldx, c, N, limit, true, &n[u][v * VEC]);
                    unpack_raw<T>(now[u].dy[v], (const T*)a.dy, m * a.lddy, c, N, limit_dy, true, &dy[u][v * VEC]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) n[u][v * VEC + i] *= now[u].rs;
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    o[i] = now[u].rs * (dy[u][e] * gm[e] - n[u][e] * c2);
                    if constexpr (RES) o[i] += res[i];
                }
                store_vec<T, NT>((T*)a.y, m * a.ldy, c, N, o);
            }
        }
    }
    float* row = a.part + (int64_t)blockIdx.x * a.pitch;
    if constexpr (S::groups > 1) {
        // join the row groups, the upper half onto the lower one
        __shared__ float join[E][TH / 2];
#pragma unroll
        for (int half = S::groups / 2; half > 0; half /= 2) {
            __syncthreads();
            if (g >= half && g < 2 * half) {
#pragma unroll
                for (int e = 0; e < E; ++e) join[e][(int)threadIdx.x - half * TPR] = ag[e];
            }
            __syncthreads();
            if (g < half) {
#pragma unroll
                for (int e = 0; e < E; ++e) ag[e] += join[e][threadIdx.x];
            }
        }
    }
    if (g > 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (t + v * TPR) * VEC + i;
            if (c < N) row[c] = ag[v * VEC + i];
        }
}

// Few elements, where a second launch costs more than reading x and dy twice
// (rms_few): the workgroups from row_wgs on sum the columns themselves, which needs
// no row's sum. TPR threads to a row; a column's rows go to 64 groups of 4 lanes.
template <typename T, int TPR, bool RES>
__global__ __launch_bounds__(256) void rms_bwd_few_kernel(RmsArgs a, int row_wgs) {
    constexpr int VEC = VecOf<T>::n, U = 8;
    __shared__ float red[4][4 * VEC];
    const int N = a.N, lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
    const int64_t limit = (a.M - 1) * a.ldx + N, limit_dy = (a.M - 1) * a.lddy + N;
    const T* x = (const T*)a.x;
    const T* dy = (const T*)a.dy;
    if ((int)blockIdx.x >= row_wgs) {
        const int c = (((int)blockIdx.x - row_wgs) * 4 + ((int)threadIdx.x & 3)) * VEC;
        float sum[VEC] = {};
        for (int64_t base = (int)threadIdx.x >> 2; base < a.M; base += 64 * U) {
            u32x4 rx[U], rdy[U];
            float rs[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t m = base + u * 64;
                rx[u] = load_raw<T, 0>(x, m * a.ldx, c, N, limit, m < a.M);
                rdy[u] = load_raw<T, 0>(dy, m * a.lddy, c, N, limit_dy, m < a.M);
                rs[u] = a.rstd[m < a.M ? m : 0];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t m = base + u * 64;
                float n[VEC], d[VEC];
                unpack_raw<T>(rx[u], x, m * a.ldx, c, N, limit, m < a.M, n);
                unpack_raw<T>(rdy[u], dy, m * a.lddy, c, N, limit_dy, m < a.M, d);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[i] = __builtin_fmaf(d[i], n[i] * rs[u], sum[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int l = 4; l < 64; l *= 2) sum[i] += __shfl_xor(sum[i], l);
            if (lane < 4) red[w][lane * VEC + i] = sum[i];
        }
        __syncthreads();
        const int i = (int)threadIdx.x, at = ((int)blockIdx.x - row_wgs) * 4 * VEC + i;
        if (i < 4 * VEC && at < N) store_param(a.dgamma, at, a.pdt, red[0][i] + red[1][i] + red[2][i] + red[3][i]);
        return;
    }
    const int t = (int)threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * (256 / TPR) + (int)threadIdx.x / TPR;
    const bool on = m < a.M;   // for the whole wave
    const float rs = a.rstd[on ? m : 0];
    float s = 0.0f;
#pragma unroll 2
    for (int c = t * VEC; on && c < N; c += TPR * VEC) {
        float n[VEC], d[VEC], gm[VEC];
        load_vec<T>(x, m * a.ldx, c, N, n);
        load_vec<T>(dy, m * a.lddy, c, N, d);
        load_params<VEC>(a.gamma, a.pdt, c, N, gm);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s = __builtin_fmaf(d[i] * (n[i] * rs), gm[i], s);
    }
    s = lanes_sum<64>(s);
    if constexpr (TPR == 256) {
        if (lane == 0) red[w][0] = s;
        __syncthreads();
        s = red[0][0] + red[1][0] + red[2][0] + red[3][0];
    }
    const float c2 = s / (float)N;
#pragma unroll 2
    for (int c = t * VEC; on && c < N; c += TPR * VEC) {
        float n[VEC], d[VEC], gm[VEC], res[VEC], o[VEC];
        load_vec<T>(x, m * a.ldx, c, N, n);
        load_vec<T>(dy, m * a.lddy, c, N, d);
        load_params<VEC>(a.gamma, a.pdt, c, N, gm);
        if constexpr (RES) load_vec<T>((const T*)a.dres, m * a.ldx, c, N, res);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            o[i] = rs * (d[i] * gm[i] - n[i] * rs * c2);
            if constexpr (RES) o[i] += res[i];
        }
        store_vec<T>((T*)a.y, m * a.ldy, c, N, o);
    }
}

// Rows of up to 32,768 columns: a workgroup's 1,024 threads have 128 registers
// each, which hold a row's vectors, packed, and the next one's where those are few
// (AHEAD; of 4 vectors they would spill: 4,096 x 30,000 bfloat16 484 us, without
// 294); the columns' sums live in LDS (128 KB), four floats of a thread at a time so
// that neighbouring lanes meet no bank twice, and gamma is read again for each row.
constexpr int kWideColumns = 32768;

template <typename T, int V, bool RES, int NT>
__global__ __launch_bounds__(kLongThreads) void rms_bwd_wide_kernel(RmsArgs a) {
    constexpr int VEC = VecOf<T>::n, Q = VEC / 4;
    static_assert(V * VEC * kLongThreads <= kWideColumns, "the sums' LDS");
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    extern __shared__ f32x4 sums[];   // [V * Q][kLongThreads]
    __shared__ float red[2][kLongThreads / 64];
    int t = (int)threadIdx.x;
    const int N = a.N;
    const int64_t limit = (a.M - 1) * a.ldx + N, limit_dy = (a.M - 1) * a.lddy + N;
#pragma unroll
    for (int q = 0; q < V * Q; ++q) sums[q * kLongThreads + t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 next_x[V], next_dy[V];
    const auto load = [&](int64_t m) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (t + v * kLongThreads) * VEC;
            next_x[v] = load_raw<T, NT>((const T*)a.x, m * a.ldx, c, N, limit, m < a.M);
            next_dy[v] = load_raw<T, NT>((const T*)a.dy, m * a.lddy, c, N, limit_dy, m < a.M);
        }
    };
    constexpr bool AHEAD = VEC * V <= 16;
    if constexpr (AHEAD) load(blockIdx.x);
    int buf = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, buf ^= 1) {
        u32x4 x[V], dy[V];
        if constexpr (!AHEAD) load(m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = next_x[v];
            dy[v] = next_dy[v];
        }
        if constexpr (AHEAD) load(m + gridDim.x);
        // What depends on a thread's columns only (gamma, addresses, which of them are
        // in the row) would be kept from row to row, in registers that are not there.
        asm volatile("" : "+v"(t));
        const float rs = a.rstd[m];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (t + v * kLongThreads) * VEC;
            float gm[VEC], n[VEC], d[VEC];
            load_params<VEC>(a.gamma, a.pdt, c, N, gm);
            unpack_raw<T>(x[v], (const T*)a.x, m * a.ldx, c, N, limit, true, n);
            unpack_raw<T>(dy[v], (const T*)a.dy, m * a.lddy, c, N, limit_dy, true, d);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s = __builtin_fmaf(d[i] * (n[i] * rs), gm[i], s);
            __builtin_amdgcn_sched_barrier(0);   // one vector's floats at a time
        }
        s = lanes_sum<64>(s);
        if ((t & 63) == 0) red[buf][t >> 6] = s;
        __syncthreads();
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kLongThreads / 64; ++k) s += red[buf][k];
        const float c2 = s / (float)N;
        // nor is there room for the floats of the first walk: unpack them again
        asm volatile("" : "+v"(t));
#pragma unroll
        for (int v = 0; v < V; ++v) asm volatile("" : "+v"(x[v]), "+v"(dy[v]));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (t + v * kLongThreads) * VEC;
            float gm[VEC], n[VEC], d[VEC], res[VEC], o[VEC];
            if constexpr (RES) load_vec<T>((const T*)a.dres, m * a.ldx, c, N, res);
            load_params<VEC>(a.gamma, a.pdt, c, N, gm);
            unpack_raw<T>(x[v], (const T*)a.x, m * a.ldx, c, N, limit, true, n);
            unpack_raw<T>(dy[v], (const T*)a.dy, m * a.lddy, c, N, limit_dy, true, d);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                f32x4 w = sums[(v * Q + q) * kLongThreads + t];
#pragma unroll
                for (int i = 4 * q; i < 4 * q + 4; ++i) {
                    n[i] *= rs;
                    w[i % 4] = __builtin_fmaf(d[i], n[i], w[i % 4]);
                    o[i] = rs * (d[i] * gm[i] - n[i] * c2);
                    if constexpr (RES) o[i] += res[i];
                }
                sums[(v * Q + q) * kLongThreads + t] = w;
            }
            store_vec<T, NT>((T*)a.y, m * a.ldy, c, N, o);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    float* row = a.part + (int64_t)blockIdx.x * a.pitch;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const f32x4 w = sums[(v * Q + q) * kLongThreads + t];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = (t + v * kLongThreads) * VEC + 4 * q + i;
                if (c < N) row[c] = w[i];
            }
        }
}

// Long rows: the row's sum first, then dx and the parameter gradient. Each
// workgroup's partial row lives in the workspace and is added to in place
// (its own columns, thread by thread), the first row's pass writing it.
template <typename T, bool RES>
__global__ __launch_bounds__(kLongThreads) void rms_bwd_long_kernel(RmsArgs a) {
    constexpr int VEC = VecOf<T>::n;
    __shared__ float red[kLongThreads / 64];
    const int N = a.N;
    float* row = a.part + (int64_t)blockIdx.x * a.pitch;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const bool first = m == blockIdx.x;
        const float rs = a.rstd[m];
        float s = 0.0f;
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
            float x[VEC], dy[VEC], gm[VEC];
            load_vec<T>((const T*)a.x, m * a.ldx, c, N, x);
            load_vec<T>((const T*)a.dy, m * a.lddy, c, N, dy);
            load_params<VEC>(a.gamma, a.pdt, c, N, gm);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s = __builtin_fmaf(dy[i] * (x[i] * rs), gm[i], s);
        }
        const float c2 = block_sum(s, red) / (float)N;
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
            float x[VEC], dy[VEC], gm[VEC], res[VEC], o[VEC], sum[VEC];
            load_vec<T>((const T*)a.x, m * a.ldx, c, N, x);
            load_vec<T>((const T*)a.dy, m * a.lddy, c, N, dy);
            load_params<VEC>(a.gamma, a.pdt, c, N, gm);
            if constexpr (RES) load_vec<T>((const T*)a.dres, m * a.ldx, c, N, res);
            if (first) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
            } else {
#pragma unroll
                for (int i = 0; i < VEC; i += 4) load_vec<float>(row, 0, c + i, N, sum + i);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float n = x[i] * rs;
                o[i] = rs * (dy[i] * gm[i] - n * c2);
                if constexpr (RES) o[i] += res[i];
                sum[i] = __builtin_fmaf(dy[i], n, sum[i]);
            }
            store_vec<T>((T*)a.y, m * a.ldy, c, N, o);
#pragma unroll
            for (int i = 0; i < VEC; i += 4) store_vec<float>(row, 0, c + i, N, sum + i);
        }
    }
}

}  // namespace dytb
