// ln_kernels.hpp - layer norm, forward and backward (gfx950).
//
// Both directions are bound by HBM traffic: the forward reads x (and the
// residual) once and writes y (and h), the backward reads x and dy (and
// dres) once and writes dx. A row therefore stays in registers between its
// statistics and its use: TPR threads hold a row as V vectors of 16 bytes
// each. TPR is the smallest power of two that covers the row up to a wave
// (several rows per wave, sums by lane exchange, no barrier); wider rows
// take a workgroup each and one barrier per reduction.
//
// The variance is the mean of squared distances from the mean, never
// E[x^2] - mean^2: within a wave a second pass over the registers, across
// the waves of a row by merging (count, mean, M2) triples,
//   mean = sum n_w mean_w / N,  M2 = sum M2_w + sum n_w (mean_w - mean)^2.
//
// The backward's parameter gradients are sums over rows: each thread adds up
// its own columns over the rows its workgroup walks, the workgroup's row
// groups are joined through LDS in group order, and one float32 row
// [dgamma | dbeta] per workgroup goes to the workspace; a second kernel sums
// those rows in a fixed order. No atomics.
//
// Measured (traced, box to box): 32,768 x 4,096 bf16 forward 98-101 us (5.4 TB/s),
// with the residual 188-212 us (5.1-5.7), backward 118 (6.8) and with the
// residual 171-185 us (5.8-6.3); 4,194,304 x 32 f16 forward 89-90 us (6.0); 100,003 x
// 255 f32, whose rows are no whole vectors, 35 and 50 us (5.8 and 6.1). A 1,024 x 64
// problem takes 3-4 us a kernel. The backward's rows of sixteen waves spill: 8,192
// x 16,384 bf16 168 us (4.8 TB/s) and with the residual 435 us (2.5), f32 268 (6.0)
// and 563 us (3.8). Rows past 16,384 columns, 4,096 x 33,000 bf16: forward 542 us (1.0
// TB/s), backward 1,774 us (0.5): they are walked again for every sum, gamma is
// read element by element and the column sums are kept in memory.
#pragma once

#include "block_common.hpp"

namespace dytb {

struct LnArgs {
    const void* x;        // forward: x; backward: x or h
    const void* r;        // forward: residual or null
    void* h;              // forward: x + r, or null
    void* y;              // forward: y; backward: dx
    const void* dy;       // backward
    const void* dres;     // backward: residual gradient or null
    const void* gamma;
    const void* beta;
    float* mean;
    float* rstd;
    float* part;          // backward: partial rows
    int64_t ldx, ldy, lddy;
    int64_t M;
    int32_t N;
    int32_t pdt;
    float eps;
    int64_t pitch;        // backward: floats between partial rows
    int32_t traffic;      // cache hints, see ln_traffic
};

// The 16 bytes that hold elements [c, c + VEC) of the row that starts at
// element `row`, without a branch: a load behind one would make every later
// wait of the loop a wait for all loads. Lanes without elements (past the
// row, or `on` false) read the tensor's first bytes; where the 16 bytes would
// end past the tensor's last element (`limit`), the last 16 bytes are read.
// The tensor has at least VEC elements.
template <typename T, int NT>
__device__ __forceinline__ u32x4 load_raw(const T* p, int64_t row, int c, int N, int64_t limit, bool on) {
    constexpr int VEC = VecOf<T>::n;
    const int64_t at = min(row + c, limit - VEC);
    const u32x4_m* from = (const u32x4_m*)(p + (on && c < N ? at : 0));
    if constexpr (NT >= 2) return __builtin_nontemporal_load(from);
    else return *from;
}

// Those elements as float32, zeros past N: clears what belongs to the next
// row (or the pitch's gap), and reads the tensor's last elements one by one
// where load_raw had to stay back.
template <typename T>
__device__ __forceinline__ void unpack_raw(u32x4 w, const T* p, int64_t row, int c, int N, int64_t limit, bool on,
                                           float* out) {
    constexpr int VEC = VecOf<T>::n;
    unpack16<T>(w, out);
    if (N % VEC == 0) {
        const bool in = on && c < N;
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[i] = in ? out[i] : 0.0f;
        return;
    }
    if (on && c < N && row + c + VEC > limit) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < N) out[i] = to_f32(p[row + c + i]);
    }
    const int n = on ? N - c : 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = i < n ? out[i] : 0.0f;
}

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, int64_t row, int c, int N, float* out) {
    constexpr int VEC = VecOf<T>::n;
    if (c + VEC <= N) {
        unpack16<T>(*(const u32x4_m*)(p + row + c), out);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[i] = c + i < N ? to_f32(p[row + c + i]) : 0.0f;
    }
}

// Parameters of the E columns of a thread (0 past N), 16 bytes at a time: every
// workgroup reads them before its first row (2,048 rows of 4,096 take 8 us, and
// 32 with loads of single elements).
template <typename P, int V, int VEC, int TPR>
__device__ __forceinline__ void load_columns_of(const P* p, int t, int N, float* out) {
    constexpr int PV = VecOf<P>::n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (t + v * TPR) * VEC;
        float* o = out + v * VEC;
        if (VEC >= PV && c + VEC <= N) {
#pragma unroll
            for (int i = 0; i < VEC; i += PV) unpack16<P>(*(const u32x4_m*)(p + c + i), o + i);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = c + i < N ? to_f32(p[c + i]) : 0.0f;
        }
    }
}

template <int V, int VEC, int TPR>
__device__ __forceinline__ void load_columns(const void* p, int dt, int t, int N, float* out) {
    if (dt == DYT_F32) load_columns_of<float, V, VEC, TPR>((const float*)p, t, N, out);
    else if (dt == DYT_BF16) load_columns_of<bf16_t, V, VEC, TPR>((const bf16_t*)p, t, N, out);
    else load_columns_of<f16_t, V, VEC, TPR>((const f16_t*)p, t, N, out);
}

template <typename T, int NT = 0>
__device__ __forceinline__ void store_vec(T* p, int64_t row, int c, int N, const float* v) {
    constexpr int VEC = VecOf<T>::n;
    if (c + VEC <= N) {
        u32x4_m* to = (u32x4_m*)(p + row + c);
        if constexpr (NT >= 1) __builtin_nontemporal_store((u32x4_m)pack16<T>(v), to);
        else *to = pack16<T>(v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < N) p[row + c + i] = dyt::from_f32<T>(v[i]);
    }
}

__device__ __forceinline__ float inv_sqrt(float v) {
    // One Newton step on the hardware estimate, which takes a subnormal for 0: small
    // values are scaled, by powers of two.
    const bool small = v < 0x1p-100f;
    if (small) v *= 0x1p60f;
    const float y = __builtin_amdgcn_rsqf(v);
    const float e = __builtin_fmaf(-v * y, y, 1.0f);
    const float z = __builtin_fmaf(0.5f * y, e, y);
    const float r = (v > 0.0f && v < INFINITY) ? z : y;   // 0 and inf keep the estimate's inf and 0
    return small ? r * 0x1p30f : r;
}

// TPR threads per row, TH per workgroup. NT: 1 nontemporal stores, 2 loads as
// well (ln_traffic).
constexpr int ln_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int TPR, int TH = ln_threads(TPR)> struct LnShape {
    static constexpr int threads = TH;
    static constexpr int groups = threads / TPR;                 // rows side by side
    static constexpr int waves = TPR > 64 ? TPR / 64 : 1;        // waves of a row
    static constexpr int L = TPR > 64 ? 64 : TPR;
};

template <typename T, int TPR, int V, int U, bool RES, int NT>
__global__ __launch_bounds__(LnShape<TPR>::threads) void ln_fwd_kernel(LnArgs a) {
    using S = LnShape<TPR>;
    constexpr int VEC = VecOf<T>::n;
    constexpr int E = V * VEC;
    const int t = (int)threadIdx.x % TPR;
    const int g = (int)threadIdx.x / TPR;
    const int N = a.N;
    float gm[E], bt[E];
    load_columns<V, VEC, TPR>(a.gamma, a.pdt, t, N, gm);
    load_columns<V, VEC, TPR>(a.beta, a.pdt, t, N, bt);
    const float inv_n = 1.0f / (float)N;
    const int64_t limit = (a.M - 1) * a.ldx + N;
    const int64_t step = (int64_t)gridDim.x * S::groups * U;
    const T* xp = (const T*)a.x;
    // rows of one iteration lie U apart by the row groups: neighbours in memory
    for (int64_t base = (int64_t)blockIdx.x * S::groups * U; base < a.M; base += step) {
        float x[U][E];
        float mean[U], m2[U];
        u32x4 raw[U][V], rres[U][RES ? V : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (t + v * TPR) * VEC;
                raw[u][v] = load_raw<T, NT>(xp, m * a.ldx, c, N, limit, m < a.M);
                if constexpr (RES) rres[u][v] = load_raw<T, NT>((const T*)a.r, m * a.ldx, c, N, limit, m < a.M);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (t + v * TPR) * VEC;
                unpack_raw<T>(raw[u][v], xp, m * a.ldx, c, N, limit, m < a.M, &x[u][v * VEC]);
                if constexpr (RES) {
                    float r[VEC];
                    unpack_raw<T>(rres[u][v], (const T*)a.r, m * a.ldx, c, N, limit, m < a.M, r);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) r[i] += x[u][v * VEC + i];
                    if (m < a.M) store_vec<T, NT>((T*)a.h, m * a.ldx, c, N, r);
                    // the layer's input is h as stored
                    unpack16<T>(pack16<T>(r), &x[u][v * VEC]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) s += x[u][e];
            s = lanes_sum<S::L>(s);
            if constexpr (S::waves == 1) {
                mean[u] = s / (float)N;   // not times 1 / N: a row of one value gets it as its mean
            } else {
                // columns of this wave
                int cnt = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int lo = ((t & ~63) + v * TPR) * VEC;
                    cnt += min(max(N - lo, 0), 64 * VEC);
                }
                mean[u] = cnt ? s / (float)cnt : 0.0f;
            }
            float q = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = x[u][v * VEC + i] - mean[u];
                    q += ((t + v * TPR) * VEC + i < N) ? d * d : 0.0f;
                }
            m2[u] = lanes_sum<S::L>(q);
        }
        if constexpr (S::waves > 1) {
            static_assert(S::groups == 1, "a row of several waves has the workgroup to itself");
            __shared__ float red[2][U][S::waves][2];
            const int w = t >> 6;
            const int buf = (int)((base / step) & 1);   // the next rows' triples go to the other half
            if ((t & 63) == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    red[buf][u][w][0] = mean[u];
                    red[buf][u][w][1] = m2[u];
                }
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float cw[S::waves], mt = 0.0f, q = 0.0f;
#pragma unroll
                for (int k = 0; k < S::waves; ++k) {
                    int cnt = 0;
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        cnt += min(max(N - (k * 64 + v * TPR) * VEC, 0), 64 * VEC);
                    cw[k] = (float)cnt;
                    mt += cw[k] * red[buf][u][k][0];
                }
                mt /= (float)N;
#pragma unroll
                for (int k = 0; k < S::waves; ++k) {
                    const float d = red[buf][u][k][0] - mt;
                    q += red[buf][u][k][1] + cw[k] * d * d;
                }
                mean[u] = mt;
                m2[u] = q;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
            if (m >= a.M) continue;
            const float rs = inv_sqrt(m2[u] * inv_n + a.eps);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    y[i] = __builtin_fmaf((x[u][e] - mean[u]) * rs, gm[e], bt[e]);
                }
                store_vec<T, NT>((T*)a.y, m * a.ldy, (t + v * TPR) * VEC, N, y);
            }
            if (t == 0) {
                a.mean[m] = mean[u];
                a.rstd[m] = rs;
            }
        }
    }
}

// Rows longer than 1,024 threads hold in registers: a workgroup per row and
// three walks over it, the second and third of which find the row in the
// last-level caches.
constexpr int kLongThreads = 1024;

__device__ __forceinline__ float block_sum(float v, float* red) {
    v = lanes_sum<64>(v);
    __syncthreads();   // the previous sum has been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kLongThreads / 64; ++k) s += red[k];
    return s;
}

template <typename T, bool RES>
__global__ __launch_bounds__(kLongThreads) void ln_fwd_long_kernel(LnArgs a) {
    constexpr int VEC = VecOf<T>::n;
    __shared__ float red[kLongThreads / 64];
    const int N = a.N;
    const float inv_n = 1.0f / (float)N;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const T* src = (const T*)a.x;
        float s = 0.0f;
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
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
            for (int i = 0; i < VEC; ++i) s += x[i];
        }
        if constexpr (RES) src = (const T*)a.h;   // each thread reads back its own stores
        const float mean = block_sum(s, red) / (float)N;
        float q = 0.0f;
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
            float x[VEC];
            load_vec<T>(src, m * a.ldx, c, N, x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = x[i] - mean;
                q += (c + i < N) ? d * d : 0.0f;
            }
        }
        const float rs = inv_sqrt(block_sum(q, red) * inv_n + a.eps);
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
            float x[VEC];
            load_vec<T>(src, m * a.ldx, c, N, x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = min(c + i, N - 1);
                x[i] = __builtin_fmaf((x[i] - mean) * rs, load_param(a.gamma, k, a.pdt),
                                      load_param(a.beta, k, a.pdt));
            }
            store_vec<T>((T*)a.y, m * a.ldy, c, N, x);
        }
        if (threadIdx.x == 0) {
            a.mean[m] = mean;
            a.rstd[m] = rs;
        }
    }
}

// U row groups at a time, and (AHEAD) the next U rows' vectors are loaded,
// still packed, before the current ones are reduced, so that a workgroup's
// loads do not wait for its sums. Workgroups of 1,024 threads have only 128
// registers a lane, spill even so (with the residual 194 of them in the 16-bit
// types, 12 without) and go without.
template <typename T, int TPR, int TH, int V, int U, bool RES, int NT, bool AHEAD = (TPR < 1024)>
__global__ __launch_bounds__(TH) void ln_bwd_kernel(LnArgs a) {
    using S = LnShape<TPR, TH>;
    constexpr int VEC = VecOf<T>::n;
    constexpr int E = V * VEC;
    const int t = (int)threadIdx.x % TPR;
    const int g = (int)threadIdx.x / TPR;
    const int N = a.N;
    float gm[E], ag[E], ab[E];
    load_columns<V, VEC, TPR>(a.gamma, a.pdt, t, N, gm);
#pragma unroll
    for (int e = 0; e < E; ++e) ag[e] = ab[e] = 0.0f;
    const float inv_n = 1.0f / (float)N;
    const int64_t limit = (a.M - 1) * a.ldx + N;
    const int64_t limit_dy = (a.M - 1) * a.lddy + N;
    const int64_t step = (int64_t)gridDim.x * S::groups * U;
    struct Raw {
        u32x4 x[V], dy[V], res[RES ? V : 1];
        float mean, rs;
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
        w.mean = a.mean[on ? m : 0];
        w.rs = a.rstd[on ? m : 0];
    };
    Raw next[U];
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
        float n[U][E], dy[U][E], s1[U], s2[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t m = base + u * S::groups + g;
                const int c = (t + v * TPR) * VEC;
                unpack_raw<T>(now[u].x[v], (const T*)a.x, m * a.ldx, c, N, limit, m < a.M, &n[u][v * VEC]);
                unpack_raw<T>(now[u].dy[v], (const T*)a.dy, m * a.lddy, c, N, limit_dy, m < a.M, &dy[u][v * VEC]);
            }
            s1[u] = s2[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // past the row's end x is 0, not the mean: dy = gamma = 0 there
                // keeps the sums clean and the columns are never stored
                const float x = (n[u][e] - now[u].mean) * now[u].rs;
                const float d = dy[u][e] * gm[e];
                ag[e] = __builtin_fmaf(dy[u][e], x, ag[e]);
                ab[e] += dy[u][e];
                s1[u] += d;
                s2[u] = __builtin_fmaf(d, x, s2[u]);
                n[u][e] = x;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s1[u] = lanes_sum<S::L>(s1[u]);
            s2[u] = lanes_sum<S::L>(s2[u]);
        }
        if constexpr (S::waves > 1) {
            __shared__ float red[2][U][S::groups][S::waves][2];
            if ((t & 63) == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    red[buf][u][g][t >> 6][0] = s1[u];
                    red[buf][u][g][t >> 6][1] = s2[u];
                }
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s1[u] = s2[u] = 0.0f;
#pragma unroll
                for (int k = 0; k < S::waves; ++k) {
                    s1[u] += red[buf][u][g][k][0];
                    s2[u] += red[buf][u][g][k][1];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * S::groups + g;
            if (m >= a.M) continue;
            const float c1 = s1[u] * inv_n, c2 = s2[u] * inv_n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float o[VEC], res[VEC];
                const int c = (t + v * TPR) * VEC;
                if constexpr (RES) unpack_raw<T>(now[u].res[v], (const T*)a.dres, m * a.ldx, c, N, limit, true, res);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    const float d = dy[u][e] * gm[e];
                    o[i] = now[u].rs * (d - c1 - n[u][e] * c2);
                    if constexpr (RES) o[i] += res[i];
                }
                store_vec<T, NT>((T*)a.y, m * a.ldy, c, N, o);
            }
        }
    }
    float* row = a.part + (int64_t)blockIdx.x * a.pitch;
    if constexpr (S::groups > 1) {
        // join the row groups, the upper half onto the lower one, one
        // gradient after the other through the same LDS
        __shared__ float join[E][TH / 2];
#pragma unroll
        for (int half = S::groups / 2; half > 0; half /= 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float* sum = k ? ab : ag;
                __syncthreads();
                if (g >= half && g < 2 * half) {
#pragma unroll
                    for (int e = 0; e < E; ++e) join[e][(int)threadIdx.x - half * TPR] = sum[e];
                }
                __syncthreads();
                if (g < half) {
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[e] += join[e][threadIdx.x];
                }
            }
        }
    }
    if (g > 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (t + v * TPR) * VEC + i;
            if (c < N) {
                row[c] = ag[v * VEC + i];
                row[N + c] = ab[v * VEC + i];
            }
        }
}

// Long rows: the row sums first, then dx and the parameter gradients. Each
// workgroup's partial row lives in the workspace and is added to in place
// (its own columns, thread by thread), the first row's pass writing it.
template <typename T, bool RES>
__global__ __launch_bounds__(kLongThreads) void ln_bwd_long_kernel(LnArgs a) {
    constexpr int VEC = VecOf<T>::n;
    __shared__ float red[kLongThreads / 64];
    const int N = a.N;
    const float inv_n = 1.0f / (float)N;
    float* row = a.part + (int64_t)blockIdx.x * a.pitch;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const bool first = m == blockIdx.x;
        const float mean = a.mean[m], rs = a.rstd[m];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
            float x[VEC], dy[VEC];
            load_vec<T>((const T*)a.x, m * a.ldx, c, N, x);
            load_vec<T>((const T*)a.dy, m * a.lddy, c, N, dy);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = min(c + i, N - 1);
                const float d = dy[i] * load_param(a.gamma, k, a.pdt);   // dy = 0 past the end
                s1 += d;
                s2 += d * ((x[i] - mean) * rs);
            }
        }
        const float c1 = block_sum(s1, red) * inv_n;
        const float c2 = block_sum(s2, red) * inv_n;
        for (int c = (int)threadIdx.x * VEC; c < N; c += kLongThreads * VEC) {
            float x[VEC], dy[VEC], res[VEC], o[VEC];
            load_vec<T>((const T*)a.x, m * a.ldx, c, N, x);
            load_vec<T>((const T*)a.dy, m * a.lddy, c, N, dy);
            if constexpr (RES) load_vec<T>((const T*)a.dres, m * a.ldx, c, N, res);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (c + i >= N) continue;
                const float n = (x[i] - mean) * rs;
                o[i] = rs * (dy[i] * load_param(a.gamma, c + i, a.pdt) - c1 - n * c2);
                if constexpr (RES) o[i] += res[i];
                row[c + i] = (first ? 0.0f : row[c + i]) + dy[i] * n;
                row[N + c + i] = (first ? 0.0f : row[N + c + i]) + dy[i];
            }
            store_vec<T>((T*)a.y, m * a.ldy, c, N, o);
        }
    }
}

}  // namespace dytb
