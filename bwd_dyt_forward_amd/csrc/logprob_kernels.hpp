// logprob_kernels.hpp - log probabilities of given tokens with entropy and top
// alternatives, and the gradient (gfx950).
//
// With z[j] = scale x[j] over a row x of V logits and a token c:
//
//   lse = log sum_j exp(z[j])        logp = z[c] - lse
//   entropy = lse - sum_j p[j] z[j]  p[j] = exp(z[j] - lse)
//   dx[j] = scale (dlogp ([j = c] - p[j]) - dentropy p[j] (z[j] - lse + entropy))
//
// Bound by HBM: the forward reads a row once, the backward reads it and writes
// its gradient; nothing of a row's length is kept in between. A thread keeps a
// running maximum m of what it has read and, relative to it,
//   s = sum exp(scale (x - m)),  t = sum (x - m) exp(scale (x - m))
// so that entropy = log s - scale t / s, without the cancellation of lse
// against a sum of raw logits; threads, and parts of a row where few rows are
// split over workgroups, are joined the same way. One exponential and about
// seven operations an element keep the vector unit four fifths as long busy as
// HBM.
//
// Alternatives: the best k by (value, lowest index), as one 64-bit key each.
// Neighbouring eight lanes share a line of memory; its maximum (three lane
// exchanges a vector) goes to LDS. The k best lines hold the k best elements,
// so only they are read again. A set's k best keys are found without a sort:
// every thread's best key is ranked among all threads' by counting, the k-th is
// a bound that at least k keys reach and, since the threads beyond it are out,
// at most k threads' keys; those few are then ranked exactly. No step depends
// on the values, so rows of equal or masked logits cost the same.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

constexpr int kLpThreads = 256;
constexpr int kLpMaxTop = 64;
constexpr float kLog2e = 0x1.715476p+0f;

struct LpArgs {
    const void* logits;
    const void* tokens;
    float* logp;          // forward's results; the backward reads entropy, lse
    float* entropy;
    float* lse;
    float* top_logp;      // [T, top]
    int64_t* top_tokens;
    const float* dlogp;   // backward, each or null
    const float* dentropy;
    void* dlogits;
    float* part;          // [T][parts][4]: m, s, t of each part of a row
    uint64_t* part_top;   // [T][parts][top]
    int64_t ld, ldd;
    int64_t T, V;
    int64_t part_len;     // columns of a part
    int32_t parts;
    int32_t top;
    int32_t token_bits;
    int32_t tpr;          // threads of a row, a power of two up to 64, or 256
    float scale;
};

struct Lse {
    float m, s, t;
};

__device__ __forceinline__ Lse lse_none() { return {-3.402823466e+38f, 0.0f, 0.0f}; }

// a and b relative to the larger maximum.
__device__ __forceinline__ Lse lse_join(Lse a, Lse b, float k2) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m - m, db = b.m - m;   // 0 or below; -inf next to an infinite maximum
    const float fa = __builtin_amdgcn_exp2f(da * k2), fb = __builtin_amdgcn_exp2f(db * k2);
    Lse r;
    r.m = m;
    r.s = fa * a.s + fb * b.s;
    // a side that is far below has a factor of 0: so has its share, whatever da
    r.t = fa * (a.t + fmaxf(da, -1e30f) * a.s) + fb * (b.t + fmaxf(db, -1e30f) * b.s);
    return r;
}

template <int CTRL>
__device__ __forceinline__ Lse lse_dpp(Lse v) { return {dpp_mov<CTRL>(v.m), dpp_mov<CTRL>(v.s), dpp_mov<CTRL>(v.t)}; }

__device__ __forceinline__ Lse lse_lane(Lse v, int from) {
    return {__shfl(v.m, from), __shfl(v.s, from), __shfl(v.t, from)};
}

// Joined over aligned groups of `lanes` lanes, in every lane (the same bits:
// the join is symmetric).
__device__ __forceinline__ Lse lse_lanes(Lse v, int lanes, float k2) {
    if (lanes >= 2) v = lse_join(v, lse_dpp<0xB1>(v), k2);
    if (lanes >= 4) v = lse_join(v, lse_dpp<0x4E>(v), k2);
    if (lanes >= 8) v = lse_join(v, lse_dpp<0x141>(v), k2);
    if (lanes >= 16) v = lse_join(v, lse_dpp<0x140>(v), k2);
    const int lane = (int)threadIdx.x & 63;
    if (lanes >= 32) v = lse_join(v, lse_lane(v, lane ^ 16), k2);
    if (lanes >= 64) v = lse_join(v, lse_lane(v, lane ^ 32), k2);
    return v;
}

// One vector's elements (-inf where there are none); returns their maximum.
template <int VEC>
__device__ __forceinline__ float lse_add(Lse& a, const float* x, float k2) {
    float mv = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < VEC; ++i) mv = fmaxf(mv, x[i]);
    if (mv > a.m) {
        const float d = a.m - mv, f = __builtin_amdgcn_exp2f(d * k2);
        a.t = f * (a.t + fmaxf(d, -1e30f) * a.s);
        a.s *= f;
        a.m = mv;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float z = x[i] - a.m;
        const float e = __builtin_amdgcn_exp2f(z * k2);
        a.s += e;
        a.t = __builtin_fmaf(fmaxf(z, -1e30f), e, a.t);   // -inf times an exact 0 would be NaN
    }
    return mv;
}

template <typename T>
__device__ __forceinline__ void logits_at(u32x4 raw, const T* p, int64_t row, int64_t c, int64_t end, float* x) {
    constexpr int VEC = VecOf<T>::n;
    unpack16<T>(raw, x);
    if (c + VEC > end) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = c + i < end ? to_f32(p[row + c + i]) : -INFINITY;
    }
}

// The 16 bytes at column c, or the tensor's first or last ones where there are
// none (see load_raw). A tensor of fewer elements than a vector is not read
// here: its only vector ends past its row and is read one by one.
__device__ const u32x4 kNoLogits = {0, 0, 0, 0};

template <typename T>
__device__ __forceinline__ u32x4 logits_raw(const T* p, int64_t row, int64_t c, int64_t end, int64_t limit) {
    constexpr int VEC = VecOf<T>::n;
    const T* from = p + (c < end ? min(row + c, limit - VEC) : 0);
    return *(const u32x4_m*)(limit < VEC ? (const T*)&kNoLogits : from);
}

template <typename T>
__device__ __forceinline__ void store_part(T* p, int64_t row, int64_t c, int64_t end, const float* v) {
    constexpr int VEC = VecOf<T>::n;
    if (c + VEC <= end) {
        *(u32x4_m*)(p + row + c) = pack16<T>(v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < end) p[row + c + i] = dyt::from_f32<T>(v[i]);
    }
}

// Maximum over aligned groups of eight lanes.
__device__ __forceinline__ float lanes_max8(float v) {
    v = fmaxf(v, dpp_mov<0xB1>(v));
    v = fmaxf(v, dpp_mov<0x4E>(v));
    return fmaxf(v, dpp_mov<0x141>(v));
}

__device__ __forceinline__ void lp_write(const LpArgs& a, int64_t m, Lse v, float x, bool real) {
    const float log_s = logf(v.s);
    const bool none = v.s == 0.0f;   // every logit is -inf
    a.lse[m] = none ? -INFINITY : __builtin_fmaf(v.m, a.scale, log_s);
    a.entropy[m] = none ? 0.0f : log_s - a.scale * v.t / v.s;
    a.logp[m] = !real ? 0.0f : none ? -INFINITY : (x - v.m) * a.scale - log_s;
}

template <typename T>
__device__ __forceinline__ void lp_finish(const LpArgs& a, int64_t m, Lse v) {
    const int64_t c = a.token_bits == 64 ? ((const int64_t*)a.tokens)[m] : (int64_t)((const int32_t*)a.tokens)[m];
    const bool real = c >= 0 && c < a.V;
    lp_write(a, m, v, real ? to_f32(((const T*)a.logits)[m * a.ld + c]) : 0.0f, real);
}

// ------------------------------------------------------------- alternatives
// Order of the values (negative zero counts as zero, NaN as the least), then
// of the places from the first on. No key is 0.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t at) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t o = x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((uint64_t)o << 32) | (0xffffffffu - at);
}

__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return o == 0 ? NAN : __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ uint32_t key_at(uint64_t key) { return 0xffffffffu - (uint32_t)key; }

struct TopShared {
    uint64_t best[kLpThreads];
    uint64_t bound;
    uint32_t count;
};

// The k-th largest of the threads' best keys (0: none), 0 if fewer threads
// have one. All threads call it; clears `count`.
__device__ __forceinline__ uint64_t top_bound(uint64_t mine, int k, TopShared& sh) {
    __syncthreads();   // what was shared before has been read
    sh.best[threadIdx.x] = mine;
    if (threadIdx.x == 0) {
        sh.bound = 0;
        sh.count = 0;
    }
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kLpThreads; ++i) above += sh.best[i] > mine ? 1 : 0;
    if (mine != 0 && above == k - 1) sh.bound = mine;   // keys are unique
    __syncthreads();
    return sh.bound;
}

__device__ __forceinline__ void top_keep(uint64_t key, uint64_t bound, uint64_t* list, TopShared& sh) {
    if (key != 0 && key >= bound) list[atomicAdd(&sh.count, 1u)] = key;
}

// Writes the first k of the list's keys in their order to out(place, key).
template <typename F>
__device__ __forceinline__ void top_rank(const uint64_t* list, int k, const TopShared& sh, F&& out) {
    __syncthreads();
    const int n = (int)sh.count;
    for (int i = (int)threadIdx.x; i < n; i += kLpThreads) {
        const uint64_t key = list[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += list[j] > key ? 1 : 0;
        if (above < k) out(above, key);
    }
}

// --------------------------------------------------------------- forward
// A row to tpr lanes, several rows to a workgroup (V up to a few vectors a
// lane), or a row or a part of one to the workgroup (tpr == 256).
template <typename T, bool TOP>
__global__ __launch_bounds__(kLpThreads) void lp_fwd_kernel(LpArgs a) {
    constexpr int VEC = VecOf<T>::n;
    constexpr int LINE = 8 * VEC;   // elements of a line: eight lanes' vectors
    constexpr int U = 4;
    extern __shared__ uint64_t dyn[];
    const T* p = (const T*)a.logits;
    const float k2 = a.scale * kLog2e;
    const int64_t limit = (a.T - 1) * a.ld + a.V;
    const int tpr = TOP ? kLpThreads : a.tpr;
    const int t = (int)threadIdx.x & (tpr - 1), g = (int)threadIdx.x / tpr;
    const int64_t item = (int64_t)blockIdx.x * (kLpThreads / tpr) + g;   // (row, part)
    const int64_t m = item / a.parts, part = item - m * a.parts;
    const bool on = m < a.T;
    const int64_t row = on ? m * a.ld : 0;
    const int64_t c0 = part * a.part_len, end = on ? min(c0 + a.part_len, a.V) : 0;
    float* line_max = (float*)dyn;
    Lse v = lse_none();
    for (int64_t c = c0 + (int64_t)t * VEC; c - (int64_t)t * VEC < end; c += (int64_t)U * tpr * VEC) {
        u32x4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = logits_raw<T>(p, row, c + (int64_t)u * tpr * VEC, end, limit);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t cu = c + (int64_t)u * tpr * VEC;
            if (cu - (int64_t)t * VEC >= end) continue;   // for all lanes of the row
            float x[VEC];
            logits_at<T>(raw[u], p, row, cu, end, x);
            float mv = lse_add<VEC>(v, x, k2);
            if constexpr (TOP) {
                mv = lanes_max8(mv);
                if ((t & 7) == 0 && cu < end) line_max[(cu - c0) / LINE] = mv;
            }
        }
    }
    v = lse_lanes(v, tpr >= 64 ? 64 : tpr, k2);
    if (tpr == kLpThreads) {
        __shared__ Lse red[kLpThreads / 64];
        if ((t & 63) == 0) red[t >> 6] = v;
        __syncthreads();
        v = lse_join(lse_join(red[0], red[1], k2), lse_join(red[2], red[3], k2), k2);
    }
    if (t == 0 && on) {
        if (a.parts == 1) {
            lp_finish<T>(a, m, v);
        } else {
            float* to = a.part + item * 4;
            to[0] = v.m;
            to[1] = v.s;
            to[2] = v.t;
        }
    }
    if constexpr (TOP) {
        __shared__ TopShared sh;
        __shared__ uint64_t lines[kLpMaxTop];
        const int k = a.top;
        const int n_lines = (int)((end - c0 + LINE - 1) / LINE);
        uint64_t* list = dyn + (a.part_len / LINE + 2) / 2;   // behind the lines' maxima
        // the k best lines: each thread has every 256th
        uint64_t best = 0;
        for (int i = (int)threadIdx.x; i < n_lines; i += kLpThreads) best = max(best, top_key(line_max[i], (uint32_t)i));
        uint64_t bound = top_bound(best, k, sh);
        for (int i = (int)threadIdx.x; i < n_lines; i += kLpThreads)
            top_keep(top_key(line_max[i], (uint32_t)i), bound, list, sh);
        if (threadIdx.x < kLpMaxTop) lines[threadIdx.x] = 0;
        top_rank(list, k, sh, [&](int place, uint64_t key) { lines[place] = key; });
        __syncthreads();
        // their elements, a vector to a lane: 32 lines at a time
        uint64_t key[kLpMaxTop / 32][VEC];
        best = 0;
#pragma unroll
        for (int h = 0; h < kLpMaxTop / 32; ++h) {
            const int at = h * 32 + ((int)threadIdx.x >> 3);
            const uint64_t line = at < k ? lines[at] : 0;
            const int64_t c = c0 + (int64_t)key_at(line) * LINE + ((int)threadIdx.x & 7) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                key[h][i] = line != 0 && c + i < end ? top_key(to_f32(p[row + c + i]), (uint32_t)(c + i)) : 0;
                best = max(best, key[h][i]);
            }
        }
        bound = top_bound(best, k, sh);
#pragma unroll
        for (int h = 0; h < kLpMaxTop / 32; ++h)
#pragma unroll
            for (int i = 0; i < VEC; ++i) top_keep(key[h][i], bound, list, sh);
        top_rank(list, k, sh, [&](int place, uint64_t best_key) {
            if (a.parts > 1) {
                a.part_top[item * k + place] = best_key;
            } else {
                const float log_s = logf(v.s);
                a.top_tokens[m * k + place] = key_at(best_key);
                a.top_logp[m * k + place] = v.s == 0.0f ? -INFINITY : (key_value(best_key) - v.m) * a.scale - log_s;
            }
        });
        // a part of fewer than k elements
        if (a.parts > 1 && (int)threadIdx.x < k && threadIdx.x >= sh.count) a.part_top[item * k + threadIdx.x] = 0;
    }
}

// The parts of a row, up to 256 of them.
template <typename T, bool TOP>
__global__ __launch_bounds__(kLpThreads) void lp_join_kernel(LpArgs a) {
    __shared__ Lse red[kLpThreads / 64];
    const int64_t m = blockIdx.x;
    const int t = (int)threadIdx.x;
    const float k2 = a.scale * kLog2e;
    Lse v = lse_none();
    if (t < a.parts) {
        const float* from = a.part + (m * a.parts + t) * 4;
        v = {from[0], from[1], from[2]};
    }
    v = lse_lanes(v, 64, k2);
    if ((t & 63) == 0) red[t >> 6] = v;
    __syncthreads();
    v = lse_join(lse_join(red[0], red[1], k2), lse_join(red[2], red[3], k2), k2);
    if (t == 0) lp_finish<T>(a, m, v);
    if constexpr (TOP) {
        extern __shared__ uint64_t list[];
        __shared__ TopShared sh;
        const int k = a.top, n = a.parts * k;
        const uint64_t* keys = a.part_top + m * n;
        uint64_t best = 0;
        for (int i = t; i < n; i += kLpThreads) best = max(best, keys[i]);
        const uint64_t bound = top_bound(best, k, sh);
        for (int i = t; i < n; i += kLpThreads) top_keep(keys[i], bound, list, sh);
        const float log_s = logf(v.s);
        top_rank(list, k, sh, [&](int place, uint64_t key) {
            a.top_tokens[m * k + place] = key_at(key);
            a.top_logp[m * k + place] = v.s == 0.0f ? -INFINITY : (key_value(key) - v.m) * a.scale - log_s;
        });
    }
}

// -------------------------------------------------------------- backward
// Items as in the forward. A row without an upstream gradient is not read.
template <typename T>
__global__ __launch_bounds__(kLpThreads) void lp_bwd_kernel(LpArgs a) {
    constexpr int VEC = VecOf<T>::n;
    constexpr int U = 4;
    const T* p = (const T*)a.logits;
    T* out = (T*)a.dlogits;
    const int64_t limit = (a.T - 1) * a.ld + a.V;
    const int tpr = a.tpr;
    const int t = (int)threadIdx.x & (tpr - 1), g = (int)threadIdx.x / tpr;
    const int64_t item = (int64_t)blockIdx.x * (kLpThreads / tpr) + g;
    const int64_t m = item / a.parts, part = item - m * a.parts;
    if (m >= a.T) return;
    const int64_t row = m * a.ld, to = m * a.ldd;
    const int64_t c0 = part * a.part_len, end = min(c0 + a.part_len, a.V);
    const int64_t token = a.token_bits == 64 ? ((const int64_t*)a.tokens)[m] : (int64_t)((const int32_t*)a.tokens)[m];
    const bool real = token >= 0 && token < a.V;
    const float lse = a.lse[m], h = a.entropy[m];
    const float up = real && a.dlogp ? a.dlogp[m] : 0.0f;
    const float ue = a.dentropy ? a.dentropy[m] : 0.0f;
    if ((up == 0.0f && ue == 0.0f) || lse == -INFINITY) {
        const float zero[VEC] = {};
        for (int64_t c = c0 + (int64_t)t * VEC; c < end; c += (int64_t)tpr * VEC) store_part<T>(out, to, c, end, zero);
        return;
    }
    // dx = -scale p (up + ue (z - lse + h)), and scale up more at the token
    const float base = -a.scale * (up + ue * h), slope = -a.scale * ue;
    for (int64_t c = c0 + (int64_t)t * VEC; c < end; c += (int64_t)U * tpr * VEC) {
        u32x4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = logits_raw<T>(p, row, c + (int64_t)u * tpr * VEC, end, limit);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t cu = c + (int64_t)u * tpr * VEC;
            if (cu >= end) continue;
            float x[VEC];
            logits_at<T>(raw[u], p, row, cu, end, x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float z = __builtin_fmaf(x[i], a.scale, -lse);
                const float e = __builtin_amdgcn_exp2f(z * kLog2e);
                x[i] = e * __builtin_fmaf(fmaxf(z, -1e30f), slope, base);
            }
            if (real && (uint64_t)(token - cu) < (uint64_t)VEC) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (token == cu + i) x[i] = __builtin_fmaf(a.scale, up, x[i]);
            }
            store_part<T>(out, to, cu, end, x);
        }
    }
}

}  // namespace dytb
