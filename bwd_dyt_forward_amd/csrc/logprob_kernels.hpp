// logprob_kernels.hpp - log probabilities of given tokens with entropy and top
// alternatives, and the gradient (gfx950).
//
// With z[j] = scale x[j] over a row x of V logits and a token c:
//
//   lse = log sum_j exp(z[j])        logp = z[c] - lse
//   entropy = lse - sum_j p[j] z[j]  p[j] = exp(z[j] - lse)
//   dx[j] = scale (dlogp ([j = c] - p[j]) - dentropy p[j] (z[j] - lse + entropy))
//
// The forward reads a row once, the backward reads it and writes its gradient;
// nothing of a row's length is kept in between. A thread works in powers of two:
// with y = k x, k = scale log2(e), it keeps a running maximum m of the y it has
// read and, relative to it, s = sum 2^(y - m), t = sum (y - m) 2^(y - m), so that
//   lse = (m + log2 s) ln 2        entropy = (log2 s - t / s) ln 2
// without the cancellation of lse against a sum of raw logits; threads, and parts
// of a row where few rows are split over workgroups, are joined the same way.
//
// The backward is bound by HBM. In the forward the vector unit is as busy as
// HBM: one exponential (a quarter of the rate) and six other operations an
// element. Hence y - m in one fused operation, maxima of three, 32-bit places, one
// change of the maximum for 16 elements, and checks for a row's ends and for masked
// places' -inf times 0 outside of the vectors that hold none.
//
// Alternatives: the best k by (value, lowest index), as one 64-bit key each.
// Neighbouring eight lanes share a line of memory; its maximum (three lane
// exchanges a vector) goes to LDS. The k best lines hold the k best elements,
// so only they are read again. The k best of many keys are found without a sort:
// the best keys of 64 sets are ranked among each other by counting, the k-th is
// a bound that at least k keys reach and, since the sets beyond it are out, at
// most the keys of k sets; those few are then ranked exactly. No step depends
// on the values, so rows of equal or masked logits cost the same.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

constexpr int kLpThreads = 256;
constexpr int kLpMaxTop = 64;
constexpr int kLpBwdVecs = 4;   // vectors of a thread in the backward: no loop
constexpr float kLog2e = 0x1.715476p+0f;

struct LpArgs {
    const void* logits;
    const void* tokens;
    float* logp;          // forward's results; the backward reads entropy, lse
    float* entropy;
    float* lse;
    float* norm;          // [T, 3] or null: m, log2 s and the entropy, for the backward
    float* top_logp;      // [T, top]
    int64_t* top_tokens;
    const float* dlogp;   // backward, each or null
    const float* dentropy;
    void* dlogits;
    float* part;          // [T][parts][4]: m, s, t of each part of a row
    uint64_t* part_top;   // [T][parts][top]
    int64_t ld, ldd;
    int64_t T, V;
    int64_t part_len;     // places of a part, see RowPart
    int32_t parts;
    int32_t top;
    int32_t token_bits;
    int32_t tpr;          // threads of a row, a power of two up to 64, or 256
    int32_t stream;       // 1: past the last-level cache: nontemporal loads of the forward
    float scale;
    double to_ln;         // scale / k, see lp_fwd_kernel: ln 2 but for the rounding of k
};

struct Lse {
    float m, s, t;
};

// The least maximum is finite: a y of -inf (a logit of -inf, or below -2.3e38 /
// scale) then has an exponential of 0.
__device__ __forceinline__ Lse lse_none() { return {-3.402823466e+38f, 0.0f, 0.0f}; }

// (fmaxf would first bring each operand into its canonical form.)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Over aligned groups of `lanes` lanes, in every lane: the maximum, then the
// sums relative to it.
__device__ __forceinline__ float lp_max(float v, int lanes) {
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

__device__ __forceinline__ float lp_sum(float v, int lanes) {
    if (lanes >= 2) v += dpp_mov<0xB1>(v);
    if (lanes >= 4) v += dpp_mov<0x4E>(v);
    if (lanes >= 8) v += dpp_mov<0x141>(v);
    if (lanes >= 16) v += dpp_mov<0x140>(v);
    if (lanes >= 32) v = swap16_other_sum(v);
    if (lanes >= 64) v = swap32_other_sum(v);
    return v;
}

__device__ __forceinline__ Lse lse_lanes(Lse v, int lanes) {
    const float m = lp_max(v.m, lanes), d = v.m - m;   // 0 or below; NaN next to an infinite maximum
    const float f = __builtin_amdgcn_exp2f(d);
    // a lane that is far below has a factor of 0: so has its share, whatever d
    return {m, lp_sum(f * v.s, lanes), lp_sum(f * (v.t + fmaxf(d, -1e30f) * v.s), lanes)};
}

// Over a workgroup, in every thread.
__device__ __forceinline__ Lse lse_group(Lse v, Lse* waves) {
    v = lse_lanes(v, 64);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
    __syncthreads();
    return lse_lanes(waves[threadIdx.x & 3], 4);
}

template <int VEC>
__device__ __forceinline__ float vec_max(const float* x) {
    if constexpr (VEC == 8) return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
    else return max3(max3(x[0], x[1], x[2]), x[3], x[3]);
}

// N elements (-inf where there are none), `most` their maximum.
template <int N>
__device__ __forceinline__ void lse_add(Lse& a, const float* x, float most, float k2) {
    const float m = most * k2;
    if (m > a.m) {
        const float d = a.m - m, f = __builtin_amdgcn_exp2f(d);
        a.t = f * (a.t + fmaxf(d, -1e30f) * a.s);
        a.s *= f;
        a.m = m;
    }
    float t = 0.0f, z[N], e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        z[i] = __builtin_fmaf(x[i], k2, -a.m);
        e[i] = __builtin_amdgcn_exp2f(z[i]);
        a.s += e[i];
        t = __builtin_fmaf(z[i], e[i], t);
    }
    if (t != t) {   // -inf times an exact 0: once more, with the maximum that an element would cost each time
        t = 0.0f;
        asm volatile("" : "+v"(t));   // stays a branch
#pragma unroll
        for (int i = 0; i < N; ++i) t = __builtin_fmaf(fmaxf(z[i], -1e30f), e[i], t);
    }
    a.t += t;
}

// A part of a row on the 16-byte grid: its vectors are the aligned 16 bytes of
// memory, whatever the row's first address, so that rows of odd length are read
// like others (50,257 bfloat16 logits: unaligned vectors cost a tenth). Place e
// is column e - skew, of the row's V + skew places. The vectors at places lo to
// hi lie within the row; the others, at its ends, are read element by element.
template <typename T>
struct RowPart {
    static constexpr int VEC = VecOf<T>::n;
    const T* p;           // place 0 (before the row by `skew` elements)
    const T* from;        // what vectors are loaded from: p, or 16 bytes of nothing where there is no whole one
    int V, skew;
    int first, end;       // places of the part
    int lo, hi, most;     // whole vectors' places, and the last one that is loaded

    __device__ __forceinline__ RowPart(const T* logits, uint32_t m, uint32_t part, const LpArgs& a) {
        static __device__ const u32x4 none = {0, 0, 0, 0};
        const bool on = m < a.T;
        const T* row = logits + (on ? (int64_t)m * a.ld : 0);
        V = (int)a.V;
        skew = (int)(((uintptr_t)row / sizeof(T)) % VEC);
        p = row - skew;
        first = (int)part * (int)a.part_len;
        end = on ? min(first + (int)a.part_len, V + skew) : first;
        lo = max(first, skew ? VEC : 0);
        hi = min(end, (V + skew) / VEC * VEC);
        const bool some = lo < hi;
        from = some ? p : (const T*)&none;
        most = some ? hi - VEC : 0;
    }

    // The vector at e; another one where that is not whole.
    template <bool NT>
    __device__ __forceinline__ u32x4 load(int e) const {
        const u32x4* at = (const u32x4*)(from + min(max(e, min(lo, most)), most));
        if constexpr (NT) return __builtin_nontemporal_load(at);
        else return *at;
    }

    // The elements of a vector that is not whole as float32, -inf where there are none.
    __device__ __forceinline__ void elements(int e, float* x) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = in_row(e, i) ? to_f32(p[e + i]) : -INFINITY;
    }

    __device__ __forceinline__ bool in_row(int e, int i) const { return e < end && e + i >= skew && e + i < V + skew; }
    __device__ __forceinline__ bool whole(int e) const { return e >= lo && e < hi; }
};

// Maximum over aligned groups of eight lanes.
__device__ __forceinline__ float lanes_max8(float v) {
    v = fmaxf(v, dpp_mov<0xB1>(v));
    v = fmaxf(v, dpp_mov<0x4E>(v));
    return fmaxf(v, dpp_mov<0x141>(v));
}

constexpr float kLn2 = 0x1.62e43p-1f;

// A row's log sum, m + log2 s. In two float32 numbers it has their digits; added up,
// and brought to natural logarithms, it has them in 64 bits only: one lse of 15 rounds
// to 2^-21, and with it log p. (A few operations a row.) `none`: every logit is -inf.
struct RowSum {
    double log2_sum;
    float log2_s, k2;
    bool none;

    __device__ __forceinline__ RowSum(Lse v, float k2) : k2(k2), none(v.s == 0.0f) {
        // s = f 2^e with f in [1/2, 1): the error of log2 f does not grow with s
        const float e = (float)__builtin_amdgcn_frexp_expf(v.s), f = log2f(__builtin_amdgcn_frexp_mantf(v.s));
        log2_s = none ? -INFINITY : e + f;
        log2_sum = (double)v.m + ((double)e + (double)f);
    }

    // log p of a logit; to_ln: scale / k2.
    __device__ __forceinline__ float log_p(float x, double to_ln) const {
        // (what is masked in float32 would be a number in 64 bits)
        if (none || x * k2 == -INFINITY) return -INFINITY;
        return (float)(((double)x * (double)k2 - log2_sum) * to_ln);
    }
};

__device__ __forceinline__ void lp_write(const LpArgs& a, int64_t m, Lse v, float x, bool real, float k2) {
    const RowSum r(v, k2);
    a.lse[m] = r.none ? -INFINITY : (float)(r.log2_sum * a.to_ln);
    const float entropy = r.none ? 0.0f : (r.log2_s - v.t / v.s) * kLn2;
    a.entropy[m] = entropy;
    if (a.norm) {
        a.norm[3 * m] = v.m;
        a.norm[3 * m + 1] = r.log2_s;   // -inf for none
        a.norm[3 * m + 2] = entropy;
    }
    a.logp[m] = real ? r.log_p(x, a.to_ln) : 0.0f;
}

// The row's token, whether there is one, and its logit.
template <typename T>
struct RowToken {
    float x = 0.0f;
    bool real = false;

    __device__ __forceinline__ RowToken(const LpArgs& a, int64_t m) {
        if (m >= a.T) return;
        const int64_t c = a.token_bits == 64 ? ((const int64_t*)a.tokens)[m] : (int64_t)((const int32_t*)a.tokens)[m];
        real = c >= 0 && c < a.V;
        x = to_f32(((const T*)a.logits)[m * a.ld + (real ? c : 0)]);
    }
};

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

constexpr int kTopSets = 64;   // of four neighbouring threads each

struct TopShared {
    uint64_t best[kTopSets];
    uint64_t bound;
    uint32_t count;
};

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_key(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xf, 0xf, true);
    return ((uint64_t)hi << 32) | lo;
}

// The k-th largest of the sets' best keys (0: none), 0 if fewer sets have one.
// All threads call it; clears `count`. (One wave ranks 64 sets: all waves
// ranking 256 threads took 13 of a row's 18 us.)
__device__ __forceinline__ uint64_t top_bound(uint64_t mine, int k, TopShared& sh) {
    static_assert(kLpMaxTop <= kTopSets, "k sets are needed for a bound that k keys reach");
    mine = max(mine, dpp_key<0xB1>(mine));
    mine = max(mine, dpp_key<0x4E>(mine));
    __syncthreads();   // what was shared before has been read
    if ((threadIdx.x & 3) == 0) sh.best[threadIdx.x >> 2] = mine;
    if (threadIdx.x == 0) {
        sh.bound = 0;
        sh.count = 0;
    }
    __syncthreads();
    if (threadIdx.x < kTopSets) {
        const uint64_t key = sh.best[threadIdx.x];
        int above = 0;
#pragma unroll 16
        for (int i = 0; i < kTopSets; ++i) above += sh.best[i] > key ? 1 : 0;
        if (key != 0 && above == k - 1) sh.bound = key;   // keys are unique
    }
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
#pragma unroll 8
        for (int j = 0; j < n; ++j) above += list[j] > key ? 1 : 0;
        if (above < k) out(above, key);
    }
}

// --------------------------------------------------------------- forward
// ROW: a row or a part of one to the workgroup; else a row to tpr lanes, several
// rows to a workgroup (V up to a few vectors a lane). Two vectors of a thread at a
// time, the next ones loaded before the current ones are used: where all of them
// are whole, without a check, and added at once.
template <typename T, bool TOP, bool ROW, bool NT>
__global__ __launch_bounds__(kLpThreads) void lp_fwd_kernel(LpArgs a) {
    static_assert(ROW || !TOP, "alternatives take a workgroup");
    constexpr int VEC = VecOf<T>::n, U = 2;
    constexpr int LINE = 8 * VEC;   // elements of a line: eight lanes' vectors
    extern __shared__ uint64_t dyn[];
    const float k2 = a.scale * kLog2e;
    const int tpr = ROW ? kLpThreads : a.tpr;
    const int t = (int)threadIdx.x & (tpr - 1), g = ROW ? 0 : (int)threadIdx.x / tpr;
    const uint32_t item = blockIdx.x * (uint32_t)(kLpThreads / tpr) + (uint32_t)g;   // (row, part)
    const uint32_t m = item / (uint32_t)a.parts, part = item - m * (uint32_t)a.parts;
    const RowPart<T> r((const T*)a.logits, m, part, a);
    float* line_max = (float*)dyn;
    Lse v = lse_none();
    const int step = tpr * VEC;
    int base = r.first;   // the row's first lane's place: the same for all its lanes
    u32x4 next[U];
    const auto whole = [&](int b) { return ROW && b >= r.lo && b + U * step <= r.hi; };   // for all lanes
    const auto load = [&](int b) {
        if (whole(b)) {
            const char* from = (const char*)r.p;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const u32x4* at = (const u32x4*)(from + (uint32_t)(b + u * step + t * VEC) * (uint32_t)sizeof(T));
                if constexpr (NT) next[u] = __builtin_nontemporal_load(at);
                else next[u] = *at;
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) next[u] = r.template load<NT>(b + u * step + t * VEC);
        }
    };
    // the maximum of a line; `e`: the place of the lane's vector of it
    const auto line = [&](float most, int e) {
        if constexpr (TOP) {
            most = lanes_max8(most);
            if ((t & 7) == 0 && e < r.end) line_max[(uint32_t)(e - r.first) / LINE] = most;
        }
    };
    load(base);
    const RowToken<T> token(a, m);
    for (; base < r.end; base += U * step) {
        u32x4 now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        if (base + U * step < r.end) load(base + U * step);
        if (whole(base)) {
            float x[U][VEC], most[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                unpack16<T>(now[u], x[u]);
                most[u] = vec_max<VEC>(x[u]);
                line(most[u], base + u * step + t * VEC);
            }
            lse_add<U * VEC>(v, x[0], max3(most[0], most[1], most[1]), k2);
            continue;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = base + u * step, e = b + t * VEC;
            if (b >= r.end) continue;
            float x[VEC];
            unpack16<T>(now[u], x);
            if (!r.whole(e)) r.elements(e, x);
            const float most = vec_max<VEC>(x);
            line(most, e);
            lse_add<VEC>(v, x, most, k2);
        }
    }
    __shared__ Lse red[kLpThreads / 64];
    if constexpr (ROW) v = lse_group(v, red);
    else v = lse_lanes(v, tpr);
    if (t == 0 && m < a.T) {
        if (a.parts == 1) {
            lp_write(a, m, v, token.x, token.real, k2);
        } else {
            float* to = a.part + (int64_t)item * 4;
            to[0] = v.m;
            to[1] = v.s;
            to[2] = v.t;
        }
    }
    if constexpr (TOP) {
        __shared__ TopShared sh;
        __shared__ uint64_t lines[kLpMaxTop];
        const int k = a.top;
        // (none of a row's last part whose places end before it)
        const int n_lines = (max(r.end - r.first, 0) + LINE - 1) / LINE;
        uint64_t* list = dyn + (a.part_len / LINE + 1) / 2;   // behind the lines' maxima
        // the k best lines: each thread has every 256th
        uint64_t best = 0;
#pragma unroll 4
        for (int i = (int)threadIdx.x; i < n_lines; i += kLpThreads) best = max(best, top_key(line_max[i], (uint32_t)i));
        uint64_t bound = top_bound(best, k, sh);
#pragma unroll 4
        for (int i = (int)threadIdx.x; i < n_lines; i += kLpThreads)
            top_keep(top_key(line_max[i], (uint32_t)i), bound, list, sh);
        if (threadIdx.x < kLpMaxTop) lines[threadIdx.x] = 0;
        top_rank(list, k, sh, [&](int place, uint64_t key) { lines[place] = key; });
        __syncthreads();
        // their elements, a vector to a lane, 32 lines at a time, packed: their
        // keys would take the registers of two more waves
        constexpr int H = kLpMaxTop / 32;
        int place[H];
        u32x4 raw[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int at = h * 32 + ((int)threadIdx.x >> 3);
            const uint64_t line = at < k ? lines[at] : 0;
            place[h] = line == 0 ? -1 : r.first + (int)key_at(line) * LINE + ((int)threadIdx.x & 7) * VEC;
            if (place[h] >= 0) raw[h] = r.template load<false>(place[h]);
        }
        const auto each = [&](auto&& f) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if (place[h] < 0) continue;
                float x[VEC];
                unpack16<T>(raw[h], x);
                if (!r.whole(place[h])) r.elements(place[h], x);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (r.in_row(place[h], i)) f(top_key(x[i], (uint32_t)(place[h] + i - r.skew)));
            }
        };
        best = 0;
        each([&](uint64_t key) { best = max(best, key); });
        bound = top_bound(best, k, sh);
        each([&](uint64_t key) { top_keep(key, bound, list, sh); });
        const RowSum row(v, k2);
        top_rank(list, k, sh, [&](int place, uint64_t best_key) {
            if (a.parts > 1) {
                a.part_top[(int64_t)item * k + place] = best_key;
            } else {
                a.top_tokens[(int64_t)m * k + place] = key_at(best_key);
                a.top_logp[(int64_t)m * k + place] = row.log_p(key_value(best_key), a.to_ln);
            }
        });
        // a part of fewer than k elements
        if (a.parts > 1 && (int)threadIdx.x < k && threadIdx.x >= sh.count) a.part_top[(int64_t)item * k + threadIdx.x] = 0;
    }
}

// The parts of a row, up to 256 of them.
template <typename T, bool TOP>
__global__ __launch_bounds__(kLpThreads) void lp_join_kernel(LpArgs a) {
    __shared__ Lse red[kLpThreads / 64];
    const int64_t m = blockIdx.x;
    const int t = (int)threadIdx.x;
    const float k2 = a.scale * kLog2e;
    const RowToken<T> token(a, m);
    Lse v = lse_none();
    if (t < a.parts) {
        const float* from = a.part + (m * a.parts + t) * 4;
        v = {from[0], from[1], from[2]};
    }
    v = lse_group(v, red);
    if (t == 0) lp_write(a, m, v, token.x, token.real, k2);
    if constexpr (TOP) {
        extern __shared__ uint64_t list[];
        __shared__ TopShared sh;
        const int k = a.top, n = a.parts * k;
        const uint64_t* keys = a.part_top + m * n;
        uint64_t best = 0;
        for (int i = t; i < n; i += kLpThreads) best = max(best, keys[i]);
        const uint64_t bound = top_bound(best, k, sh);
        for (int i = t; i < n; i += kLpThreads) top_keep(keys[i], bound, list, sh);
        const RowSum row(v, k2);
        top_rank(list, k, sh, [&](int place, uint64_t key) {
            a.top_tokens[m * k + place] = key_at(key);
            a.top_logp[m * k + place] = row.log_p(key_value(key), a.to_ln);
        });
    }
}

// -------------------------------------------------------------- backward
// A tile of kLpBwdVecs vectors a thread of one row (or, of short rows, all of
// several): neighbouring workgroups read and write neighbouring memory. A row
// without an upstream gradient counts as zeros.
// NORM: y = k x - m - log2 s from the forward's two numbers, whose difference to k x
// is small wherever the row's logits lie; the one float32 lse is rounded by up to
// |lse| 2^-24, and with it every p of the row.
template <typename T, bool NORM>
__global__ __launch_bounds__(kLpThreads) void lp_bwd_kernel(LpArgs a) {
    constexpr int VEC = VecOf<T>::n;
    constexpr int U = kLpBwdVecs;
    const int tpr = a.tpr;
    const int t = (int)threadIdx.x & (tpr - 1), g = (int)threadIdx.x / tpr;
    const uint32_t item = blockIdx.x * (uint32_t)(kLpThreads / tpr) + (uint32_t)g;
    const uint32_t m = item / (uint32_t)a.parts, part = item - m * (uint32_t)a.parts;
    if (m >= a.T) return;
    const RowPart<T> r((const T*)a.logits, m, part, a);
    T* out = (T*)a.dlogits + (int64_t)m * a.ldd - r.skew;   // place 0
    const int e0 = r.first + t * VEC;
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = r.template load<false>(e0 + u * tpr * VEC);
    const int64_t token = a.token_bits == 64 ? ((const int64_t*)a.tokens)[m] : (int64_t)((const int32_t*)a.tokens)[m];
    const bool real = token >= 0 && token < a.V;
    const int at = real ? (int)token + r.skew : -VEC;
    const float* norm = NORM ? a.norm + 3 * (int64_t)m : nullptr;
    const float lse = NORM ? norm[0] : a.lse[m];   // or m
    const float log2_s = NORM ? norm[1] : 0.0f;
    const float h = NORM ? norm[2] : a.entropy[m];
    const float up = real && a.dlogp ? a.dlogp[m] : 0.0f;
    const float ue = a.dentropy ? a.dentropy[m] : 0.0f;
    const bool dead = (up == 0.0f && ue == 0.0f) || (NORM ? log2_s : lse) == -INFINITY;
    // dx = -scale p (up + ue (z - lse + h)), and scale up more at the token
    const float base = -a.scale * (up + ue * h), slope = -a.scale * ue * (NORM ? kLn2 : 1.0f);
    const float factor = NORM ? a.scale * kLog2e : a.scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e = e0 + u * tpr * VEC;
        if (e >= r.end) break;
        const bool whole = r.whole(e);
        float x[VEC];
        unpack16<T>(raw[u], x);
        if (!whole) r.elements(e, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float z = __builtin_fmaf(x[i], factor, -lse);
            if constexpr (NORM) z -= log2_s;
            const float p = __builtin_amdgcn_exp2f(NORM ? z : z * kLog2e);
            // (a masked place's z and large upstream gradients have products that are not finite)
            x[i] = p == 0.0f ? 0.0f : p * __builtin_fmaf(z, slope, base);
        }
        if ((uint32_t)(at - e) < (uint32_t)VEC) {   // (at a masked place too: [j = c] stays 1)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (at == e + i) x[i] = __builtin_fmaf(a.scale, up, x[i]);
        }
        if (dead) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = 0.0f;
        }
        if (whole) {
            *(u32x4_m*)(out + e) = pack16<T>(x);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (r.in_row(e, i)) out[e + i] = dyt::from_f32<T>(x[i]);
        }
    }
}

}  // namespace dytb
