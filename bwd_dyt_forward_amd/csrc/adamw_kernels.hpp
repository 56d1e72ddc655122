// adamw_kernels.hpp - an AdamW step over many tensors at once (gfx950).
//
//   g' = grad_scale g        m = beta1 m + (1 - beta1) g'
//   v = beta2 v + (1 - beta2) g'^2
//   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
//
// Bound by HBM: every operand is read and written once, in one launch for up
// to kAdamTensors tensors, whose addresses travel in the kernel's arguments (no
// copy to the device, and a captured launch keeps them). A workgroup takes a
// run of kAdamChunk elements of one tensor, found by bisection.
//
// 8-bit states: blocks of 128 elements with a float32 scale a each, the block's
// largest absolute value (2^-126 at least).
//   first moment   int8  c: a sign(c) (c / 127)^2
//   second moment  uint8 c: a (c / 255)^4
// The codes' steps shrink with the value, so that small moments beside a large
// one keep their digits: one part in 64 (first) and 64 (second) at the top, a
// value's whole size only at 1 / 16,129 of the largest first and 2.4e-10 of the
// largest second moment. A decayed average moves by less than half a step most
// of the time and would stand still if it were rounded to the nearest code; with
// a seed, the code above is taken with the probability of the value's place
// between the two, so that the codes' mean is the value. The second moment's
// code is at least 1 where the moment is not zero: it is divided by. A block is
// 16 lanes of 8 elements: its maximum takes lane exchanges only. It is taken on
// the bits, where a NaN is larger than all else: a NaN spoils its block.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

constexpr int kAdamThreads = 256;
constexpr int kAdamTensors = 44;          // of a launch: their table stays under 4 KB of arguments
constexpr int kAdamChunk = 8192;          // elements of a workgroup, a multiple of 256 x 8
constexpr int kAdamBlock = 128;
constexpr float kScaleTiny = 0x1p-126f;

struct AdamTensor {
    void* param;
    const void* grad;
    void* avg;
    void* sq;
    float* avg_scale;
    float* sq_scale;
    float* master;
    int64_t n;
    uint32_t number;      // in the caller's list: enters the random numbers
    uint32_t first;       // its first workgroup
};

struct AdamArgs {
    AdamTensor t[kAdamTensors];
    int32_t count;
    int32_t seeded;
    uint32_t seed;
    float beta1, one_beta1, beta2, one_beta2, eps;
    float keep, rate, inv_corr2;  // 1 - lr weight_decay, lr / (1 - beta1^step), 1 / (1 - beta2^step)
    double lr, weight_decay;      // for those three where the device holds lr or step
    double log_beta1, log_beta2;
    int64_t step;
    const float* lr_dev;          // each or null
    const int64_t* step_dev;
    const float* grad_scale;
};

// The kernel's only argument where it lies. A reference to the parameter
// itself would be one to a copy of the whole table in scratch memory, since
// it is indexed.
__device__ __forceinline__ const AdamArgs& adam_args() {
    return *(const AdamArgs*)__builtin_amdgcn_kernarg_segment_ptr();
}

// A 32-bit hash (the finalizer of MurmurHash3; A. Appleby, 2011).
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
    x = (x ^ (x >> 13)) * 0xC2B2AE35u;
    return x ^ (x >> 16);
}

// The next random number (xorshift; G. Marsaglia, 2003).
__device__ __forceinline__ uint32_t next_random(uint32_t x) {
    x ^= x << 13;
    x ^= x >> 17;
    return x ^ (x << 5);
}

// V elements at p, n of them there (zeros for the rest).
template <typename T, int V>
__device__ __forceinline__ void load_some(const T* p, int64_t n, float* out) {
    if (n >= V) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) unpack16<T>(*(const u32x4_m*)(p + i), out + i);
        } else if constexpr (V == 8) {
            unpack16<T>(*(const u32x4_m*)p, out);
        } else {
            uint32_t w[2];
            __builtin_memcpy(w, p, 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = to_f32(T{(uint16_t)(w[i / 2] >> (16 * (i % 2)))});
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_some(T* p, int64_t n, const float* v) {
    if (n >= V) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) *(u32x4_m*)(p + i) = pack16<T>(v + i);
        } else if constexpr (V == 8) {
            *(u32x4_m*)p = pack16<T>(v);
        } else {
            const uint32_t w[2] = {pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
            __builtin_memcpy(p, w, 8);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = dyt::from_f32<T>(v[i]);
    }
}

struct AdamStep {
    float beta1, one_beta1, beta2, one_beta2, eps, keep, rate, inv_corr2;

    __device__ __forceinline__ void operator()(float& p, float& m, float& v, float g) const {
        m = __builtin_fmaf(m, beta1, g * one_beta1);
        v = __builtin_fmaf(v, beta2, g * g * one_beta2);
        const float root = __builtin_amdgcn_sqrtf(v * inv_corr2) + eps;
        p = __builtin_fmaf(p, keep, -rate * m * __builtin_amdgcn_rcpf(root));
    }
};

__device__ __forceinline__ AdamStep adam_step(const AdamArgs& a) {
    AdamStep r{a.beta1, a.one_beta1, a.beta2, a.one_beta2, a.eps, a.keep, a.rate, a.inv_corr2};
    if (a.lr_dev || a.step_dev) {
        const double step = (double)(a.step_dev ? *a.step_dev : a.step);
        const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
        r.keep = (float)(1.0 - lr * a.weight_decay);
        r.rate = (float)(lr / -expm1(step * a.log_beta1));
        r.inv_corr2 = (float)(1.0 / -expm1(step * a.log_beta2));
    }
    return r;
}

__device__ __forceinline__ int adam_tensor(const AdamArgs& a, uint32_t wg) {
    int lo = 0, hi = a.count - 1;   // the last tensor that begins at or before wg
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.t[mid].first <= wg) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// float32 states, four elements a lane: every access of a wave is one run.
template <typename TP, typename TG, bool MASTER>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs) {
    const AdamArgs& a = adam_args();
    constexpr int V = 4;
    const AdamTensor& x = a.t[adam_tensor(a, blockIdx.x)];
    const AdamStep step = adam_step(a);
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int64_t base = (int64_t)(blockIdx.x - x.first) * kAdamChunk;
    const int64_t end = min(base + kAdamChunk, x.n);
#pragma unroll 2
    for (int64_t i = base + (int64_t)threadIdx.x * V; i < end; i += kAdamThreads * V) {
        const int64_t n = end - i;
        float p[V], g[V], m[V], v[V];
        if constexpr (MASTER) load_some<float, V>(x.master + i, n, p);
        else load_some<TP, V>((const TP*)x.param + i, n, p);
        load_some<TG, V>((const TG*)x.grad + i, n, g);
        load_some<float, V>((const float*)x.avg + i, n, m);
        load_some<float, V>((const float*)x.sq + i, n, v);
#pragma unroll
        for (int j = 0; j < V; ++j) step(p[j], m[j], v[j], g[j] * gs);
        if constexpr (MASTER) store_some<float, V>(x.master + i, n, p);
        store_some<TP, V>((TP*)x.param + i, n, p);
        store_some<float, V>((float*)x.avg + i, n, m);
        store_some<float, V>((float*)x.sq + i, n, v);
    }
}

// Maximum of the bits over aligned groups of 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}

__device__ __forceinline__ float block_max(uint32_t v) {
    v = dpp_max_u32<0xB1>(v);
    v = dpp_max_u32<0x4E>(v);
    v = dpp_max_u32<0x141>(v);
    v = dpp_max_u32<0x140>(v);
    return __uint_as_float(max(v, __float_as_uint(kScaleTiny)));
}

// The codes' values. c: the code as a float.
__device__ __forceinline__ float avg_value(float c, float a) { return c * __builtin_fabsf(c) * (1.0f / 16129.0f) * a; }

__device__ __forceinline__ float sq_value(float c, float a) {
    const float r = c * c * (1.0f / 65025.0f);   // c * c is exact
    return r * r * a;
}

__device__ __forceinline__ int avg_code(uint32_t w, int i) { return (int)(int8_t)(w >> (8 * i)); }

// The code for y = 127^2 |m| / a: of the two around it the upper one if the
// random number is below y's place between them.
__device__ __forceinline__ float avg_round(float y, float random) {
    const float low = fminf(__builtin_floorf(__builtin_amdgcn_sqrtf(y)), 126.0f);
    const float above = __builtin_fmaf(-low, low, y);
    return random * __builtin_fmaf(2.0f, low, 1.0f) < above ? low + 1.0f : low;
}

// The same for y = 255^4 v / a; a moment that is not zero gets no code 0.
__device__ __forceinline__ float sq_round(float y, float random, bool some) {
    const float low = fminf(__builtin_floorf(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(y))), 254.0f);
    const float l2 = low * low;
    const float above = __builtin_fmaf(-l2, l2, y);
    const float gap = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(4.0f, low, 6.0f), low, 4.0f), low, 1.0f);
    const float c = random * gap < above ? low + 1.0f : low;
    return some ? fmaxf(c, 1.0f) : c;
}

template <typename TP, typename TG, bool MASTER>
__global__ __launch_bounds__(kAdamThreads) void adamw8_kernel(AdamArgs) {
    const AdamArgs& a = adam_args();
    constexpr int V = 8;
    const AdamTensor& x = a.t[adam_tensor(a, blockIdx.x)];
    const AdamStep step = adam_step(a);
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int64_t base = (int64_t)(blockIdx.x - x.first) * kAdamChunk;
    const int64_t end = min(base + kAdamChunk, x.n);
    const uint32_t at_step = (uint32_t)(a.step_dev ? *a.step_dev : a.step);
    const uint32_t key = mix32(a.seed + 0x9E3779B9u * at_step) ^ mix32(0x85EBCA77u * (x.number + 1u));
    // whole blocks: the lanes past the end take part in the maxima
    const int64_t stop = base + (end - base + kAdamBlock - 1) / kAdamBlock * kAdamBlock;
    for (int64_t i = base + (int64_t)threadIdx.x * V; i < stop; i += kAdamThreads * V) {
        const int64_t n = end - i;
        float p[V], g[V], m[V], v[V];
        uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
        if constexpr (MASTER) load_some<float, V>(x.master + i, n, p);
        else load_some<TP, V>((const TP*)x.param + i, n, p);
        load_some<TG, V>((const TG*)x.grad + i, n, g);
        if (n >= V) {
            __builtin_memcpy(cm, (const uint8_t*)x.avg + i, 8);
            __builtin_memcpy(cv, (const uint8_t*)x.sq + i, 8);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) {
                    cm[j / 4] |= (uint32_t)((const uint8_t*)x.avg)[i + j] << (8 * (j % 4));
                    cv[j / 4] |= (uint32_t)((const uint8_t*)x.sq)[i + j] << (8 * (j % 4));
                }
        }
        const float am = x.avg_scale[i / kAdamBlock], av = x.sq_scale[i / kAdamBlock];
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            m[j] = avg_value((float)avg_code(cm[j / 4], j % 4), am);
            v[j] = sq_value((float)((cv[j / 4] >> (8 * (j % 4))) & 255u), av);
            step(p[j], m[j], v[j], g[j] * gs);
            if (j < n) {
                top_m = max(top_m, __float_as_uint(m[j]) & 0x7fffffffu);
                top_v = max(top_v, __float_as_uint(v[j]) & 0x7fffffffu);
            }
        }
        const float new_m = block_max(top_m), new_v = block_max(top_v);
        const float inv_m = 1.0f / new_m, inv_v = 1.0f / new_v;
        const uint64_t vec = (uint64_t)i / V;
        uint32_t r = mix32((uint32_t)vec ^ key ^ mix32((uint32_t)(vec >> 32))) | 1u;
        cm[0] = cm[1] = cv[0] = cv[1] = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j) r = next_random(r);
            const float r1 = a.seeded ? ((float)(r >> 16) + 0.5f) * 0x1p-16f : 0.5f;
            const float r2 = a.seeded ? ((float)(r & 0xffffu) + 0.5f) * 0x1p-16f : 0.5f;
            float c = avg_round(__builtin_fabsf(m[j]) * inv_m * 16129.0f, r1);
            c = m[j] < 0.0f && c > 0.0f ? 256.0f - c : c;   // two's complement
            cm[j / 4] = __builtin_amdgcn_cvt_pk_u8_f32(c, j % 4, cm[j / 4]);
            c = sq_round(v[j] * inv_v * 4228250625.0f, r2, v[j] > 0.0f);
            cv[j / 4] = __builtin_amdgcn_cvt_pk_u8_f32(c, j % 4, cv[j / 4]);
        }
        if (n >= V) {
            __builtin_memcpy((uint8_t*)x.avg + i, cm, 8);
            __builtin_memcpy((uint8_t*)x.sq + i, cv, 8);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) {
                    ((uint8_t*)x.avg)[i + j] = (uint8_t)(cm[j / 4] >> (8 * (j % 4)));
                    ((uint8_t*)x.sq)[i + j] = (uint8_t)(cv[j / 4] >> (8 * (j % 4)));
                }
        }
        if ((threadIdx.x & 15) == 0) {
            x.avg_scale[i / kAdamBlock] = new_m;
            x.sq_scale[i / kAdamBlock] = new_v;
        }
        if constexpr (MASTER) store_some<float, V>(x.master + i, n, p);
        store_some<TP, V>((TP*)x.param + i, n, p);
    }
}

// The values that codes stand for. `avg` holds the codes, `param` the values;
// `number`: 0 the first moment, 1 the second.
template <typename TO>
__global__ __launch_bounds__(kAdamThreads) void adamw_values_kernel(AdamArgs) {
    const AdamArgs& a = adam_args();
    constexpr int V = 8;
    const AdamTensor& x = a.t[adam_tensor(a, blockIdx.x)];
    const int64_t base = (int64_t)(blockIdx.x - x.first) * kAdamChunk;
    const int64_t end = min(base + kAdamChunk, x.n);
#pragma unroll 2
    for (int64_t i = base + (int64_t)threadIdx.x * V; i < end; i += kAdamThreads * V) {
        const int64_t n = end - i;
        uint32_t c[2] = {0, 0};
        if (n >= V) {
            __builtin_memcpy(c, (const uint8_t*)x.avg + i, 8);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) c[j / 4] |= (uint32_t)((const uint8_t*)x.avg)[i + j] << (8 * (j % 4));
        }
        const float s = x.avg_scale[i / kAdamBlock];
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = x.number ? sq_value((float)((c[j / 4] >> (8 * (j % 4))) & 255u), s)
                            : avg_value((float)avg_code(c[j / 4], j % 4), s);
        store_some<TO, V>((TO*)x.param + i, n, v);
    }
}

}  // namespace dytb
