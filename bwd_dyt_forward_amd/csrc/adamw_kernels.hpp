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

#include <type_traits>

#include "ln_kernels.hpp"

namespace dytb {

constexpr int kAdamThreads = 256;
constexpr int kAdamTensors = 44;          // of a launch: their table stays under 4 KB of arguments
// Elements of a workgroup: what 256 threads hold at once; with 8-bit states,
// where the arithmetic is the bound, more (8,192 for 2,048: 798 us for 815).
constexpr int kAdamChunk = 2048, kAdamChunk8 = 8192;
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
    float keep, rate, root_corr2; // 1 - lr weight_decay, lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
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

// A 32-bit hash (the finalizer of a published one: A. Appleby, 2011).
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

// 8 and 16 bytes at an element's (or a code's) alignment.
typedef uint32_t u32x2_m __attribute__((ext_vector_type(2), aligned(1)));

template <bool NT>
__device__ __forceinline__ u32x4 load16(const void* p) {
    if constexpr (NT) return __builtin_nontemporal_load((const u32x4_m*)p);
    else return *(const u32x4_m*)p;
}

template <bool NT>
__device__ __forceinline__ u32x2 load8(const void* p) {
    if constexpr (NT) return __builtin_nontemporal_load((const u32x2_m*)p);
    else return *(const u32x2_m*)p;
}

template <bool NT>
__device__ __forceinline__ void store16(void* p, u32x4 v) {
    if constexpr (NT) __builtin_nontemporal_store((u32x4_m)v, (u32x4_m*)p);
    else *(u32x4_m*)p = v;
}

template <bool NT>
__device__ __forceinline__ void store8(void* p, u32x2 v) {
    if constexpr (NT) __builtin_nontemporal_store((u32x2_m)v, (u32x2_m*)p);
    else *(u32x2_m*)p = v;
}

// V elements at p, n of them there (zeros for the rest).
template <typename T, int V, int NT = 0>
__device__ __forceinline__ void load_some(const T* p, int64_t n, float* out) {
    if (n >= V) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) unpack16<T>(load16<(NT & 2) != 0>(p + i), out + i);
        } else if constexpr (V == 8) {
            unpack16<T>(load16<(NT & 2) != 0>(p), out);
        } else {
            const u32x2 w = load8<(NT & 2) != 0>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = to_f32(T{(uint16_t)(w[i / 2] >> (16 * (i % 2)))});
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}

template <typename T, int V, int NT = 0>
__device__ __forceinline__ void store_some(T* p, int64_t n, const float* v) {
    if (n >= V) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) store16<(NT & 1) != 0>(p + i, pack16<T>(v + i));
        } else if constexpr (V == 8) {
            store16<(NT & 1) != 0>(p, pack16<T>(v));
        } else {
            store8<(NT & 1) != 0>(p, u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])});
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = dyt::from_f32<T>(v[i]);
    }
}

struct AdamStep {
    float beta1, one_beta1, beta2, one_beta2, eps, keep, rate, root_corr2;

    // Returns the second moment's root. SMALL: of subnormal moments too, which the
    // hardware's root takes for 0 (with an eps of 0 the step would be infinite); free beside
    // float32 states, while 8-bit states, where the arithmetic is the bound, hold no such moments.
    template <bool SMALL>
    __device__ __forceinline__ float step(float& p, float& m, float& v, float g) const {
        m = __builtin_fmaf(m, beta1, g * one_beta1);
        v = __builtin_fmaf(v, beta2, g * g * one_beta2);
        const bool small = SMALL && v < 0x1p-100f;
        float root = __builtin_amdgcn_sqrtf(small ? v * 0x1p60f : v);
        if (small) root *= 0x1p-30f;
        const float inv = __builtin_amdgcn_rcpf(__builtin_fmaf(root, root_corr2, eps));
        p = __builtin_fmaf(-rate * m, inv, p * keep);
        return root;
    }
};

__device__ __forceinline__ AdamStep adam_step(const AdamArgs& a) {
    AdamStep r{a.beta1, a.one_beta1, a.beta2, a.one_beta2, a.eps, a.keep, a.rate, a.root_corr2};
    if (a.lr_dev || a.step_dev) {
        const double step = (double)(a.step_dev ? *a.step_dev : a.step);
        const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
        r.keep = (float)(1.0 - lr * a.weight_decay);
        r.rate = (float)(lr / -expm1(step * a.log_beta1));
        r.root_corr2 = (float)(1.0 / sqrt(-expm1(step * a.log_beta2)));
    }
    return r;
}

// The tensor of a workgroup: the last that begins at or before it, found by all
// lanes at once.
__device__ __forceinline__ int adam_tensor(const AdamArgs& a, uint32_t wg) {
    static_assert(kAdamTensors <= 64, "a lane for each");
    const int lane = (int)threadIdx.x & 63;
    const bool before = lane < a.count && a.t[min(lane, kAdamTensors - 1)].first <= wg;
    return __builtin_amdgcn_readfirstlane(__popcll(__ballot(before)) - 1);
}

// float32 states, four elements a lane: every access of a wave is one run. All
// loads of a workgroup's chunk are on their way before its first store (the
// compiler may not move one before a store: the tensors could be the same).
// STREAM: nontemporal loads and stores where the tensors pass the last-level
// cache. 332 million bfloat16 parameters with masters: 1,803 us with a loop of
// two loads ahead, 1,754 so, 1,653 nontemporal (5.6 TB/s of eight streams).
template <typename TP, typename TG, bool MASTER, bool STREAM>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs) {
    constexpr int NT = STREAM ? 3 : 0, V = 4, U = kAdamChunk / (kAdamThreads * V);
    const AdamArgs& a = adam_args();
    const AdamTensor& x = a.t[adam_tensor(a, blockIdx.x)];
    const int64_t base = (int64_t)(blockIdx.x - x.first) * kAdamChunk + (int64_t)threadIdx.x * V;
    const AdamStep step = adam_step(a);
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    // whole: no element past the end, known for the workgroup
    const auto run = [&](auto whole) {
        float p[U][V], g[U][V], m[U][V], v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + u * kAdamThreads * V, n = decltype(whole)::value ? V : x.n - i;
            if constexpr (MASTER) load_some<float, V, NT>(x.master + i, n, p[u]);
            else load_some<TP, V, NT>((const TP*)x.param + i, n, p[u]);
            load_some<TG, V, NT>((const TG*)x.grad + i, n, g[u]);
            load_some<float, V, NT>((const float*)x.avg + i, n, m[u]);
            load_some<float, V, NT>((const float*)x.sq + i, n, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = base + u * kAdamThreads * V, n = decltype(whole)::value ? V : x.n - i;
#pragma unroll
            for (int j = 0; j < V; ++j) step.step<true>(p[u][j], m[u][j], v[u][j], g[u][j] * gs);
            if constexpr (MASTER) store_some<float, V, NT>(x.master + i, n, p[u]);
            store_some<TP, V, NT>((TP*)x.param + i, n, p[u]);
            store_some<float, V, NT>((float*)x.avg + i, n, m[u]);
            store_some<float, V, NT>((float*)x.sq + i, n, v[u]);
        }
    };
    if ((int64_t)(blockIdx.x - x.first + 1) * kAdamChunk <= x.n) run(std::true_type{});
    else run(std::false_type{});
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

__device__ __forceinline__ int avg_code(uint32_t w, int i) { return (int)(int8_t)(w >> (8 * i)); }

__device__ __forceinline__ float sq_code(uint32_t w, int i) { return (float)((w >> (8 * i)) & 255u); }

// Of the two codes c and c + 1 around y = 127^2 |m| / a, the upper one if u =
// (random + 0.5) / 65536 is below y's place between them, y > c^2 + u (2 c + 1). That
// is (c + u)^2 + u (1 - u): the square root of y - u (1 - u), and 1/2 - u added,
// rounds to it. (y may pass 127^2 by a rounding.) `inv` is 1 / a, without 127^2: with
// it the factor of a block below 127^2 / 2^128 would be infinite.
__device__ __forceinline__ float avg_round(float m, float inv, float random) {
    const float h = __builtin_fmaf(random, -0x1p-16f, 0.5f);   // 1/2 - u
    const float w = __builtin_fmaf(h, h, -0.25f);              // -u (1 - u)
    const float root = __builtin_amdgcn_sqrtf(fmaxf(__builtin_fmaf(__builtin_fabsf(m) * inv, 16129.0f, w), 0.0f));
    return fminf(__builtin_rintf(root + h), 127.0f);
}

// The upper code likewise for y = z^2 = 255^4 v / a; a moment that is not zero gets no code 0.
// (256, where a rounding takes y past 255^4, becomes 255 as it is packed.)
__device__ __forceinline__ float sq_round(float z, float random) {
    const float low = __builtin_floorf(__builtin_amdgcn_sqrtf(z));
    const float l2 = low * low;
    const float above = __builtin_fmaf(-l2, l2, z * z);
    // (4 low^3 + 6 low^2 + 4 low + 1) / 65536
    const float gap = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(0x1p-14f, low, 0x1.8p-14f), low, 0x1p-14f), low, 0x1p-16f);
    const float c = random * gap < above ? low + 1.0f : low;
    return fmaxf(c, __builtin_amdgcn_fmed3f(z * 0x1p100f, 0.0f, 1.0f));
}

// Bound by arithmetic: about 62 operations and four of a quarter of the rate an
// element. Hence one root of v for the step and for its code, factors of a block
// in front of the loop over its elements (a lane's eight), codes of both signs
// as c + 128 until they are packed, and an instance of its own for rounding at
// random. Loads and stores are ordinary ones: nontemporal loads give 16 million
// bfloat16 parameters 42 us for 39 (with masters 58 for 42), 40 million 89 for 84 (119 for
// 127), 60 million 126 for 131, 120 million 262 for 258, 300 million with masters 945 for 926.
template <typename TP, typename TG, bool MASTER, bool SEEDED>
__global__ __launch_bounds__(kAdamThreads) void adamw8_kernel(AdamArgs) {
    constexpr int V = 8;
    const AdamArgs& a = adam_args();
    const AdamTensor& x = a.t[adam_tensor(a, blockIdx.x)];
    const AdamStep step = adam_step(a);
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int64_t base = (int64_t)(blockIdx.x - x.first) * kAdamChunk8;
    const int64_t end = min(base + kAdamChunk8, x.n);
    const uint32_t at_step = (uint32_t)(a.step_dev ? *a.step_dev : a.step);
    const uint32_t key = mix32(a.seed + 0x9E3779B9u * at_step) ^ mix32(0x85EBCA77u * (x.number + 1u));
    // whole blocks: the lanes past the end take part in the maxima, with zeros
    const int64_t stop = base + (end - base + kAdamBlock - 1) / kAdamBlock * kAdamBlock;
    for (int64_t i = base + (int64_t)threadIdx.x * V; i < stop; i += kAdamThreads * V) {
        const int64_t n = end - i;
        float p[V], g[V], m[V], root[V];
        u32x2 cm = {0, 0}, cv = {0, 0};
        if constexpr (MASTER) load_some<float, V>(x.master + i, n, p);
        else load_some<TP, V>((const TP*)x.param + i, n, p);
        load_some<TG, V>((const TG*)x.grad + i, n, g);
        if (n >= V) {
            cm = load8<false>((const uint8_t*)x.avg + i);
            cv = load8<false>((const uint8_t*)x.sq + i);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) {
                    cm[j / 4] |= (uint32_t)((const uint8_t*)x.avg)[i + j] << (8 * (j % 4));
                    cv[j / 4] |= (uint32_t)((const uint8_t*)x.sq)[i + j] << (8 * (j % 4));
                }
        }
        // beta1 a: a / 127^2 would be subnormal, with few digits, in blocks below 2e-34
        AdamStep of_block = step;
        of_block.beta1 *= x.avg_scale[i / kAdamBlock];
        const float av = __builtin_amdgcn_sqrtf(x.sq_scale[i / kAdamBlock]) * (1.0f / 65025.0f);
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float c = (float)avg_code(cm[j / 4], j % 4), c2 = sq_code(cv[j / 4], j % 4);
            m[j] = c * __builtin_fabsf(c) * (1.0f / 16129.0f);   // the moment / a
            const float r = c2 * c2 * av;
            float v = r * r;
            root[j] = of_block.step<false>(p[j], m[j], v, g[j] * gs);
            top_m = max(top_m, __float_as_uint(m[j]) & 0x7fffffffu);
            top_v = max(top_v, __float_as_uint(v));
        }
        const float new_m = block_max(top_m), new_v = block_max(top_v);
        const float inv_m = __builtin_amdgcn_rcpf(new_m), inv_v = 65025.0f * __builtin_amdgcn_rsqf(new_v);
        const uint64_t vec = (uint64_t)i / V;
        uint32_t r = SEEDED ? mix32((uint32_t)vec ^ key ^ mix32((uint32_t)(vec >> 32))) | 1u : 0u;
        cm = cv = u32x2{0, 0};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (SEEDED && j) r = next_random(r);
            const float r1 = SEEDED ? (float)(r >> 16) + 0.5f : 32768.0f;
            const float r2 = SEEDED ? (float)(r & 0xffffu) + 0.5f : 32768.0f;
            const float c = avg_round(m[j], inv_m, r1);
            cm[j / 4] = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_copysignf(c, m[j]) + 128.0f, j % 4, cm[j / 4]);
            cv[j / 4] = __builtin_amdgcn_cvt_pk_u8_f32(sq_round(root[j] * inv_v, r2), j % 4, cv[j / 4]);
        }
        cm ^= 0x80808080u;   // c + 128 to two's complement
        if (n >= V) {
            store8<false>((uint8_t*)x.avg + i, cm);
            store8<false>((uint8_t*)x.sq + i, cv);
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
// `number`: 0 the first moment, 1 the second. Ordinary loads: both moments of 20
// million parameters to bfloat16 19 us, with nontemporal loads 24; of 60 million 68 and 60;
// of 90 million 100 and 100; of 300 million 314 and 318.
template <typename TO>
__global__ __launch_bounds__(kAdamThreads) void adamw_values_kernel(AdamArgs) {
    const AdamArgs& a = adam_args();
    constexpr int V = 8;
    const AdamTensor& x = a.t[adam_tensor(a, blockIdx.x)];
    const int64_t base = (int64_t)(blockIdx.x - x.first) * kAdamChunk8;
    const int64_t end = min(base + kAdamChunk8, x.n);
#pragma unroll 2
    for (int64_t i = base + (int64_t)threadIdx.x * V; i < end; i += kAdamThreads * V) {
        const int64_t n = end - i;
        uint32_t c[2] = {0, 0};
        if (n >= V) {
            const u32x2 w = load8<false>((const uint8_t*)x.avg + i);
            c[0] = w[0];
            c[1] = w[1];
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) c[j / 4] |= (uint32_t)((const uint8_t*)x.avg)[i + j] << (8 * (j % 4));
        }
        const float s = x.avg_scale[i / kAdamBlock];
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float cm = (float)avg_code(c[j / 4], j % 4), cv = sq_code(c[j / 4], j % 4);
            const float r = cv * cv * (1.0f / 65025.0f);   // the square is exact
            v[j] = x.number ? r * r * s : cm * __builtin_fabsf(cm) * (1.0f / 16129.0f) * s;
        }
        store_some<TO, V>((TO*)x.param + i, n, v);
    }
}

}  // namespace dytb
