// block_common.hpp - what the layer norm and attention kernels share: wave
// reductions, 16-byte vector access at element alignment, dtype dispatch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dyt.h"
#include "dyt_math.hpp"

namespace dytb {

using dyt::bf16_t;
using dyt::f16_t;
using dyt::to_f32;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at the alignment of a 2-byte element: the GPU runs global memory
// instructions in unaligned mode, so rows of any length take them.
typedef uint32_t u32x4_m __attribute__((ext_vector_type(4), aligned(2)));

template <typename T> struct VecOf { static constexpr int n = 16 / (int)sizeof(T); };

template <typename T>
__device__ __forceinline__ void unpack16(u32x4 w, float* out) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            T lo{(uint16_t)(w[i] & 0xffffu)}, hi{(uint16_t)(w[i] >> 16)};
            out[2 * i] = to_f32(lo);
            out[2 * i + 1] = to_f32(hi);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (__is_same(T, bf16_t)) return dyt::pack2_bf16(lo, hi);
    else return dyt::pack2_f16(lo, hi);
}

template <typename T>
__device__ __forceinline__ u32x4 pack16(const float* v) {
    u32x4 w;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
    return w;
}

// An element of a float32, bfloat16 or float16 array chosen at run time
// (parameters, bias tables: read once per workgroup, so not worth a kernel
// instance per type).
__device__ __forceinline__ float load_param(const void* p, int64_t i, int dt) {
    if (dt == DYT_F32) return ((const float*)p)[i];
    if (dt == DYT_BF16) return to_f32(((const bf16_t*)p)[i]);
    return to_f32(((const f16_t*)p)[i]);
}

__device__ __forceinline__ void store_param(void* p, int64_t i, int dt, float v) {
    if (dt == DYT_F32) ((float*)p)[i] = v;
    else if (dt == DYT_BF16) ((bf16_t*)p)[i] = dyt::from_f32<bf16_t>(v);
    else ((f16_t*)p)[i] = dyt::from_f32<f16_t>(v);
}

// Sums over aligned groups of L lanes (L a power of two up to 64), in every
// lane: lane exchanges within 16 by DPP, across 16 and 32 by the row swaps,
// so no LDS traffic. The tree is the same in every lane: equal bits.
template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

__device__ __forceinline__ float swap32_other_sum(float v) {
    const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(
        __float_as_uint(v), __float_as_uint(v), false, false));
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

__device__ __forceinline__ float swap32_max(float v) {
    const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(
        __float_as_uint(v), __float_as_uint(v), false, false));
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

__device__ __forceinline__ float swap16_other_sum(float v) {
    const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(
        __float_as_uint(v), __float_as_uint(v), false, false));
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (L >= 2) v += dpp_mov<0xB1>(v);    // lane ^ 1
    if constexpr (L >= 4) v += dpp_mov<0x4E>(v);    // lane ^ 2
    if constexpr (L >= 8) v += dpp_mov<0x141>(v);   // mirrored within 8
    if constexpr (L >= 16) v += dpp_mov<0x140>(v);  // mirrored within 16
    if constexpr (L >= 32) v = swap16_other_sum(v);
    if constexpr (L >= 64) v = swap32_other_sum(v);
    return v;
}

}  // namespace dytb
