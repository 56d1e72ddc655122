// attn_tile.hpp - matrix-core fragments and LDS tiles of the attention
// kernels (gfx950).
//
// Every product is built from 32 x 32 accumulator tiles: lane l holds column
// n = l % 32 and, in register i = 0..15, row 8 (i / 4) + 4 (l / 32) + i % 4.
// A fragment is 8 elements of a 16-long contraction: half h = l / 32 of the
// lanes supplies slots 8 h .. 8 h + 7 of row (A) or column (B) l % 32. For
// the 16-bit types that is one 32x32x16 instruction; for float32 eight
// 32x32x2 ones, slot j of both halves together, so all kernels are written
// once.
//
// The second product of each pair contracts over the accumulator's rows. Its
// B fragments need no exchange between lanes: registers 8 s .. 8 s + 7 of a
// lane are already one fragment, whose slot j of half h stands for row
// 16 s + 8 (j / 4) + 4 h + j % 4. The A side is read in that same order
// (load_col_frag), by the LDS's transposing read for the 16-bit types.
//
// LDS tiles are row-major, rows of DP elements cut into 16-byte chunks; the
// chunk at column position c of row r is stored at position c ^ f(r)
// (swizzle()), so that the 16 rows one read instruction covers at a time
// fall on different banks without padding: the tiles are filled by
// direct-to-LDS loads, which write 1,024 contiguous bytes per wave
// instruction. Columns past D and rows past the end come out as zeros: their
// lanes ask for an offset past the buffer descriptor's end.
#pragma once

#include "block_common.hpp"
#include "dyt_block.h"

namespace dytb {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

extern __shared__ __attribute__((aligned(1024))) char smem[];

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLn2 = 0x1.62e43p-1f;

template <typename T> struct FragOf { typedef u32x4 type; };
template <> struct FragOf<float> { typedef f32x8 type; };
template <typename T> using Frag = typename FragOf<T>::type;

template <typename T>
__device__ __forceinline__ f32x16 mma(const Frag<T>& a, const Frag<T>& b, f32x16 c) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
        return c;
    } else if constexpr (__is_same(T, bf16_t)) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
}

// Eight accumulator registers as a fragment (rounded to T: the operands of
// the 16-bit matrix instructions are 16-bit, and the error of the rounding,
// half a step of each probability, averages out over the keys).
template <typename T>
__device__ __forceinline__ Frag<T> pack_frag(const float* v) {
    Frag<T> f;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
    }
    return f;
}

template <typename T, int DP> struct Tile {
    static constexpr int row_bytes = DP * (int)sizeof(T);
    static constexpr int cpr = row_bytes / 16;   // chunks per row

    // f(row): see the file comment. The 256 bytes of the 64 banks hold
    // 16 / cpr rows (or one row, or a part); 16 consecutive rows get 16
    // different positions, 4 consecutive rows different 32-byte pairs.
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (sizeof(T) == 2) {
            if constexpr (cpr == 16) { const int u = row & 15; return ((u & 7) << 1) | (u >> 3); }
            else if constexpr (cpr == 8) { const int u = (row >> 1) & 7; return ((u & 3) << 1) | (u >> 2); }
            else { const int u = (row >> 2) & 3; return ((u & 1) << 1) | (u >> 1); }
        } else {
            if constexpr (cpr % 16 == 0) return row & 15;
            else return (row >> 1) & 7;
        }
    }

    static __device__ __forceinline__ int offset(int row, int chunk) {
        return row * row_bytes + ((chunk ^ swizzle(row)) << 4);
    }

    // Contraction slots ds * 16 .. + 15 of one row.
    static __device__ __forceinline__ Frag<T> row_frag(int tile, int row, int ds, int h) {
        if constexpr (sizeof(T) == 2) {
            return *(const u32x4*)(smem + tile + offset(row, ds * 2 + h));
        } else {
            const f32x4 lo = *(const f32x4*)(smem + tile + offset(row, ds * 4 + h * 2));
            const f32x4 hi = *(const f32x4*)(smem + tile + offset(row, ds * 4 + h * 2 + 1));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // Column dt * 32 + lane % 32, rows row0 .. row0 + 15 in accumulator order.
    static __device__ __forceinline__ Frag<T> col_frag(int tile, int row0, int dt, int lane) {
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            const int r = lane & 15, g = lane >> 4;
            const int row = 4 * (g >> 1) + (r >> 2);
            const int chunk = dt * 4 + (g & 1) * 2 + ((r & 3) >> 1);
            const int at = (r & 1) * 8;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_ptr)(smem + tile + row0 * row_bytes + offset(row, chunk) + at));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_ptr)(smem + tile + row0 * row_bytes + offset(row + 8, chunk) + at));
            const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
            return u32x4{x[0], x[1], y[0], y[1]};
        } else {
            const int c = dt * 32 + (lane & 31), h = lane >> 5;
            f32x8 f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = row0 + 8 * (j / 4) + 4 * h + (j % 4);
                f[j] = *(const float*)(smem + tile + offset(row, c >> 2) + (c & 3) * 4);
            }
            return f;
        }
    }
};

// One 16-byte load per lane straight into LDS at `lds` + 16 lane. One wait
// state between the write of m0 and its use.
__device__ __forceinline__ void load_to_lds16(const i32x4& rsrc, uint32_t lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(rsrc) : "memory");
}

__device__ __forceinline__ i32x4 descriptor(const void* base) {
    const uint64_t addr = (uint64_t)base;
    i32x4 rsrc;
    rsrc[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)addr);
    rsrc[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(addr >> 32) & 0xffffu));
    rsrc[2] = 0x7fffffff;
    rsrc[3] = 0x00020000;
    return rsrc;
}

__device__ __forceinline__ uint32_t lds_address(int at) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem + (uint32_t)at;
}

// 4 bytes per lane to `lds` + 4 lane.
__device__ __forceinline__ void load_to_lds4(const void* base, int lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :: "s"(lds_address(lds)), "v"(off), "s"(descriptor(base)) : "memory");
}

// Waits for this wave's direct-to-LDS loads; the barrier that follows makes
// them everyone's.
__device__ __forceinline__ void loads_landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Rows of a [S, H, D] slice, `pack` heads to a position: row r is position
// r / pack, head r % pack. magic = ceil(2^20 / pack) divides numbers below
// 2^20 / pack exactly.
struct Rows {
    const char* base;
    int64_t ss, hs;   // bytes
    int32_t pack, magic;
    int32_t vec;      // 16-byte accesses allowed, strides fit 32-bit offsets
};

__device__ __forceinline__ int div_pack(int r, const Rows& w) {
    return w.pack == 1 ? r : (int)(((uint32_t)r * (uint32_t)w.magic) >> 20);
}

constexpr uint32_t kOutside = 0x80000000u;

// Rows row0 .. row0 + ROWS - 1 (zeros from `end` on) into the tile at `lds`,
// by NW waves. i0 = row0 / pack, rem0 = row0 % pack.
template <typename T, int DP, int ROWS, int NW>
__device__ __forceinline__ void stage(int lds, const Rows& w, int row0, int i0, int rem0, int end, int D) {
    typedef Tile<T, DP> TL;
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const char* base = w.base + (int64_t)i0 * w.ss;
    if (w.vec) {
        constexpr int NI = ROWS * TL::cpr / 64 / NW;
        static_assert(NI * 64 * NW == ROWS * TL::cpr, "whole wave instructions");
        const i32x4 rsrc = descriptor(base);
        const uint32_t ss = (uint32_t)w.ss, hs = (uint32_t)w.hs;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int slot = (wave * NI + i) * 64 + lane;
            const int lr = slot / TL::cpr;
            const int chunk = (slot % TL::cpr) ^ TL::swizzle(lr);
            const int di = div_pack(rem0 + lr, w);
            const int g = rem0 + lr - di * w.pack;
            uint32_t off = (uint32_t)di * ss + (uint32_t)g * hs + (uint32_t)chunk * 16u;
            off = (row0 + lr < end && chunk * (16 / (int)sizeof(T)) < D) ? off : kOutside;
            load_to_lds16(rsrc, lds_address(lds + (wave * NI + i) * 1024), off);
        }
    } else {
        constexpr int VEC = 16 / (int)sizeof(T);
        for (int slot = (int)threadIdx.x; slot < ROWS * TL::cpr; slot += NW * 64) {
            const int lr = slot / TL::cpr;
            const int chunk = (slot % TL::cpr) ^ TL::swizzle(lr);
            const int di = div_pack(rem0 + lr, w);
            const int g = rem0 + lr - di * w.pack;
            const T* p = (const T*)(base + (int64_t)di * w.ss + (int64_t)g * w.hs);
            T e[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int d = chunk * VEC + k;
                e[k] = T{};
                if (row0 + lr < end && d < D) e[k] = p[d];
            }
            __builtin_memcpy(smem + lds + slot * 16, e, 16);
        }
    }
}

// Fragment of columns d0 .. d0 + 7 of a row in global memory; zeros past D
// and for rows that are not there.
template <typename T>
__device__ __forceinline__ Frag<T> global_frag(const char* row, int d0, int D, bool vec, bool there) {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
        f = u32x4{0, 0, 0, 0};
        if (there) {
            if (vec) {
                if (d0 < D) f = *(const u32x4*)(row + d0 * 2);
            } else {
                const uint16_t* p = (const uint16_t*)row;
                uint16_t e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[j] = 0;
                    if (d0 + j < D) e[j] = p[d0 + j];
                }
                __builtin_memcpy(&f, e, 16);
            }
        }
    } else {
        const float* p = (const float*)row;
        if (vec) {
            f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
            if (there && d0 < D) lo = *(const f32x4*)(p + d0);
            if (there && d0 + 4 < D) hi = *(const f32x4*)(p + d0 + 4);
            f = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j] = 0.0f;
                if (there && d0 + j < D) f[j] = p[d0 + j];
            }
        }
    }
    return f;
}

template <typename T>
__device__ __forceinline__ float frag_dot(const Frag<T>& a, const Frag<T>& b) {
    float s = 0.0f;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(a[j], b[j], s);
    } else {
        float x[8], y[8];
        unpack16<T>(a, x);
        unpack16<T>(b, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(x[j], y[j], s);
    }
    return s;
}

// Writes acc[DP / 32] (columns of the output in the accumulator's rows, one
// output row per lane column) times `mul` to the row at `row`. The two
// halves of the lanes trade 8-byte pieces so that each stores 16 bytes.
template <typename T, int DP>
__device__ __forceinline__ void store_acc(char* row, const f32x16* acc, float mul, int D, bool vec, bool there,
                                          int h) {
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = acc[dt][8 * a + j] * mul;
            if constexpr (sizeof(T) == 2) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
                const u32x2 s0 = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false));
                const u32x2 s1 = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false));
                const u32x4 out = {s0[0], s1[0], s0[1], s1[1]};
                const int d = dt * 32 + a * 16 + 8 * h;
                if (there) {
                    if (vec) {
                        if (d < D) *(u32x4*)(row + d * 2) = out;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (d + j < D) ((uint16_t*)row)[d + j] = (uint16_t)(out[j / 2] >> (16 * (j & 1)));
                    }
                }
            } else {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int d = dt * 32 + a * 16 + b * 8 + 4 * h;
                    if (there) {
                        if (vec) {
                            if (d < D) *(f32x4*)(row + d * 4) = f32x4{v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]};
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (d + j < D) ((float*)row)[d + j] = v[4 * b + j];
                        }
                    }
                }
            }
        }
    }
}

// float32 rows of DP elements in the workspace.
template <int DP>
__device__ __forceinline__ void store_part(float* row, const f32x16* acc, float mul, bool there, int h) {
    store_acc<float, DP>((char*)row, acc, mul, DP, true, there, h);
}

// ------------------------------------------------------------- the problem
struct Borders {
    int32_t n, e, bidirectional, reach;   // reach: smallest distance of the last bucket
    int32_t at[DYT_ATTN_MAX_BUCKETS];
};

struct Strides {
    int64_t b, s, h;   // bytes
};

struct AttnArgs {
    const char *q, *k, *v, *o, *dout;
    char *out, *dq, *dk, *dv;
    Strides qs, ks, vs, os, dos, dqs, dks, dvs;
    float* stats;          // [B, Hq, Sq]
    const int32_t* lens;
    const int32_t* starts;
    const void* table;
    void* dtable;
    float* part;           // partial results, see the kernels
    float* part_ml;
    float* rows;           // backward: [2][B, Hq, Sq]: log2 of the sums, delta
    float* rest;           // backward, dq split: [nsplit][B, Hq, Sq], what delta is off by
    float* tpart;          // backward: [units * blocks * nsplit][buckets]
    int32_t B, Sq, Sk, Hq, Hkv, D, G;
    int32_t pack, magic, units;   // units = B * Hq / pack
    int32_t blocks, nsplit, per_split;   // row (or key) blocks per unit, splits of the other axis
    int32_t causal, table_dt, buckets;
    int32_t vec_q, vec_k, vec_v, vec_o, vec_do, vec_out;   // vec_out: every output
    float scale;
    Borders borders;
};

// The sum of float32 parts, see attn_sum_kernel.
struct SumArgs {
    const float* part;
    int64_t stride;
    int32_t parts;
    char* out;
    Strides os;
    int64_t total;
    int32_t rows, pack, hu, D;
    float* delta;
    const float* rest;
};

struct Work {
    int u, block, split, b, head, kv, start, len;
    int64_t flat;   // index of (u, split, block)
};

// Workgroup -> (unit, split, block). Workgroups go round the 8 XCDs in turn;
// each XCD gets a contiguous run of the work, so the blocks that read one
// key head's keys and values share an L2. Under a causal mask the blocks
// with most to do come first.
__device__ __forceinline__ bool find_work(const AttnArgs& a, Work& w, bool last_first) {
    const int per_unit = a.blocks * a.nsplit;
    const int64_t total = (int64_t)a.units * per_unit;
    const int64_t chunk = (total + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= chunk || t >= total) return false;
    w.flat = t;
    w.u = (int)(t / per_unit);
    const int rem = (int)(t - (int64_t)w.u * per_unit);
    w.split = rem / a.blocks;
    w.block = rem - w.split * a.blocks;
    if (last_first) w.block = a.blocks - 1 - w.block;
    const int hu = a.Hq / a.pack;
    w.b = w.u / hu;
    w.head = (w.u - w.b * hu) * a.pack;
    w.kv = w.head / a.G;
    w.len = a.Sk;
    if (a.lens) w.len = min(max(a.lens[w.b], 0), a.Sk);
    // positions beyond +-2^30 see and measure what those do (Sq, Sk <= 2^29)
    w.start = a.Sk - a.Sq;
    if (a.starts) w.start = min(max(a.starts[w.b], -(1 << 30)), 1 << 30);
    return true;
}

__device__ __forceinline__ int bucket_of(const Borders& o, int rel) {
    int d = max(-rel, 0), first = 0;
    if (o.bidirectional) {
        d = abs(rel);
        first = rel > 0 ? o.n : 0;
    }
    int b = min(d, o.e - 1);
    for (int t = o.e; t < o.n; ++t) b += d >= o.at[t] ? 1 : 0;
    return first + b;
}

// The bias by relative position, in log2 units, in LDS at float index
// rel + reach + kPad for rel within reach + kPad of 0. A 32 x 32 tile that
// touches (-reach, reach) stays inside; all others have one bias.
constexpr int kPad = 64;
constexpr int kColBytes = DYT_ATTN_MAX_BUCKETS * 4;   // LDS for the table's column, before the entries

__device__ __forceinline__ int bias_entries(const Borders& o) { return 2 * (o.reach + kPad); }

// `col` has room for the table's column: one load per bucket, then the
// positions gather from LDS (a dependent global load per position took 6 us
// of a small problem's kernel). Ends in a barrier's need: the caller's next
// barrier makes the entries visible.
__device__ __forceinline__ void fill_bias(float* lds, float* col, const AttnArgs& a, int head) {
    const int n = bias_entries(a.borders);
    for (int x = (int)threadIdx.x; x < a.buckets; x += (int)blockDim.x)
        col[x] = load_param(a.table, (int64_t)x * a.Hq + head, a.table_dt) * kLog2e;
    __syncthreads();
    for (int x = (int)threadIdx.x; x < n; x += (int)blockDim.x)
        lds[x] = col[bucket_of(a.borders, x - a.borders.reach - kPad)];
}

__device__ __forceinline__ int acc_row(int i, int h) { return 8 * (i / 4) + 4 * h + (i % 4); }

}  // namespace dytb
