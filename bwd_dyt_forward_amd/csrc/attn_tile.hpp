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
// LDS tiles are row-major, rows of DP elements cut into 16-byte chunks. A read
// of 16 bytes a lane takes 16 rows of one chunk at a time, the transposing
// read 4 neighbouring rows of 4 neighbouring chunks; both should touch each
// of the 64 banks once. For the 16-bit types chunk c of row r is therefore
// stored at c ^ f(r), where f sends 16 rows to 16 different positions and 4
// neighbouring rows to different groups of 4 (measured: no conflicts; with
// one chunk of padding per row instead the transposing reads took four times
// their cycles and the dk/dv kernel 14% longer). Float32 rows, read in single
// words by the second product, are padded by one chunk. The tiles are filled
// by direct-to-LDS loads, which write 1,024 contiguous bytes per wave
// instruction, so each lane asks for the chunk its place belongs to; lanes on
// padding, on columns past D or on rows past the end ask for an offset past
// the buffer descriptor's end, which brings zeros.
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

// ------------------------------------------- tiles and LDS of the instances
// NW waves of a workgroup own 32 rows (dk/dv: keys) each, SL slices of them
// share those and take different parts of each tile of the long axis.
// es: element bytes, dp: padded head dimension.

constexpr int kMaxLds = 160 * 1024;

constexpr int attn_tile_bytes(int es, int dp, int rows) {
    return (rows * (dp * es + (es == 4 ? 16 : 0)) + 1023) / 1024 * 1024;
}

// Forward and dq: keys per tile.
constexpr int attn_tile_rows(int es, int nw, int sl) { return sl > 1 ? 32 * sl : es == 2 && nw > 1 ? 64 : 32; }
constexpr int attn_lds_bytes(int es, int dp, int nw, int sl) {
    return 4 * attn_tile_bytes(es, dp, attn_tile_rows(es, nw, sl));
}

// The dk/dv kernel holds 4 dp / 32 accumulators and its keys' and values'
// fragments. Above dp = 64 that leaves room for one wave per SIMD; with the
// values' fragments in LDS (which has bandwidth to spare) two fit, and hide
// each other's waits. Tiles of 32 rows a slice keep its LDS small.
constexpr bool dkv_vals_in_lds(int es, int dp) { return es == 2 && dp > 64; }
constexpr int attn_dkv_tile_rows(int es, int dp, int nw, int sl) {
    return sl > 1 ? 32 * sl : nw > 1 && es == 2 && dp <= 64 ? 64 : 32;
}
constexpr int attn_dkv_lds_bytes(int es, int dp, int nw, int sl) {
    const int rows = attn_dkv_tile_rows(es, dp, nw, sl);
    return 4 * attn_tile_bytes(es, dp, rows) + 16 * (rows > 64 ? rows : 64) +
           (dkv_vals_in_lds(es, dp) ? nw * (dp / 16) * 1024 : 0);
}

// Waves per SIMD that an instance's registers have to leave room for; instances
// that need less, such as the forward's at dp <= 64, hold more. (Asking for three
// or four at dp <= 64 makes some spill: forward 62 -> 82 us at 4 x 16 heads of
// 2,048 with four, dk/dv 105 -> 187 us at 8 x 16 heads of 1,024 with three.)
constexpr int attn_waves(int es) { return es == 4 ? 1 : 2; }

// dq's second walk, see attn_bwd.hpp.
constexpr int kRefineKeys = 256;

// LDS floats of the bias gradient: each wave's scratch for one tile's
// diagonals and its sums by relative position.
constexpr int kDiagPitch = 33;
constexpr int kDiagFloats = 32 * kDiagPitch;
constexpr int dbias_floats(int entries, int waves) { return waves * (kDiagFloats + entries); }

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
    static constexpr bool xored = sizeof(T) == 2;
    static constexpr int cpr = DP * (int)sizeof(T) / 16;   // chunks per row
    static constexpr int chunks = xored ? cpr : cpr + 1;
    static constexpr int pitch = chunks * 16;
    // Chunk bits that f changes; the row pitch is a multiple of 16 (mask + 1).
    static constexpr int mask = !xored ? 0 : cpr == 16 ? 15 : cpr == 8 ? 7 : 3;

    // Bytes of a tile: whole wave instructions.
    static constexpr int bytes(int rows) { return attn_tile_bytes((int)sizeof(T), DP, rows); }

    // f(row). The banks hold 16 chunks: one row of 16 chunks, two of 8, four
    // of 4, and rows of 12 start at 0, 12, 8, 4 in turn.
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (!xored) return 0;
        else if constexpr (cpr == 16) return ((row & 3) << 2) | ((row >> 2) & 3);
        else if constexpr (cpr == 8) return ((row & 2) << 1) | ((row >> 2) & 3);
        else return (row >> 2) & 3;
    }

    // A lane's base for row_frag and col_frag; at() moves it to another chunk.
    static __device__ __forceinline__ int row_lane(int lane) {
        const int row = lane & 31, h = lane >> 5;
        if constexpr (xored) return row * pitch + ((h ^ swizzle(row)) << 4);
        else return row * pitch + h * 32;
    }
    static __device__ __forceinline__ int col_lane(int lane, int more) {
        if constexpr (xored) {
            // 16 lanes of the transposing read give 4 rows of 16 columns
            const int r = lane & 15, g = lane >> 4;
            const int row = 4 * (g >> 1) + (r >> 2) + more;
            return row * pitch + (((((g & 1) << 1) | ((r & 3) >> 1)) ^ swizzle(row)) << 4) + (r & 1) * 8;
        } else {
            return 4 * (lane >> 5) * pitch + (lane & 31) * 4 + more * pitch;
        }
    }
    // chunk: a multiple of what the lane's own chunk number stays below.
    static __device__ __forceinline__ int at(int base, int chunk) {
        return (base ^ ((chunk & mask) << 4)) + ((chunk & ~mask) << 4);
    }

    // Contraction slots ds * 16 .. + 15 of row n * 32 + lane % 32 of the tile
    // at byte `tile`.
    static __device__ __forceinline__ Frag<T> row_frag(int lane_at, int tile, int n, int ds) {
        if constexpr (xored) {
            return *(const u32x4*)(smem + at(lane_at, ds * 2) + (tile + n * 32 * pitch));
        } else {
            const char* p = smem + lane_at + (tile + n * 32 * pitch + ds * 64);
            const f32x4 lo = *(const f32x4*)p, hi = *(const f32x4*)(p + 16);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // Column dt * 32 + lane % 32, rows row0 .. row0 + 15 in accumulator order;
    // row0 is a multiple of 16. lane_at: col_lane(lane, 0), lane_at8: (lane, 8).
    static __device__ __forceinline__ Frag<T> col_frag(int lane_at, int lane_at8, int tile, int row0, int dt) {
        if constexpr (xored) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_ptr)(smem + at(lane_at, dt * 4) + (tile + row0 * pitch)));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_ptr)(smem + at(lane_at8, dt * 4) + (tile + row0 * pitch)));
            const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
            return u32x4{x[0], x[1], y[0], y[1]};
        } else {
            const char* p = smem + lane_at + (tile + row0 * pitch + dt * 128);
            f32x8 f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = *(const float*)(p + (8 * (j / 4) + (j % 4)) * pitch);
            return f;
        }
    }
};

// Calls step(buffer, position) for begin, begin + by, .. below end, the
// buffer 0 and 1 in turn as compile-time constants (LDS addresses then differ
// by the instructions' own offsets).
template <int V> struct Int { static constexpr int value = V; };

template <typename F>
__device__ __forceinline__ void alternate(int begin, int end, int by, F&& step) {
    for (int x = begin; x < end; x += by) {
        step(Int<0>{}, x);
        x += by;
        if (x >= end) break;
        step(Int<1>{}, x);
    }
}

// One 16-byte load per lane straight into LDS at `lds` + 16 lane. The wait
// states stand between what may have written the operands and the load: one
// after m0, five after a vector instruction that wrote a descriptor register
// (a read lane, a restored spill), which the compiler does not add for asm.
__device__ __forceinline__ void load_to_lds16(const i32x4& rsrc, uint32_t lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(rsrc) : "memory", "m0");
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
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :: "s"(lds_address(lds)), "v"(off), "s"(descriptor(base)) : "memory", "m0");
}

// Waits for this wave's direct-to-LDS loads; the barrier that follows makes
// them everyone's.
__device__ __forceinline__ void loads_landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Rows of a [S, H, D] slice, `pack` heads to a position: row r is position
// r / pack, head r % pack.
struct Rows {
    const char* base;
    int64_t ss, hs;   // bytes
    int32_t pack;
};

constexpr uint32_t kOutside = 0x80000000u;

// A tensor's rows on their way through LDS tiles of ROWS rows, by NW waves:
// `take` rows to a tile (whole positions; the rest of the tile is zeros), so
// that a lane's offsets are the same for every tile and only the base moves.
// VEC: 16-byte loads straight into LDS (aligned, a tile's offsets in 31
// bits); otherwise element by element.
template <typename T, int DP, int ROWS, int NW, bool VEC> struct Stream {
    typedef Tile<T, DP> TL;
    static constexpr int slots = ROWS * TL::chunks;
    static constexpr int instrs = (slots + 63) / 64;
    static constexpr int NI = (instrs + NW - 1) / NW;
    const char* base;
    int64_t step;
    uint32_t off[VEC ? NI : 1];

    // Slot i of this lane: wave instruction i * NW + wave.
    static __device__ __forceinline__ void place(int wave, int lane, int i, int& row, int& chunk) {
        const int slot = (i * NW + wave) * 64 + lane;
        row = slot / TL::chunks;
        chunk = (slot - row * TL::chunks) ^ TL::swizzle(row);
    }

    __device__ __forceinline__ void start(const Rows& w, int position, int take, int D, int wave, int lane) {
        base = w.base + (int64_t)position * w.ss;
        step = (int64_t)(take / w.pack) * w.ss;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                int row, chunk;
                place(wave, lane, i, row, chunk);
                const int di = row / w.pack, g = row - di * w.pack;
                const uint32_t at = (uint32_t)di * (uint32_t)w.ss + (uint32_t)g * (uint32_t)w.hs + (uint32_t)chunk * 16u;
                off[i] = row < take && chunk < TL::cpr && chunk * (16 / (int)sizeof(T)) < D ? at : kOutside;
            }
        }
    }

    // The next tile's rows into the tile at `lds`; `left` of them are there,
    // the others, and with SKIP the first `skip`, come out as zeros.
    template <bool SKIP = false>
    __device__ __forceinline__ void fetch(int lds, const Rows& w, int left, int take, int D, int wave, int lane,
                                          int skip = 0) {
        if constexpr (VEC) {
            const i32x4 rsrc = descriptor(base);
            const uint32_t to = lds_address(lds + wave * 1024);
            if (left >= take && (!SKIP || skip <= 0)) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (instrs % NW == 0 || i * NW + wave < instrs) load_to_lds16(rsrc, to + i * NW * 1024, off[i]);
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    int row, chunk;
                    place(wave, lane, i, row, chunk);
                    const uint32_t at = (!SKIP || row >= skip) && row < left ? off[i] : kOutside;
                    if (instrs % NW == 0 || i * NW + wave < instrs) load_to_lds16(rsrc, to + i * NW * 1024, at);
                }
            }
        } else {
            constexpr int N = 16 / (int)sizeof(T);
            for (int x = (int)threadIdx.x; x < ROWS * TL::cpr; x += NW * 64) {
                const int row = x / TL::cpr, chunk = x - row * TL::cpr;
                const int di = row / w.pack, g = row - di * w.pack;
                const T* p = (const T*)(base + (int64_t)di * w.ss + (int64_t)g * w.hs);
                T e[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int d = chunk * N + k;
                    e[k] = T{};
                    if ((!SKIP || row >= skip) && row < min(left, take) && d < D) e[k] = p[d];
                }
                __builtin_memcpy(smem + lds + row * TL::pitch + ((chunk ^ TL::swizzle(row)) << 4), e, 16);
            }
        }
        base += step;
    }
};

// Fragment of columns d0 .. d0 + 7 of a row in global memory; zeros past D
// and for rows that are not there.
template <typename T, bool VEC>
__device__ __forceinline__ Frag<T> global_frag(const char* row, int d0, int D, bool there) {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
        f = u32x4{0, 0, 0, 0};
        if (there) {
            if constexpr (VEC) {
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
        if constexpr (VEC) {
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
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void store_acc(char* row, const f32x16* acc, float mul, int D, bool there, int h) {
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
                    if constexpr (VEC) {
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
                        if constexpr (VEC) {
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

// Adds up the accumulators of the SL slices (waves that hold the same rows of
// the output and took different parts of the long axis) in slice order, in
// the waves of slice `owner`. Boxes of 16 bytes per lane at the start of LDS,
// whose tiles every wave is done with after the first barrier.
template <int DP, int NW, int SL>
__device__ __forceinline__ void join_slices(f32x16* acc, int g, int sl, int owner, int lane) {
    __syncthreads();
    char* box = smem + (g * (DP / 8) * 64 + lane) * 16;
    constexpr int step = NW * (DP / 8) * 1024;
    if (sl != owner) {
        char* to = box + (sl < owner ? sl : sl - 1) * step;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *(f32x4*)(to + (dt * 4 + k) * 1024) =
                    f32x4{acc[dt][4 * k], acc[dt][4 * k + 1], acc[dt][4 * k + 2], acc[dt][4 * k + 3]};
    }
    __syncthreads();
    if (sl == owner) {
#pragma unroll
        for (int x = 0; x < SL - 1; ++x)
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x4 v = *(const f32x4*)(box + x * step + (dt * 4 + k) * 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[dt][4 * k + j] += v[j];
                }
    }
}

// float32 rows of DP elements in the workspace.
template <int DP>
__device__ __forceinline__ void store_part(float* row, const f32x16* acc, float mul, bool there, int h) {
    store_acc<float, DP, true>((char*)row, acc, mul, DP, there, h);
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
    float* tpart;          // backward: [units * blocks * nsplit][entries]
    int32_t B, Sq, Sk, Hq, Hkv, D, G;
    int32_t pack, units;   // units = B * Hq / pack
    int32_t blocks, nsplit, per_split;   // row (or key) blocks per unit, splits of the other axis
    int32_t together, zigzag;            // units an XCD takes at a time and how, see find_work
    int32_t causal, table_dt, buckets;
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
    // a second sum of the same shape (dv beside dk), or null
    const float* part2;
    char* out2;
    Strides os2;
};

struct Work {
    int u, block, split, b, head, kv, start, len;
    int64_t flat;   // index of (u, split, block)
};

// Workgroup -> (unit, split, block). Workgroups go round the 8 XCDs in turn,
// each of which has an L2 of its own: of every 8 units (neighbouring heads,
// of about the same length) each XCD takes one whole, so that the blocks
// that read one key head's keys and values share an L2 and a batch of ragged
// lengths still spreads evenly. Units beyond a multiple of 8, and units of
// one block, whose keys nobody else reads, go round block by block.
//
// Under a causal mask the blocks' work falls from one end to the other
// (`heavy_last`: the last block has most). An XCD then takes `together` of its
// units at a time, the heaviest blocks of all of them first, and where a CU
// holds several workgroups (`zigzag`) every second row of 32 (its CUs) the
// other way, so that those of a CU add up to the same work: with one unit after
// the other, each heaviest first, some CUs got four of the longest blocks and
// others four of the shortest (forward of 64 units of 16 blocks, D = 64: 87 us,
// now 62). A CU with one workgroup at a time takes the heaviest left when it
// is free (dk/dv of 16 units of 32 blocks, D = 128: 691 us with the rows
// turned, 655 without).
__device__ __forceinline__ bool find_work(const AttnArgs& a, Work& w, bool heavy_last) {
    const int per_unit = a.blocks * a.nsplit;
    const int64_t bid = blockIdx.x;
    const int whole = a.blocks > 1 ? a.units / 8 * 8 : 0;
    int rem;
    if (bid < (int64_t)whole * per_unit) {
        const int i = (int)(bid >> 3);
        const int each = a.together * per_unit, group = i / each;
        const int n = min(a.together, whole / 8 - group * a.together);   // units of this group
        int r = i - group * each;
        if (a.zigzag) {
            const int row = r >> 5;
            if ((row & 1) && row * 32 + 32 <= n * per_unit) r = row * 32 + 31 - (r & 31);
        }
        rem = r / n;
        w.u = (group * a.together + (r - rem * n)) * 8 + (int)(bid & 7);
    } else {
        const int i = (int)(bid - (int64_t)whole * per_unit);
        const int k = i / per_unit;
        w.u = whole + k;
        rem = i - k * per_unit;
    }
    if (w.u >= a.units) return false;
    if (a.causal) {
        w.block = rem / a.nsplit;
        w.split = rem - w.block * a.nsplit;
        if (heavy_last) w.block = a.blocks - 1 - w.block;
    } else {
        w.split = rem / a.blocks;
        w.block = rem - w.split * a.blocks;
    }
    w.flat = (int64_t)w.u * per_unit + w.split * a.blocks + w.block;
    const int hu = a.Hq / a.pack;
    w.b = w.u / hu;
    w.head = (w.u - w.b * hu) * a.pack;
    w.kv = w.head / a.G;
    w.len = a.Sk;
    if (a.lens) w.len = min(max(a.lens[w.b], 0), a.Sk);
    // positions beyond +-2^30 see and measure what those do (Sq, Sk <= 2^28)
    w.start = a.Sk - a.Sq;
    if (a.starts) w.start = min(max(a.starts[w.b], -(1 << 30)), 1 << 30);
    return true;
}

// The bias by relative position, in log2 units, in LDS at float index
// rel + reach + kPad for rel within reach + kPad of 0. A 32 x 32 tile that
// touches (-reach, reach) stays inside; all others have one bias.
constexpr int kPad = 64;
__device__ __forceinline__ int bias_entries(const Borders& o) { return 2 * (o.reach + kPad); }

// Entries [lo, hi) of bucket t.
__device__ __forceinline__ void bucket_range(const Borders& o, int t, int& lo, int& hi) {
    const int mid = o.reach + kPad;   // entry of position 0
    const bool later = t >= o.n;      // bidirectional: keys after the query
    const int u = later ? t - o.n : t;
    const int from = o.at[u], to = o.at[min(u + 1, o.n - 1)];
    const bool last = u + 1 == o.n;
    if (later) {
        lo = mid + max(from, 1);   // distance 0 is the other direction's
        hi = last ? 2 * mid : mid + to;
    } else {
        lo = last ? 0 : mid - to + 1;
        hi = t == 0 && !o.bidirectional ? 2 * mid : mid - from + 1;   // every later key
    }
}

// Eight lanes per bucket write its run of entries (a search per entry through
// the borders took 6 us of a small problem's kernel; a single lane per
// bucket is held up by the longest run).
__device__ __forceinline__ void fill_bias(float* lds, const AttnArgs& a, int head) {
    for (int t = (int)threadIdx.x / 8; t < a.buckets; t += (int)blockDim.x / 8) {
        const float x = load_param(a.table, (int64_t)t * a.Hq + head, a.table_dt) * kLog2e;
        int lo, hi;
        bucket_range(a.borders, t, lo, hi);
        for (int i = lo + ((int)threadIdx.x & 7); i < hi; i += 8) lds[i] = x;
    }
}

__device__ __forceinline__ int acc_row(int i, int h) { return 8 * (i / 4) + 4 * h + (i % 4); }

}  // namespace dytb
