// embed_kernels.hpp - embedding lookup and its gradient (gfx950).
//
//   y[t] = scale weight[token_t]        dweight[v] (+)= scale sum_{t: token_t = v} dy[t]
//
// Both are copies of rows and bound by HBM: the lookup reads a row and writes
// one for each token, the gradient reads dy once and writes every row of
// dweight once (zeros for tokens that do not occur).
//
// The gradient sorts the tokens with their places (a stable radix sort, 9 bits
// a pass, so that equal tokens stay in the order of their places), cuts the
// sorted list into chunks of equal length, however often a token occurs, and
// sums each chunk's runs of equal tokens in registers. A run that lies within
// its chunk is written to its row at once. One that passes a chunk's border
// leaves a float32 row in the workspace: the part that begins in a chunk in
// that chunk's second row ("tail"), a part that only goes on there in its first
// ("head"); a last kernel adds tail and heads up in order. No atomics on
// floating-point values: the order of every sum is that of the places.
#pragma once

#include "ln_kernels.hpp"

namespace dytb {

constexpr int kRadixBits = 9, kRadix = 1 << kRadixBits;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortTile = 16384;        // tokens of a workgroup where several share a pass
constexpr int64_t kSortOne = 65536;     // up to here one workgroup sorts alone, in one launch
constexpr int kEmbVec = 8;              // columns of a thread

// The token at place t, or V where there is none.
__device__ __forceinline__ uint32_t token_at(const void* tokens, int bits, int64_t t, int64_t V) {
    const int64_t v = bits == 64 ? ((const int64_t*)tokens)[t] : (int64_t)((const int32_t*)tokens)[t];
    return (uint32_t)(v >= 0 && v < V ? v : V);
}

// kEmbVec elements at p, of which n are there; zeros for the rest.
template <typename T>
__device__ __forceinline__ void load_cols(const T* p, int n, float* out) {
    constexpr int W = VecOf<T>::n;
    if (n >= kEmbVec) {
#pragma unroll
        for (int i = 0; i < kEmbVec; i += W) unpack16<T>(*(const u32x4_m*)(p + i), out + i);
    } else {
#pragma unroll
        for (int i = 0; i < kEmbVec; ++i) out[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}

// The same without a branch before the load (load_raw): the loads of several
// rows then wait for nothing between them. `limit`: the tensor's elements, at
// least a vector of them. Lanes that are off load the tensor's first bytes.
template <typename T> struct RawCols { u32x4 w[kEmbVec / VecOf<T>::n]; };

template <typename T>
__device__ __forceinline__ RawCols<T> load_raw_cols(const T* p, int64_t row, int c, int D, int64_t limit, bool on) {
    constexpr int W = VecOf<T>::n;
    RawCols<T> r;
#pragma unroll
    for (int i = 0; i < kEmbVec / W; ++i) r.w[i] = load_raw<T, 0>(p, row, c + i * W, D, limit, on);
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack_cols(const RawCols<T>& r, const T* p, int64_t row, int c, int D, int64_t limit,
                                            bool on, float* out) {
    constexpr int W = VecOf<T>::n;
#pragma unroll
    for (int i = 0; i < kEmbVec / W; ++i) unpack_raw<T>(r.w[i], p, row, c + i * W, D, limit, on, out + i * W);
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_cols(T* p, int n, const float* v) {
    constexpr int W = VecOf<T>::n;
    if (n >= kEmbVec) {
#pragma unroll
        for (int i = 0; i < kEmbVec; i += W) {
            if constexpr (NT) __builtin_nontemporal_store((u32x4_m)pack16<T>(v + i), (u32x4_m*)(p + i));
            else *(u32x4_m*)(p + i) = pack16<T>(v + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kEmbVec; ++i)
            if (i < n) p[i] = dyt::from_f32<T>(v[i]);
    }
}

struct EmbedArgs {
    const void* weight;   // forward
    const void* dy;       // backward
    const void* tokens;
    void* out;            // y or dweight
    uint32_t* keys[2];    // sorted tokens and places, two of each
    uint32_t* places[2];
    uint32_t* counts;     // [kRadix][tiles]
    float* part;          // [chunks][2][D]
    int64_t ldw, ldy;     // pitch of weight or dweight, of y or dy
    int64_t T, V;
    int32_t D;
    int32_t token_bits;
    int32_t tpr;          // threads of a row, a power of two up to 256
    int32_t chunk;        // sorted tokens of a chunk
    int32_t chunks;
    int32_t col_tiles;    // of tpr * kEmbVec columns
    int32_t sum_wgs;      // workgroups that sum; the rest write zero rows
    int32_t accumulate;
    float scale;
};

// ----------------------------------------------------------------- lookup
// U rows of a thread at a time: their tokens, then their loads. U = 1: also for
// a weight of fewer elements than a vector.
template <typename TW, typename TY, int U>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedArgs a) {
    const int64_t limit = (a.V - 1) * a.ldw + a.D;
    const TW* wp = (const TW*)a.weight;
    const int t = (int)threadIdx.x & (a.tpr - 1), g = (int)threadIdx.x / a.tpr, groups = 256 / a.tpr;
    const int64_t step = (int64_t)gridDim.x * groups * U;
    for (int64_t base = (int64_t)blockIdx.x * groups * U + g; base < a.T; base += step) {
        uint32_t tok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t m = base + u * groups;
            tok[u] = m < a.T ? token_at(a.tokens, a.token_bits, m, a.V) : (uint32_t)a.V;
        }
        for (int c = t * kEmbVec; c < a.D; c += a.tpr * kEmbVec) {
            RawCols<TW> raw[U];
            if constexpr (U > 1) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    raw[u] = load_raw_cols<TW>(wp, (int64_t)tok[u] * a.ldw, c, a.D, limit, tok[u] < (uint32_t)a.V);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t m = base + u * groups;
                const bool on = tok[u] < (uint32_t)a.V;
                const int64_t row = (int64_t)tok[u] * a.ldw;
                float w[kEmbVec];
                if constexpr (U > 1) unpack_cols<TW>(raw[u], wp, row, c, a.D, limit, on, w);
                else load_cols<TW>(wp + (on ? row + c : 0), on ? a.D - c : 0, w);
#pragma unroll
                for (int i = 0; i < kEmbVec; ++i) w[i] = on ? w[i] * a.scale : 0.0f;
                if (m < a.T) store_cols<TY>((TY*)a.out + m * a.ldy + c, a.D - c, w);
            }
        }
    }
}

// ------------------------------------------------------------------- sort
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Lanes of the wave whose digit is this lane's, among those that are on.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool on) {
    uint64_t same = __ballot(on);
#pragma unroll
    for (int b = 0; b < kRadixBits; ++b) {
        const uint64_t ones = __ballot((digit >> b) & 1);
        same &= ((digit >> b) & 1) ? ones : ~ones;
    }
    return same;
}

// The key and place that pass `pass` reads at i.
__device__ __forceinline__ uint32_t sort_key(const EmbedArgs& a, int pass, int64_t i) {
    return pass ? a.keys[pass & 1][i] : token_at(a.tokens, a.token_bits, i, a.V);
}

// Counts of the digits of this wave's tokens [lo, hi).
__device__ __forceinline__ void count_digits(const EmbedArgs& a, int pass, int64_t lo, int64_t hi, uint32_t* cnt) {
    const int lane = (int)threadIdx.x & 63;
    for (int64_t i = lo + lane; i < hi; i += 64)
        atomicAdd(&cnt[(sort_key(a, pass, i) >> (pass * kRadixBits)) & (kRadix - 1)], 1u);
}

// Moves this wave's tokens [lo, hi) to their places; cnt[digit]: the place of
// the wave's next token of that digit.
__device__ __forceinline__ void scatter_digits(const EmbedArgs& a, int pass, int64_t lo, int64_t hi, uint32_t* cnt) {
    const int lane = (int)threadIdx.x & 63;
    uint32_t* to_key = a.keys[(pass + 1) & 1];
    uint32_t* to_place = a.places[(pass + 1) & 1];
    for (int64_t at = lo; at < hi; at += 64) {
        const int64_t i = at + lane;
        const bool on = i < hi;
        const uint32_t key = on ? sort_key(a, pass, i) : 0u;
        const uint32_t place = on ? (pass ? a.places[pass & 1][i] : (uint32_t)i) : 0u;
        const uint32_t digit = (key >> (pass * kRadixBits)) & (kRadix - 1);
        const uint64_t same = same_digit(digit, on);
        const uint64_t below = same & ((1ull << lane) - 1);
        const uint32_t first = on ? cnt[digit] : 0u;
        wave_fence();   // every lane has read before the first of each digit writes
        if (on && below == 0) cnt[digit] = first + (uint32_t)__popcll(same);
        wave_fence();
        if (on) {
            const uint32_t to = first + (uint32_t)__popcll(below);
            to_key[to] = key;
            to_place[to] = place;
        }
    }
}

// The wave's part of the tokens [lo, hi).
__device__ __forceinline__ void wave_part(int64_t lo, int64_t hi, int64_t& from, int64_t& to) {
    const int64_t per = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    from = min(lo + ((int64_t)threadIdx.x >> 6) * per, hi);
    to = min(from + per, hi);
}

// Exclusive sums over the workgroup's values in thread order.
__device__ __forceinline__ uint32_t exclusive_sum(uint32_t v, uint32_t* waves) {
    const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();   // the sums before have been read
    if (lane == 63) waves[w] = s;
    __syncthreads();
    uint32_t before = 0;
    for (int k = 0; k < w; ++k) before += waves[k];
    return before + s - v;
}

// All passes by one workgroup.
__global__ __launch_bounds__(kSortThreads) void embed_sort_one_kernel(EmbedArgs a, int passes) {
    __shared__ uint32_t cnt[kSortWaves][kRadix];
    __shared__ uint32_t sums[kSortWaves];
    int64_t lo, hi;
    wave_part(0, a.T, lo, hi);
    for (int pass = 0; pass < passes; ++pass) {
        for (int i = (int)threadIdx.x; i < kSortWaves * kRadix; i += kSortThreads) cnt[0][i] = 0;
        __syncthreads();
        count_digits(a, pass, lo, hi, cnt[threadIdx.x >> 6]);
        __syncthreads();
        const int d = (int)threadIdx.x;
        uint32_t total = 0;
        if (d < kRadix)
            for (int w = 0; w < kSortWaves; ++w) total += cnt[w][d];
        uint32_t at = exclusive_sum(total, sums);
        if (d < kRadix)
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t n = cnt[w][d];
                cnt[w][d] = at;
                at += n;
            }
        __syncthreads();
        scatter_digits(a, pass, lo, hi, cnt[threadIdx.x >> 6]);
        __threadfence_block();
        __syncthreads();
    }
}

// One pass by many workgroups: counts of each tile, their sums in the order
// (digit, tile), and the moves.
__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedArgs a, int pass) {
    __shared__ uint32_t cnt[kRadix];
    if (threadIdx.x < kRadix) cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * kSortTile, hi = min(lo + kSortTile, a.T);
    int64_t from, to;
    wave_part(lo, hi, from, to);
    count_digits(a, pass, from, to, cnt);
    __syncthreads();
    if (threadIdx.x < kRadix) a.counts[(int64_t)threadIdx.x * gridDim.x + blockIdx.x] = cnt[threadIdx.x];
}

__global__ __launch_bounds__(kSortThreads) void embed_scan_kernel(uint32_t* counts, int64_t n) {
    __shared__ uint32_t sums[kSortWaves];
    const int64_t per = (n + kSortThreads - 1) / kSortThreads;
    const int64_t lo = min((int64_t)threadIdx.x * per, n), hi = min(lo + per, n);
    uint32_t s = 0;
    for (int64_t i = lo; i < hi; ++i) s += counts[i];
    uint32_t at = exclusive_sum(s, sums);
    for (int64_t i = lo; i < hi; ++i) {
        const uint32_t c = counts[i];
        counts[i] = at;
        at += c;
    }
}

__global__ __launch_bounds__(kSortThreads) void embed_scatter_kernel(EmbedArgs a, int pass) {
    __shared__ uint32_t cnt[kSortWaves][kRadix];
    const int64_t lo = (int64_t)blockIdx.x * kSortTile, hi = min(lo + kSortTile, a.T);
    int64_t from, to;
    wave_part(lo, hi, from, to);
    for (int i = (int)threadIdx.x; i < kSortWaves * kRadix; i += kSortThreads) cnt[0][i] = 0;
    __syncthreads();
    count_digits(a, pass, from, to, cnt[threadIdx.x >> 6]);
    __syncthreads();
    const int d = (int)threadIdx.x;
    if (d < kRadix) {
        uint32_t at = a.counts[(int64_t)d * gridDim.x + blockIdx.x];
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t n = cnt[w][d];
            cnt[w][d] = at;
            at += n;
        }
    }
    __syncthreads();
    scatter_digits(a, pass, from, to, cnt[threadIdx.x >> 6]);
}

// ------------------------------------------------------------------- sums
template <typename TW>
__device__ __forceinline__ void put_row(const EmbedArgs& a, uint32_t key, int c, const float* acc) {
    TW* p = (TW*)a.out + (int64_t)key * a.ldw + c;
    float v[kEmbVec];
    if (a.accumulate) {
        load_cols<TW>(p, a.D - c, v);
#pragma unroll
        for (int i = 0; i < kEmbVec; ++i) v[i] = __builtin_fmaf(acc[i], a.scale, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kEmbVec; ++i) v[i] = acc[i] * a.scale;
    }
    store_cols<TW>(p, a.D - c, v);
}

// Sums of the runs of chunks, tpr threads to a chunk and column tile, U rows
// of dy on their way (U = 1: also for a dy of fewer elements than a vector); and (workgroups from sum_wgs on, 256 rows each) zeros
// for the rows of tokens that do not occur.
template <typename TY, typename TW, int U>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedArgs a, int sorted) {
    const uint32_t* keys = a.keys[sorted];
    const uint32_t V = (uint32_t)a.V;
    if ((int)blockIdx.x >= a.sum_wgs) {
        __shared__ uint8_t absent[256];
        const int64_t v0 = (int64_t)((int)blockIdx.x - a.sum_wgs) * 256, v = v0 + threadIdx.x;
        int64_t lo = 0, hi = a.T;   // the first key of at least v
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if ((int64_t)keys[mid] < v) lo = mid + 1;
            else hi = mid;
        }
        absent[threadIdx.x] = v < a.V && (lo == a.T || (int64_t)keys[lo] != v);
        __syncthreads();
        const int t = (int)threadIdx.x & (a.tpr - 1), g = (int)threadIdx.x / a.tpr, groups = 256 / a.tpr;
        const float zero[kEmbVec] = {};
        for (int r = g; r < 256; r += groups) {
            if (!absent[r]) continue;
            for (int c = t * kEmbVec; c < a.D; c += a.tpr * kEmbVec)
                store_cols<TW, true>((TW*)a.out + (v0 + r) * a.ldw + c, a.D - c, zero);
        }
        return;
    }
    const int t = (int)threadIdx.x & (a.tpr - 1), g = (int)threadIdx.x / a.tpr, groups = 256 / a.tpr;
    const int chunk = (int)(blockIdx.x / a.col_tiles) * groups + g;
    const int c = ((int)(blockIdx.x % a.col_tiles) * a.tpr + t) * kEmbVec;
    if (chunk >= a.chunks || c >= a.D) return;
    const int64_t lo = (int64_t)chunk * a.chunk, hi = min(lo + a.chunk, a.T);
    const uint32_t* places = a.places[sorted];
    const uint32_t before = lo > 0 ? keys[lo - 1] : V, after = hi < a.T ? keys[hi] : V;
    float acc[kEmbVec];
#pragma unroll
    for (int i = 0; i < kEmbVec; ++i) acc[i] = 0.0f;
    uint32_t run = keys[lo];
    bool head = lo > 0 && run == before;
    float* part = a.part + (int64_t)chunk * 2 * a.D + c;
    const TY* dy = (const TY*)a.dy;
    const int64_t limit = (a.T - 1) * a.ldy + a.D;
    for (int64_t at = lo; at < hi; at += U) {
        uint32_t key[U];
        int64_t from[U];
        RawCols<TY> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = min(at + u, hi - 1);
            key[u] = keys[i];
            from[u] = (int64_t)places[i] * a.ldy;
        }
        if constexpr (U > 1) {
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = load_raw_cols<TY>(dy, from[u], c, a.D, limit, key[u] < V);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at + u >= hi) break;
            if (key[u] != run) {
                // the run ends here
                if (run < V) {
                    if (head) store_cols<float>(part, a.D - c, acc);
                    else put_row<TW>(a, run, c, acc);
                }
                head = false;
                run = key[u];
#pragma unroll
                for (int i = 0; i < kEmbVec; ++i) acc[i] = 0.0f;
            }
            float row[kEmbVec];
            if constexpr (U > 1) unpack_cols<TY>(raw[u], dy, from[u], c, a.D, limit, key[u] < V, row);
            else load_cols<TY>(dy + from[u] + c, a.D - c, row);
#pragma unroll
            for (int i = 0; i < kEmbVec; ++i) acc[i] += row[i];
        }
    }
    if (run >= V) return;
    const bool goes_on = hi < a.T && after == run;
    if (head) store_cols<float>(part, a.D - c, acc);
    else if (goes_on) store_cols<float>(part + a.D, a.D - c, acc);
    else put_row<TW>(a, run, c, acc);
}

// A run that begins in chunk blockIdx.x and goes on: its tail and the heads of
// the chunks after it. 256 columns to a workgroup, 4 a lane; its waves take
// slices of the heads, joined in order.
constexpr int kJoinWaves = 16;

template <typename TW>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(EmbedArgs a, int sorted) {
    __shared__ float red[kJoinWaves][256];
    const uint32_t* keys = a.keys[sorted];
    const int64_t lo = (int64_t)blockIdx.x * a.chunk, hi = lo + a.chunk;   // never the last chunk
    const uint32_t run = keys[hi - 1];
    if (run >= (uint32_t)a.V || keys[hi] != run) return;   // it does not go on
    if (lo > 0 && keys[lo] == run && keys[lo - 1] == run) return;   // it began before
    int64_t x = hi, y = a.T;   // the end of the run
    while (x < y) {
        const int64_t mid = (x + y) / 2;
        if (keys[mid] <= run) x = mid + 1;
        else y = mid;
    }
    const int last = (int)((x - 1) / a.chunk);   // the last chunk with a part of it
    const int n = last - (int)blockIdx.x;        // heads
    const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
    const int per = (n + kJoinWaves - 1) / kJoinWaves;
    const int from = (int)blockIdx.x + 1 + min(w * per, n), to = (int)blockIdx.x + 1 + min((w + 1) * per, n);
    for (int c0 = (int)blockIdx.y * 256; c0 < a.D; c0 += (int)gridDim.y * 256) {
        float s[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + j * 64 + lane;
            if (c >= a.D) continue;
            if (w == 0) s[j] = a.part[((int64_t)blockIdx.x * 2 + 1) * a.D + c];
#pragma unroll 8
            for (int k = from; k < to; ++k) s[j] += a.part[(int64_t)k * 2 * a.D + c];
        }
        __syncthreads();   // the columns before have been read
#pragma unroll
        for (int j = 0; j < 4; ++j) red[w][j * 64 + lane] = s[j];
        __syncthreads();
        if (threadIdx.x < 256 && c0 + (int)threadIdx.x < a.D) {
            const int c = c0 + (int)threadIdx.x;
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kJoinWaves; ++k) v += red[k][threadIdx.x];
            TW* p = (TW*)a.out + (int64_t)run * a.ldw + c;
            *p = dyt::from_f32<TW>(a.accumulate ? __builtin_fmaf(v, a.scale, to_f32(*p)) : v * a.scale);
        }
    }
}

}  // namespace dytb
