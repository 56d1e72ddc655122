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
// One workgroup of 16 waves sorts up to kSortOne tokens alone, in one launch;
// beyond, workgroups of 4 waves take a tile each and a pass is two launches. The
// whole gradient (64 bfloat16 columns, V of 500, 50,000 and 300,000: one, two and three
// passes) with one workgroup and with many, in us: 2,049 tokens 21.3, 21.6, 37.2 and
// 24.4, 30.5, 51.4; 4,096 tokens 23.9, 26.8, 45.5 and 25.2, 32.1, 52.8; 6,000 tokens 26.6,
// 32.9, 59.2 and 24.6, 33.0, 55.7; 8,192 tokens 29.5, 37.4, 67.8 and 24.9, 33.0, 55.1;
// 16,384 tokens 39.4, 59.6, 111.4 and 24.0, 35.3, 58.9.
constexpr int kSortOneWaves = 16, kSortManyWaves = 4;
constexpr int64_t kSortOne = 5120;
constexpr int kSortTile = 1024;
constexpr int kScanTiles = 64;          // up to here every workgroup adds up the tiles before it itself
constexpr int kEmbVec = 8;              // columns of a thread
constexpr int kZeroRows = 64;           // most rows that a workgroup looks up and clears at once

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

template <typename T>
__device__ __forceinline__ void store_cols(T* p, int n, const float* v) {
    constexpr int W = VecOf<T>::n;
    if (n >= kEmbVec) {
#pragma unroll
        for (int i = 0; i < kEmbVec; i += W) *(u32x4_m*)(p + i) = pack16<T>(v + i);
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
    uint32_t* counts;     // [kRadix][tiles], then the digits' totals [kRadix]
    uint32_t tiles;
    float* part;          // [chunks][2][D]
    int64_t ldw, ldy;     // pitch of weight or dweight, of y or dy
    int64_t T, V;
    int32_t D;
    int32_t token_bits;
    int32_t tpr;          // threads of a row or of a column tile of it, up to 256
    int32_t chunk;        // sorted tokens of a chunk
    int32_t chunks;
    int32_t col_tiles;    // of tpr * kEmbVec columns
    int32_t sum_wgs;      // workgroups that sum; the rest write zero rows
    int32_t zero_rows;    // rows that a workgroup looks up and clears at once
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
    const int g = (int)threadIdx.x / a.tpr, t = (int)threadIdx.x - g * a.tpr, groups = 256 / a.tpr;
    const int64_t step = (int64_t)gridDim.x * groups * U;
    if (g >= groups) return;   // what is left over of 256 threads
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

__device__ __forceinline__ uint32_t digit_of(uint32_t key, int pass) {
    return (key >> (pass * kRadixBits)) & (kRadix - 1);
}

// Four rounds of a wave's tokens [from, to): 64 neighbours each, all loads on
// their way before the first is used.
constexpr int kRounds = 4;

__device__ __forceinline__ void load_keys(const EmbedArgs& a, int pass, uint32_t from, uint32_t to, uint32_t* key) {
    const uint32_t* keys = a.keys[pass & 1];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t i = min(from + r * 64 + (threadIdx.x & 63), to - 1);
        key[r] = pass ? keys[i] : token_at(a.tokens, a.token_bits, i, a.V);
    }
}

// The wave's part of the tokens [lo, hi).
template <int WAVES>
__device__ __forceinline__ void wave_part(uint32_t lo, uint32_t hi, uint32_t& from, uint32_t& to) {
    const uint32_t per = ((hi - lo + WAVES - 1) / WAVES + 63) / 64 * 64;
    from = min(lo + (threadIdx.x >> 6) * per, hi);
    to = min(from + per, hi);
}

__device__ __forceinline__ void count_digits(const EmbedArgs& a, int pass, uint32_t from, uint32_t to, uint32_t* cnt) {
    for (uint32_t at = from; at < to; at += 64 * kRounds) {
        uint32_t key[kRounds];
        load_keys(a, pass, at, to, key);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (at + r * 64 + (threadIdx.x & 63) < to) atomicAdd(&cnt[digit_of(key[r], pass)], 1u);
    }
}

// Moves the wave's tokens to their places; cnt[digit]: the place of its next
// token of that digit.
__device__ __forceinline__ void move_tokens(const EmbedArgs& a, int pass, uint32_t from, uint32_t to, uint32_t* cnt) {
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t* places = a.places[pass & 1];
    uint32_t* to_key = a.keys[(pass + 1) & 1];
    uint32_t* to_place = a.places[(pass + 1) & 1];
    for (uint32_t at = from; at < to; at += 64 * kRounds) {
        uint32_t key[kRounds], place[kRounds];
        load_keys(a, pass, at, to, key);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint32_t i = min(at + r * 64 + lane, to - 1);
            place[r] = pass ? places[i] : i;
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (at + r * 64 >= to) break;   // for the whole wave
            const bool on = at + r * 64 + lane < to;
            const uint32_t digit = digit_of(key[r], pass);
            const uint64_t same = same_digit(digit, on);
            const uint64_t below = same & ((1ull << lane) - 1);
            const uint32_t first = cnt[digit];
            wave_fence();   // every lane has read before the first of each digit writes
            if (on && below == 0) cnt[digit] = first + (uint32_t)__popcll(same);
            wave_fence();
            if (on) {
                const uint32_t p = first + (uint32_t)__popcll(below);
                to_key[p] = key[r];
                to_place[p] = place[r];
            }
        }
    }
}

// Exclusive sums over the workgroup's values in thread order, and their total.
template <int WAVES>
__device__ __forceinline__ uint32_t exclusive_sum(uint32_t v, uint32_t* waves, uint32_t& total) {
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
    total = 0;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
        before += k < w ? waves[k] : 0u;
        total += waves[k];
    }
    return before + s - v;
}

// All passes by one workgroup. Its digits are counted with LDS atomics (whole
// numbers: no order).
__global__ __launch_bounds__(kSortOneWaves * 64) void embed_sort_one_kernel(EmbedArgs a, int passes) {
    __shared__ uint32_t cnt[kSortOneWaves][kRadix];
    __shared__ uint32_t sums[kSortOneWaves];
    uint32_t from, to;
    wave_part<kSortOneWaves>(0, (uint32_t)a.T, from, to);
    uint32_t* mine = cnt[threadIdx.x >> 6];
    for (int pass = 0; pass < passes; ++pass) {
        for (int i = (int)threadIdx.x; i < kSortOneWaves * kRadix; i += kSortOneWaves * 64) cnt[0][i] = 0;
        __syncthreads();
        count_digits(a, pass, from, to, mine);
        __syncthreads();
        const int d = (int)threadIdx.x;
        uint32_t n = 0, total;
        if (d < kRadix)
            for (int w = 0; w < kSortOneWaves; ++w) n += cnt[w][d];
        uint32_t at = exclusive_sum<kSortOneWaves>(n, sums, total);
        if (d < kRadix)
            for (int w = 0; w < kSortOneWaves; ++w) {
                const uint32_t x = cnt[w][d];
                cnt[w][d] = at;
                at += x;
            }
        __syncthreads();
        move_tokens(a, pass, from, to, mine);
        __threadfence_block();
        __syncthreads();   // the next pass reads what all waves wrote
    }
}

// A pass's digits of each tile. (Counting them for the next pass where the
// tokens are moved to would save this launch, but the atomics meet: most tokens
// share their upper digit. 62 us a pass of 32,768 tokens.)
__global__ __launch_bounds__(kSortManyWaves * 64) void embed_count_kernel(EmbedArgs a, int pass) {
    __shared__ uint32_t cnt[kRadix];
    for (int d = (int)threadIdx.x; d < kRadix; d += kSortManyWaves * 64) cnt[d] = 0;
    __syncthreads();
    const uint32_t lo = blockIdx.x * kSortTile, hi = min(lo + kSortTile, (uint32_t)a.T);
    uint32_t from, to;
    wave_part<kSortManyWaves>(lo, hi, from, to);
    count_digits(a, pass, from, to, cnt);
    __syncthreads();
    for (int d = (int)threadIdx.x; d < kRadix; d += kSortManyWaves * 64) a.counts[(size_t)d * a.tiles + blockIdx.x] = cnt[d];
}

// Each digit's sums over the tiles before, a wave for each digit.
__global__ __launch_bounds__(256) void embed_scan_kernel(uint32_t* counts, uint32_t tiles) {
    const uint32_t lane = threadIdx.x & 63;
    const size_t d = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    uint32_t* row = counts + d * tiles;
    uint32_t total = 0;
    for (uint32_t i0 = 0; i0 < tiles; i0 += 64) {
        const uint32_t i = i0 + lane;
        const uint32_t v = i < tiles ? row[i] : 0u;
        uint32_t s = v;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const uint32_t x = (uint32_t)__shfl_up((int)s, o);
            if ((int)lane >= o) s += x;
        }
        if (i < tiles) row[i] = total + s - v;
        total += (uint32_t)__shfl((int)s, 63);
    }
    if (lane == 0) counts[(size_t)kRadix * tiles + d] = total;
}

// One pass.
__global__ __launch_bounds__(kSortManyWaves * 64) void embed_move_kernel(EmbedArgs a, int pass) {
    __shared__ uint32_t cnt[kSortManyWaves][kRadix];
    __shared__ uint32_t sums[kSortManyWaves];
    constexpr int TH = kSortManyWaves * 64;
    const uint32_t lo = blockIdx.x * kSortTile, hi = min(lo + kSortTile, (uint32_t)a.T);
    uint32_t from, to;
    wave_part<kSortManyWaves>(lo, hi, from, to);
    uint32_t* mine = cnt[threadIdx.x >> 6];
    for (int i = (int)threadIdx.x; i < kSortManyWaves * kRadix; i += TH) cnt[0][i] = 0;
    __syncthreads();
    count_digits(a, pass, from, to, mine);
    const uint32_t* counts = a.counts;
    uint32_t smaller = 0;   // tokens of the digits of the rounds before
    for (int d = (int)threadIdx.x; d < kRadix; d += TH) {
        const uint32_t* row = counts + (size_t)d * a.tiles;
        uint32_t before = 0, all = 0, total;
        if (a.tiles <= kScanTiles) {
#pragma unroll 8
            for (uint32_t i = 0; i < a.tiles; ++i) {
                const uint32_t n = row[i];
                all += n;
                before += i < blockIdx.x ? n : 0u;
            }
        } else {
            before = row[blockIdx.x];
            all = counts[(size_t)kRadix * a.tiles + d];
        }
        uint32_t at = smaller + before + exclusive_sum<kSortManyWaves>(all, sums, total);
        smaller += total;
        // (the barriers of the sum stand between the waves' counts and this)
        for (int w = 0; w < kSortManyWaves; ++w) {
            const uint32_t x = cnt[w][d];
            cnt[w][d] = at;
            at += x;
        }
    }
    __syncthreads();
    move_tokens(a, pass, from, to, mine);
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
// of dy on their way (U = 1: also for a dy of fewer elements than a vector);
// and (workgroups from sum_wgs on, zero_rows rows each) zeros for the rows of
// tokens that do not occur.
template <typename TY, typename TW, int U>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedArgs a, int sorted) {
    const uint32_t* keys = a.keys[sorted];
    const uint32_t V = (uint32_t)a.V;
    if ((int)blockIdx.x >= a.sum_wgs) {
        __shared__ uint8_t absent[kZeroRows];
        // 16 bytes to a lane: whole lines to a wave
        constexpr int W = VecOf<TW>::n;
        const int lanes = min((a.D + W - 1) / W, 256), groups = 256 / lanes;
        const int g = (int)threadIdx.x / lanes, t = (int)threadIdx.x - g * lanes;
        const float zero[W] = {};
        const int64_t step = (int64_t)(gridDim.x - a.sum_wgs) * a.zero_rows;
        for (int64_t v0 = (int64_t)((int)blockIdx.x - a.sum_wgs) * a.zero_rows; v0 < a.V; v0 += step) {
            const int64_t v = v0 + threadIdx.x;
            __syncthreads();   // the rows before have been looked up
            if (threadIdx.x < a.zero_rows) {
                int64_t lo = 0, hi = a.T;   // the first key of at least v
                while (lo < hi) {
                    const int64_t mid = (lo + hi) / 2;
                    if ((int64_t)keys[mid] < v) lo = mid + 1;
                    else hi = mid;
                }
                absent[threadIdx.x] = v < a.V && (lo == a.T || (int64_t)keys[lo] != v);
            }
            __syncthreads();
            for (int r = g < groups ? g : a.zero_rows; r < a.zero_rows; r += groups) {
                if (!absent[r]) continue;
                for (int c = t * W; c < a.D; c += lanes * W) store_vec<TW, 0>((TW*)a.out, (v0 + r) * a.ldw, c, a.D, zero);
            }
        }
        return;
    }
    const int g = (int)threadIdx.x / a.tpr, t = (int)threadIdx.x - g * a.tpr, groups = 256 / a.tpr;
    const int chunk = (int)(blockIdx.x / a.col_tiles) * groups + g;
    const int c = ((int)(blockIdx.x % a.col_tiles) * a.tpr + t) * kEmbVec;
    if (g >= groups || chunk >= a.chunks || c >= a.D) return;
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

// Few tokens and a small dweight, in one launch in place of three: a workgroup has
// every gridDim.x-th row (the frequent tokens are often neighbours) and 128 columns
// (blockIdx.y), looks all tokens through, lists those of its rows in the order of
// their places, and sums 16 threads to a token. Rows of more than kFewAlone tokens
// are cut into 16 slices, joined in order.
constexpr int kFewTokens = 2048, kFewRows = 64, kFewAlone = 8;

template <typename TY, typename TW>
__global__ __launch_bounds__(256) void embed_few_kernel(EmbedArgs a) {
    constexpr int K = kFewTokens / 256, U = 8;
    __shared__ uint32_t list[kFewTokens];     // row << 16 | place, in the order of the places
    __shared__ uint16_t order[kFewTokens];    // the places, row by row
    __shared__ uint32_t count[kFewRows], first[kFewRows + 1], waves[K][4];
    __shared__ float red[16][16 * kEmbVec];
    const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
    const uint64_t below = (1ull << lane) - 1;
    const uint32_t v0 = blockIdx.x, apart = gridDim.x, none = kFewRows;
    const int mine = (int)(((uint32_t)a.V - v0 + apart - 1) / apart);
    uint32_t tok[K];
    uint64_t in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) tok[k] = k * 256 + tid < a.T ? token_at(a.tokens, a.token_bits, k * 256 + tid, a.V) : (uint32_t)a.V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t r = tok[k] / apart;
        tok[k] = tok[k] < (uint32_t)a.V && tok[k] - r * apart == v0 ? r : none;
        in[k] = __ballot(tok[k] != none);
        if (lane == 0) waves[k][w] = (uint32_t)__popcll(in[k]);
    }
    if (tid < kFewRows) count[tid] = 0;
    __syncthreads();
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        uint32_t at = n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at += i < w ? waves[k][i] : 0u;
            n += waves[k][i];
        }
        if (tok[k] != none) {
            list[at + (uint32_t)__popcll(in[k] & below)] = tok[k] << 16 | (uint32_t)(k * 256 + tid);
            atomicAdd(&count[tok[k]], 1u);
        }
    }
    __syncthreads();
    // lane r, in every wave: row r's tokens and the first of them in `order`
    const uint32_t of_row = count[lane];
    uint32_t end = of_row;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)end, d);
        if (lane >= d) end += o;
    }
    if (w == 0) first[lane + 1] = end;
    if (tid == 0) first[0] = 0;
    for (uint64_t todo = __ballot(of_row > 0 && (lane & 3) == w); todo; todo &= todo - 1) {
        const int r = __ffsll((unsigned long long)todo) - 1;
        uint32_t at = (uint32_t)__shfl((int)(end - of_row), r);
        for (uint32_t i = 0; i < n; i += 64) {
            const uint32_t e = i + lane < n ? list[i + lane] : 0xffffffffu;
            const uint64_t same = __ballot(e >> 16 == (uint32_t)r);
            if (e >> 16 == (uint32_t)r) order[at + (uint32_t)__popcll(same & below)] = (uint16_t)e;
            at += (uint32_t)__popcll(same);
        }
    }
    __syncthreads();
    const int g = tid / 16, t = tid % 16, c0 = (int)blockIdx.y * 16 * kEmbVec, c = c0 + t * kEmbVec;
    const TY* dy = (const TY*)a.dy;
    const int64_t limit = (a.T - 1) * a.ldy + a.D;
    const auto sum = [&](uint32_t lo, uint32_t hi, float* acc) {
        for (uint32_t at = lo; at < hi; at += U) {
            RawCols<TY> raw[U];
            int64_t from[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                from[u] = (int64_t)order[min(at + u, hi - 1)] * a.ldy;
                raw[u] = load_raw_cols<TY>(dy, from[u], c, a.D, limit, true);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float row[kEmbVec];
                unpack_cols<TY>(raw[u], dy, from[u], c, a.D, limit, at + u < hi, row);
#pragma unroll
                for (int i = 0; i < kEmbVec; ++i) acc[i] += row[i];
            }
        }
    };
    for (int r = g; r < mine; r += 16) {
        const uint32_t lo = first[r], hi = first[r + 1];
        if (hi - lo > kFewAlone || c >= a.D) continue;
        float acc[kEmbVec] = {};
        sum(lo, hi, acc);
        if (hi > lo) put_row<TW>(a, v0 + r * apart, c, acc);
        else if (!a.accumulate) store_cols<TW>((TW*)a.out + (int64_t)(v0 + r * apart) * a.ldw + c, a.D - c, acc);
    }
    for (uint64_t todo = __ballot(of_row > kFewAlone); todo; todo &= todo - 1) {   // the same in every wave
        const int r = __ffsll((unsigned long long)todo) - 1;
        const uint32_t lo = first[r], k = first[r + 1] - lo, per = (k + 15) / 16;
        float acc[kEmbVec] = {};
        sum(lo + min(g * per, k), lo + min((g + 1) * per, k), acc);
        __syncthreads();   // the row before has been joined
#pragma unroll
        for (int i = 0; i < kEmbVec; ++i) red[g][t * kEmbVec + i] = acc[i];
        __syncthreads();
        if (tid < 16 * kEmbVec && c0 + tid < a.D) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += red[i][tid];
            TW* p = (TW*)a.out + (int64_t)(v0 + r * apart) * a.ldw + c0 + tid;
            *p = dyt::from_f32<TW>(a.accumulate ? __builtin_fmaf(s, a.scale, to_f32(*p)) : s * a.scale);
        }
    }
}

// Runs that begin in a chunk and go on: the tail and the heads of the chunks
// after it. A workgroup looks at kJoinChunks borders between chunks (a launch
// of one each would take longer to hand out than to run: 65 us of 1,023
// borders, 8 column tiles and 16 waves) and takes 256 columns of each such run, 4 a
// lane; its waves take slices of the heads, joined in order.
constexpr int kJoinWaves = 8, kJoinChunks = 4;

template <typename TW>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(EmbedArgs a, int sorted) {
    __shared__ float red[kJoinWaves][256];
    const uint32_t* keys = a.keys[sorted];
    const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
    // lane i: whether a run of chunk first + i goes on there, which, and in how
    // many chunks (found from both ends of a doubling step: most runs are short)
    const int first = (int)blockIdx.x * kJoinChunks;
    uint32_t run = 0;
    int heads = 0;
    bool some = false;
    if (lane < kJoinChunks && first + lane < a.chunks - 1) {
        const int64_t lo = (int64_t)(first + lane) * a.chunk, hi = lo + a.chunk;
        run = keys[hi - 1];
        const bool began_before = lo > 0 && keys[lo] == run && keys[lo - 1] == run;
        some = run < (uint32_t)a.V && keys[hi] == run && !began_before;
        if (some) {
            const int left = a.chunks - 1 - (first + lane);   // chunks after this one
            const auto goes = [&](int n) { return n <= left && keys[(int64_t)(first + lane + n) * a.chunk] == run; };
            int no = 2;
            while (goes(no)) no *= 2;
            heads = no / 2;
            while (heads + 1 < no) {
                const int mid = (heads + no) / 2;
                if (goes(mid)) heads = mid;
                else no = mid;
            }
        }
    }
    for (uint64_t todo = __ballot(some); todo; todo &= todo - 1) {   // the same in every wave
        const int i = __ffsll((unsigned long long)todo) - 1;
        const uint32_t key = (uint32_t)__shfl((int)run, i);
        const int chunk = first + i;
        const int n = __shfl(heads, i);
        const int per = (n + kJoinWaves - 1) / kJoinWaves;
        const int from = chunk + 1 + min(w * per, n), to = chunk + 1 + min((w + 1) * per, n);
        for (int c0 = (int)blockIdx.y * 256; c0 < a.D; c0 += (int)gridDim.y * 256) {
            const int c = min(c0 + lane * 4, a.D);
            float s[4] = {}, v[4];
            if (w == 0) load_vec<float>(a.part, ((int64_t)chunk * 2 + 1) * a.D, c, a.D, s);
#pragma unroll 8
            for (int k = from; k < to; ++k) {
                load_vec<float>(a.part, (int64_t)k * 2 * a.D, c, a.D, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] += v[j];
            }
            __syncthreads();   // the sums before have been read
#pragma unroll
            for (int j = 0; j < 4; ++j) red[w][lane * 4 + j] = s[j];
            __syncthreads();
            const int col = c0 + (int)threadIdx.x;
            if (threadIdx.x < 256 && col < a.D) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kJoinWaves; ++k) sum += red[k][threadIdx.x];
                TW* p = (TW*)a.out + (int64_t)key * a.ldw + col;
                *p = dyt::from_f32<TW>(a.accumulate ? __builtin_fmaf(sum, a.scale, to_f32(*p)) : sum * a.scale);
            }
        }
    }
}

}  // namespace dytb
