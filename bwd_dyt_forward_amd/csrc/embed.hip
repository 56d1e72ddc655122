// embed.hip - C ABI of the embedding lookup and its gradient (include/dyt_lm.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "block_host.hpp"
#include "dyt_lm.h"
#include "embed_kernels.hpp"

namespace dytb {
namespace {

constexpr int64_t kMaxRows = 0x7ffffffe;

int embed_shape(int64_t T, int64_t V, int64_t D) {
    if (T < 0 || V < 0 || D < 0 || T > kMaxRows || V > kMaxRows || D > ((int64_t)1 << 30)) return DYT_ERR_INVALID_ARG;
    return DYT_OK;
}

// Threads of a row: its vectors, or an even share of them where they are more
// than 256. Not rounded up to a power of two: no step exchanges lanes, and 40
// vectors in 64 threads leave a third of the loads undone.
int threads_per_row(int64_t D) {
    const int64_t vecs = (D + kEmbVec - 1) / kEmbVec, tiles = (vecs + 255) / 256;
    return (int)((vecs + tiles - 1) / std::max<int64_t>(tiles, 1));
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Chunks of the sorted tokens: enough for 1,024 workgroups of 256 threads with
// eight rows each on their way, and 16 tokens at least, so that the float32
// rows that a chunk may leave (two) stay well below the rows it reads.
struct EmbedPlan {
    int tpr, groups, col_tiles, passes, sorted;
    int64_t chunk, chunks, tiles;
    size_t keys, counts, part, bytes;   // bytes of each piece
};

EmbedPlan embed_plan(int64_t T, int64_t V, int64_t D) {
    EmbedPlan p{};
    p.tpr = std::max(1, threads_per_row(D));
    p.groups = 256 / p.tpr;
    p.col_tiles = (int)((D + p.tpr * kEmbVec - 1) / (p.tpr * kEmbVec));
    const int64_t want = std::max<int64_t>(1, (int64_t)1024 * p.groups / p.col_tiles);
    p.chunk = std::min<int64_t>(std::max<int64_t>(16, up((T + want - 1) / want, 8)), 1 << 30);
    p.chunks = (T + p.chunk - 1) / p.chunk;
    p.passes = 1;
    while (V >> (kRadixBits * p.passes)) ++p.passes;   // the tokens and V itself, where there is none
    p.sorted = p.passes & 1;
    p.tiles = (T + kSortTile - 1) / kSortTile;
    p.keys = (size_t)up(T * 4, 16);
    p.counts = T > kSortOne ? (size_t)(p.tiles + 1) * kRadix * 4 : 0;
    p.part = (size_t)p.chunks * 2 * D * 4;
    p.bytes = 4 * p.keys + std::max(p.counts, p.part);   // the sums begin where the sort has ended
    return p;
}

// Whether the gradient takes one launch (embed_few_kernel). On the device, so and in
// three launches: 1,504 tokens of 32 with 128 bfloat16 columns 7.8 and 18.5 us, 2,048
// of 8,192 with 128 9.3 and 25.2, 2,000 of 2,048 with 2,048 17.0 and 31.0, 2,048 of
// 8,192 with 2,048 (2^24 elements, where writing them is most of it) 27.9 and 33.1;
// 2,048 equal tokens with 8 columns, which one workgroup adds up, 26.9 and 20.9.
// (D: the grid's second axis takes 65,535.)
bool embed_few(int64_t T, int64_t V, int64_t D) {
    return T > 0 && T <= kFewTokens && V <= kFewRows * 1024 && D <= (1 << 20) && V * D <= (1 << 24) && T * D >= kEmbVec;
}

template <typename F>
void with_type(int dt, F&& f) {
    if (dt == DYT_F32) f((float*)nullptr);
    else if (dt == DYT_BF16) f((bf16_t*)nullptr);
    else f((f16_t*)nullptr);
}

int embed_forward(const void* weight, int64_t ldw, const void* tokens, void* y, int64_t ldy, int64_t T, int64_t V,
                  int64_t D, float scale, int wdt, int ydt, int bits, void* stream) {
    if (int e = embed_shape(T, V, D)) return e;
    if (!dtype_ok(wdt) || !dtype_ok(ydt)) return DYT_ERR_UNSUPPORTED_DTYPE;
    if (ldw == 0) ldw = D;
    if (ldy == 0) ldy = D;
    if ((bits != 32 && bits != 64) || !std::isfinite(scale) || !pitch_ok(V, D, ldw) || !pitch_ok(T, D, ldy))
        return DYT_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return DYT_OK;
    if (!tokens || !y || (V > 0 && !weight)) return DYT_ERR_INVALID_ARG;
    const int64_t sw = dtype_size(wdt), sy = dtype_size(ydt);
    if (!aligned({weight}, sw) || !aligned({y}, sy) || !aligned({tokens}, bits / 8)) return DYT_ERR_MISALIGNED;
    const Range in[] = {{weight, V ? ((V - 1) * ldw + D) * sw : 0}, {tokens, T * (bits / 8)}};
    const Range out[] = {{y, ((T - 1) * ldy + D) * sy}};
    if (!disjoint(in, 2, out, 1)) return DYT_ERR_INVALID_ARG;
    EmbedArgs a{};
    a.weight = weight; a.tokens = tokens; a.out = y; a.ldw = ldw; a.ldy = ldy; a.T = T; a.V = V; a.D = (int32_t)D;
    a.token_bits = bits; a.tpr = threads_per_row(D); a.scale = scale;
    // four rows of a thread at a time once every CU has several workgroups of them
    const int64_t groups = 256 / a.tpr;
    const bool many = T >= groups * 4 * 512 && V * D >= kEmbVec;
    const bool some = V * D >= kEmbVec;
    with_type(wdt, [&](auto* w) {
        with_type(ydt, [&](auto* o) {
            using TW = std::remove_pointer_t<decltype(w)>;
            using TY = std::remove_pointer_t<decltype(o)>;
            const auto grid = [&](int u) { return (unsigned)std::min<int64_t>((T + groups * u - 1) / (groups * u), 1 << 14); };
            if (many) embed_fwd_kernel<TW, TY, 4><<<grid(4), 256, 0, (hipStream_t)stream>>>(a);
            else if (some) embed_fwd_kernel<TW, TY, 2><<<grid(2), 256, 0, (hipStream_t)stream>>>(a);
            else embed_fwd_kernel<TW, TY, 1><<<grid(1), 256, 0, (hipStream_t)stream>>>(a);
        });
    });
    return hip_status();
}

int embed_backward(const void* dy, int64_t lddy, const void* tokens, void* dw, int64_t lddw, void* ws, size_t ws_bytes,
                   int64_t T, int64_t V, int64_t D, float scale, int ydt, int wdt, int bits, int accumulate,
                   void* stream) {
    if (int e = embed_shape(T, V, D)) return e;
    if (!dtype_ok(wdt) || !dtype_ok(ydt)) return DYT_ERR_UNSUPPORTED_DTYPE;
    if (lddw == 0) lddw = D;
    if (lddy == 0) lddy = D;
    if ((bits != 32 && bits != 64) || (accumulate != 0 && accumulate != 1) || !std::isfinite(scale) ||
        !pitch_ok(V, D, lddw) || !pitch_ok(T, D, lddy))
        return DYT_ERR_INVALID_ARG;
    if (V == 0 || D == 0 || (T == 0 && accumulate)) return DYT_OK;
    if (!dw || (T > 0 && (!dy || !tokens))) return DYT_ERR_INVALID_ARG;
    const int64_t sw = dtype_size(wdt), sy = dtype_size(ydt);
    if (!aligned({dw}, sw) || !aligned({dy}, sy) || !aligned({tokens}, bits / 8)) return DYT_ERR_MISALIGNED;
    const EmbedPlan p = embed_plan(T, V, D);
    // Zero rows of a workgroup: some 128 KB, so that others write while it looks its rows
    // up (128,000 rows of 8 KB: 210 us with 16 and 220 with 64; 50,000 of 640 bytes 56 and 48).
    const int64_t zero_rows = std::min<int64_t>(std::max<int64_t>((128 << 10) / (D * sw), 16), kZeroRows);
    const int64_t zero_wgs = accumulate ? 0 : std::min<int64_t>((V + zero_rows - 1) / zero_rows, 1 << 20);
    const int64_t sum_wgs = (p.chunks + p.groups - 1) / p.groups * p.col_tiles;
    if (T > 0 && (ws_bytes < p.bytes || !ws)) return DYT_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned({ws}, 16)) return DYT_ERR_MISALIGNED;
    const Range in[] = {{dy, T ? ((T - 1) * lddy + D) * sy : 0}, {tokens, T * (bits / 8)}};
    const Range out[] = {{dw, ((V - 1) * lddw + D) * sw}, {ws, T ? (int64_t)p.bytes : 0}};
    if (!disjoint(in, 2, out, 2)) return DYT_ERR_INVALID_ARG;
    EmbedArgs a{};
    a.dy = dy; a.tokens = tokens; a.out = dw; a.ldw = lddw; a.ldy = lddy; a.T = T; a.V = V; a.D = (int32_t)D;
    uint8_t* at = (uint8_t*)ws;
    for (int k = 0; k < 2; ++k, at += p.keys) a.keys[k] = (uint32_t*)at;
    for (int k = 0; k < 2; ++k, at += p.keys) a.places[k] = (uint32_t*)at;
    a.counts = (uint32_t*)at;
    a.part = (float*)at;
    a.tiles = (uint32_t)p.tiles;
    a.token_bits = bits; a.tpr = p.tpr; a.chunk = (int32_t)p.chunk; a.chunks = (int32_t)p.chunks;
    a.col_tiles = p.col_tiles; a.sum_wgs = (int32_t)sum_wgs; a.zero_rows = (int32_t)zero_rows; a.accumulate = accumulate; a.scale = scale;
    const hipStream_t s = (hipStream_t)stream;
    if (embed_few(T, V, D)) {
        // 1,024 workgroups where there are rows for them
        const int64_t tiles = (D + 16 * kEmbVec - 1) / (16 * kEmbVec);
        const int64_t rows = std::min<int64_t>(std::max<int64_t>((V * tiles + 1023) / 1024, 1), kFewRows);
        const dim3 grid((unsigned)((V + rows - 1) / rows), (unsigned)tiles);
        with_type(wdt, [&](auto* w) {
            with_type(ydt, [&](auto* o) {
                embed_few_kernel<std::remove_pointer_t<decltype(o)>, std::remove_pointer_t<decltype(w)>>
                    <<<grid, 256, 0, s>>>(a);
            });
        });
        return hip_status();
    }
    if (T > 0 && T <= kSortOne) {
        embed_sort_one_kernel<<<1, kSortOneWaves * 64, 0, s>>>(a, p.passes);
    } else if (T > 0) {
        const unsigned tiles = (unsigned)p.tiles, threads = kSortManyWaves * 64;
        for (int pass = 0; pass < p.passes; ++pass) {
            embed_count_kernel<<<tiles, threads, 0, s>>>(a, pass);
            if (p.tiles > kScanTiles) embed_scan_kernel<<<kRadix / 4, 256, 0, s>>>(a.counts, a.tiles);
            embed_move_kernel<<<tiles, threads, 0, s>>>(a, pass);
        }
    }
    with_type(wdt, [&](auto* w) {
        using TW = std::remove_pointer_t<decltype(w)>;
        with_type(ydt, [&](auto* o) {
            using TY = std::remove_pointer_t<decltype(o)>;
            const unsigned grid = (unsigned)(sum_wgs + zero_wgs);
            if (T * D >= kEmbVec) embed_sum_kernel<TY, TW, 8><<<grid, 256, 0, s>>>(a, p.sorted);
            else embed_sum_kernel<TY, TW, 1><<<grid, 256, 0, s>>>(a, p.sorted);
        });
        if (p.chunks > 1) {
            const dim3 grid((unsigned)((p.chunks - 1 + kJoinChunks - 1) / kJoinChunks), (unsigned)std::min<int64_t>((D + 255) / 256, 1024));
            embed_join_kernel<TW><<<grid, 64 * kJoinWaves, 0, s>>>(a, p.sorted);
        }
    });
    return hip_status();
}

}  // namespace
}  // namespace dytb

using namespace dytb;

extern "C" {

int dyt_embed_forward(const void* weight, int64_t ldw, const void* tokens, void* y, int64_t ldy, int64_t T, int64_t V,
                      int64_t D, float scale, int w_dtype, int y_dtype, int token_bits, void* stream) {
    return embed_forward(weight, ldw, tokens, y, ldy, T, V, D, scale, w_dtype, y_dtype, token_bits, stream);
}

size_t dyt_embed_backward_workspace_size(int64_t T, int64_t V, int64_t D) {
    if (embed_shape(T, V, D) || T == 0 || V == 0 || D == 0) return 0;
    return embed_plan(T, V, D).bytes;
}

int dyt_embed_backward(const void* dy, int64_t lddy, const void* tokens, void* dweight, int64_t lddw, void* workspace,
                       size_t workspace_bytes, int64_t T, int64_t V, int64_t D, float scale, int dy_dtype, int dw_dtype,
                       int token_bits, int accumulate, void* stream) {
    return embed_backward(dy, lddy, tokens, dweight, lddw, workspace, workspace_bytes, T, V, D, scale, dy_dtype,
                          dw_dtype, token_bits, accumulate, stream);
}

}  // extern "C"
