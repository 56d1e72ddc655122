// attn_fwd.hpp - attention forward (gfx950).
//
// One pass over the keys with the running maximum and sum of the softmax.
// A wave owns 32 query rows, a workgroup of NW waves 32 NW; the keys and
// values pass through LDS in double-buffered tiles. S^T = K Q^T puts a query
// in each lane (column), so the softmax's maximum and sum over keys are
// in-lane operations plus one exchange between the lane halves, and the
// probabilities are already the B fragments of O^T = V^T P^T.
//
// Rows are (position, head of the group) pairs: the G query heads that share
// a key head are rows of one unit, so its keys and values are read once for
// all of them (single tokens most of all). With the bias, whose table has a
// column per head, each query head is a unit of its own (pack = 1).
//
// The reference maximum only moves when a row's maximum has grown by more
// than 2^8 over it (then the accumulators are rescaled): probabilities stay
// below 2^8, well inside every type, and the sums are float32.
//
// Where there are too few blocks of rows to fill the card, SL waves (slices)
// share the rows and take 32 keys of each tile each; they join their maxima,
// sums and outputs through LDS at the end. Few rows over many keys are
// also split along the keys: each split leaves its unnormalised float32 output
// and (maximum, sum) in the workspace and attn_join_kernel joins them in split
// order.
//
// Measured (traced, box to box): causal 2 x 4,096, 32 query over 8 key heads, D = 128
// bf16 305-316 us (870-900 TFLOP/s of the visible pairs' products), 8,192 keys in
// full 270-282 us (970-1,020 TFLOP/s); two waves per SIMD for the registers, whose
// matrix cores (36% busy) and vector unit (34%) work one after the other within a
// wave. At D = 64 (an exponential and six operations per pair beside 256 flop) the
// vector unit is 49% and the matrix cores 22% busy: 4 x 16 heads of 2,048 causal with
// the bias 63 us. Single tokens are bound by HBM: 8 x 8 key heads of up to 16,384
// keys, D = 128, 75 us (4.5 TB/s). Head dimensions off 16 bytes go element by
// element in single waves: 8 x 16 heads of 1,024, D = 100, 1,060 us (104: 92).
#pragma once

#include "attn_tile.hpp"

namespace dytb {

template <typename T, int DP, int NW, int SL, bool BIAS, bool VEC>
__global__ __launch_bounds__(NW * SL * 64, attn_waves(sizeof(T))) void attn_fwd_kernel(AttnArgs a) {
    static_assert(NW == 1 || SL == 1);
    typedef Tile<T, DP> TL;
    constexpr int KT = attn_tile_rows(sizeof(T), NW, SL);
    constexpr int NS = KT / 32 / SL, KB = TL::bytes(KT);
    Work w;
    if (!find_work(a, w, true)) return;
    const int lane = (int)threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int sl = SL > 1 ? wave : 0;   // this wave's slice: keys 32 sl .. 32 sl + 31 of each tile
    const int rows = a.Sq * a.pack;
    const int row0 = (w.block * NW + (SL > 1 ? 0 : wave)) * 32;
    const int row = row0 + (lane & 31);
    const bool there = row < rows;
    const int rr = min(row, rows - 1);
    const int pos_i = rr / a.pack, g = rr - pos_i * a.pack;
    const int pos = w.start + pos_i;
    const int imin = min(row0, rows - 1) / a.pack;
    const int imax = min(row0 + 31, rows - 1) / a.pack;
    int end = min(w.len, (w.split + 1) * a.per_split);
    if (a.causal) end = min(end, w.start + (min((w.block + 1) * NW * 32, rows) - 1) / a.pack + 1);
    const int begin = w.split * a.per_split;

    const Rows kr = {a.k + w.b * a.ks.b + w.kv * a.ks.h, a.ks.s, 0, 1};
    const Rows vr = {a.v + w.b * a.vs.b + w.kv * a.vs.h, a.vs.s, 0, 1};
    const float c = a.scale * kLog2e;

    Stream<T, DP, KT, NW * SL, VEC> ks, vs;
    ks.start(kr, begin, KT, a.D, wave, lane);
    vs.start(vr, begin, KT, a.D, wave, lane);
    if (begin < end) {
        ks.fetch(0, kr, end - begin, KT, a.D, wave, lane);
        vs.fetch(2 * KB, vr, end - begin, KT, a.D, wave, lane);
    }
    const int mine = sl * 32 * TL::pitch;
    const int row_at = TL::row_lane(lane) + mine, col_at = TL::col_lane(lane, 0) + mine;
    const int col_at8 = TL::col_lane(lane, 8) + mine;
    float* bias = (float*)(smem + 4 * KB);
    if constexpr (BIAS) fill_bias(bias, a, w.head);

    Frag<T> q[DP / 16];
    {
        const char* p = a.q + w.b * a.qs.b + (int64_t)pos_i * a.qs.s + (int64_t)(w.head + g) * a.qs.h;
#pragma unroll
        for (int ds = 0; ds < DP / 16; ++ds) q[ds] = global_frag<T, VEC>(p, ds * 16 + 8 * h, a.D, there);
    }
    f32x16 o[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] = 0.0f;
    // m: reference maximum; units of the raw product without bias, of log2
    // with it. l: this lane's part of the sum.
    float m = -INFINITY, l = 0.0f;
    const float mc = BIAS ? 1.0f : c;
    const float grow = 8.0f / mc;

    alternate(begin, end, KT, [&](auto which, int j0) __attribute__((always_inline)) {
        constexpr int buf = decltype(which)::value;
        loads_landed();
        __syncthreads();
        if (j0 + KT < end) {
            ks.fetch((buf ^ 1) * KB, kr, end - j0 - KT, KT, a.D, wave, lane);
            vs.fetch(2 * KB + (buf ^ 1) * KB, vr, end - j0 - KT, KT, a.D, wave, lane);
        }
        const int first = j0 + sl * 32;
        if (row0 >= rows || (SL > 1 && first >= end) || (a.causal && first > w.start + imax)) return;
        constexpr int kt = buf * KB, vt = 2 * KB + buf * KB;
        f32x16 s[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[n][i] = 0.0f;
#pragma unroll
            for (int ds = 0; ds < DP / 16; ++ds)
                s[n] = mma<T>(TL::row_frag(row_at, kt, n, ds), q[ds], s[n]);
        }
        if constexpr (BIAS) {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int js = first + n * 32;
                const int reach = a.borders.reach, after = a.borders.bidirectional ? reach : 0;
                const bool far_after = js - (w.start + imax) >= after;
                if (js + 31 - (w.start + imin) > -reach && !far_after) {
                    const float* at = bias + (js - pos + reach + kPad + 4 * h);
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[n][i] = __builtin_fmaf(s[n][i], c, at[8 * (i / 4) + (i % 4)]);
                } else {
                    const float one = bias[far_after ? 2 * (reach + kPad) - 1 : 0];
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[n][i] = __builtin_fmaf(s[n][i], c, one);
                }
            }
        }
        if (first + NS * 32 > end || (a.causal && first + NS * 32 - 1 > w.start + imin)) {
            const int last = a.causal ? min(end - 1, pos) : end - 1;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[n][i] = first + n * 32 + acc_row(i, h) <= last ? s[n][i] : -INFINITY;
        }
        float mt = s[0][0];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) mt = fmaxf(mt, s[n][i]);
        mt = swap32_max(mt);
        if (__any(mt > m + grow)) {
            const float mn = fmaxf(m, mt);
            const float f = __builtin_amdgcn_exp2f((m - (mn == -INFINITY ? 0.0f : mn)) * mc);
            l *= f;
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[dt][i] *= f;
            m = mn;
        }
        const float mm = (m == -INFINITY ? 0.0f : m) * mc;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = __builtin_amdgcn_exp2f(BIAS ? s[n][i] - mm : __builtin_fmaf(s[n][i], c, -mm));
                l += p[i];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Frag<T> pf = pack_frag<T>(p + 8 * k);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt)
                    o[dt] = mma<T>(TL::col_frag(col_at, col_at8, vt, n * 32 + k * 16, dt), pf, o[dt]);
            }
        }
    });
    if (row0 >= rows) return;
    l = swap32_other_sum(l);
    float ml = (m == -INFINITY ? 0.0f : m) * mc;   // log2 units
    if constexpr (SL > 1) {
        // the slices' common maximum and sum, then their outputs
        float* stat = (float*)(smem + SL * DP * 128);   // [SL][maximum, sum][32 rows], past the boxes
        __syncthreads();
        if (h == 0) {
            stat[sl * 64 + lane] = l > 0.0f ? ml : -INFINITY;
            stat[sl * 64 + 32 + lane] = l;
        }
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < SL; ++k) M = fmaxf(M, stat[k * 64 + (lane & 31)]);
        M = M == -INFINITY ? 0.0f : M;
        const float f = l > 0.0f ? __builtin_amdgcn_exp2f(ml - M) : 0.0f;
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < SL; ++k)
            l += __builtin_amdgcn_exp2f(stat[k * 64 + (lane & 31)] - M) * stat[k * 64 + 32 + (lane & 31)];
        ml = M;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] *= f;
        join_slices<DP, 1, SL>(o, 0, sl, 0, lane);
        if (sl) return;
    }
    if (a.nsplit == 1) {
        char* out = a.out + w.b * a.os.b + (int64_t)pos_i * a.os.s + (int64_t)(w.head + g) * a.os.h;
        store_acc<T, DP, VEC>(out, o, l > 0.0f ? 1.0f / l : 0.0f, a.D, there, h);
        if (there && h == 0)
            a.stats[((int64_t)w.b * a.Hq + w.head + g) * a.Sq + pos_i] =
                l > 0.0f ? (ml + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
    } else {
        const int64_t at = ((int64_t)w.split * a.units + w.u) * rows + row;
        store_part<DP>(a.part + at * DP, o, 1.0f, there, h);
        if (there && h == 0) {
            a.part_ml[2 * at] = l > 0.0f ? ml : -INFINITY;
            a.part_ml[2 * at + 1] = l;
        }
    }
}

// Joins the splits of a row: o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s
// with M the largest m_s. JG groups of DP / 4 threads share a row, group g
// taking splits g, g + JG, ..; the groups are added in order. A row of many
// splits (a single token's) is a chain of dependent loads otherwise: 9.5 us
// for 16 splits of 256 rows with one group.
template <typename T, int DP, int JG>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    constexpr int TPR = DP / 4, PER = 256 / (TPR * JG);
    const int rows = a.Sq * a.pack;
    const int64_t total = (int64_t)a.units * rows;
    const int slot = (int)threadIdx.x / (TPR * JG);
    const int g = (int)threadIdx.x / TPR % JG;
    const int64_t at = (int64_t)blockIdx.x * PER + slot;
    const int d = ((int)threadIdx.x % TPR) * 4;
    const bool in = slot < PER && at < total;
    float M = -INFINITY, l = 0.0f, mm = 0.0f, o[4] = {0, 0, 0, 0};
    if (in) {
#pragma unroll 8
        for (int s = 0; s < a.nsplit; ++s) M = fmaxf(M, a.part_ml[2 * (s * total + at)]);
        mm = M == -INFINITY ? 0.0f : M;
#pragma unroll 4
        for (int s = g; s < a.nsplit; s += JG) {
            // an empty split has weight 2^-inf = 0 and a part of zeros
            const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * (s * total + at)] - mm);
            l += f * a.part_ml[2 * (s * total + at) + 1];
            const f32x4 v = *(const f32x4*)(a.part + (s * total + at) * DP + d);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] += f * v[k];
        }
    }
    if constexpr (JG > 1) {
        __shared__ float join[256][5];
#pragma unroll
        for (int k = 0; k < 4; ++k) join[threadIdx.x][k] = o[k];
        join[threadIdx.x][4] = l;
        __syncthreads();
        if (g == 0) {
#pragma unroll
            for (int j = 1; j < JG; ++j) {
                const int from = min((int)threadIdx.x + j * TPR, 255);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] += join[from][k];
                l += join[from][4];
            }
        }
    }
    if (!in || g) return;
    const int u = (int)(at / rows), r = (int)(at - (int64_t)u * rows);
    const int hu = a.Hq / a.pack;
    const int b = u / hu, i = r / a.pack, head = (u - b * hu) * a.pack + (r - i * a.pack);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    T* out = (T*)(a.out + b * a.os.b + (int64_t)i * a.os.s + (int64_t)head * a.os.h);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (d + k < a.D) out[d + k] = dyt::from_f32<T>(o[k] * inv);
    if (d == 0)
        a.stats[((int64_t)b * a.Hq + head) * a.Sq + i] =
            l > 0.0f ? (mm + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

}  // namespace dytb
