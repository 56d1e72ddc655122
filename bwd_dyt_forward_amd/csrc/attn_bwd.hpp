// attn_bwd.hpp - attention backward (gfx950).
//
// The probabilities are recomputed from q, k and the forward's log sums.
// Two kernels, so that no sum is shared between workgroups and none needs
// atomics:
//   dq   a wave owns 32 query rows and walks the keys: S^T = K Q^T,
//        dP^T = V dO^T, dS = P (dP - delta), dQ^T += K^T dS^T. It takes
//        delta = do . o of its rows first and leaves delta and the log sums
//        (in log2 units) in the workspace for
//   dkv  a wave owns 32 keys and walks the query rows that see them, of all
//        heads of the group: S = Q K^T, dP = dO V^T, dV^T += dO^T P,
//        dK^T += Q^T dS.
// That is seven products where one kernel would do five, but the sixth and
// seventh cost less than a float32 dq summed through memory: they read
// nothing that is not in LDS already.
//
// o is rounded to its type, so delta is off by a little in every pair of the
// row, which a sum over many pairs (dtable) shows: but the row's dS have to
// add up to zero, so the dq kernel adds their sum to the delta it leaves.
// In dq itself the error is one of three roundings of the same size, less by
// the number of keys the softmax spreads over. Blocks of rows that see up to
// kRefineKeys keys, all in one split, take it out in a second walk over them
// (`refine`, 16-bit types): two products over a short length, in long causal
// sequences for the first few blocks only.
//
// Both take a split of their long axis where there are few blocks; the
// splits' float32 parts are summed in split order by attn_sum_kernel.
//
// Bias gradient (dkv kernel): tiles beyond the reach of the last bucket add
// to one sum per lane. In the others the pairs of one relative position form
// a diagonal: each lane writes its 16 values of dS into a wave's scratch at
// [(key - query + 31) % 32][key], then lane t adds up diagonal t - 31 and
// adds the sum to the wave's array of sums by relative position. At the end
// the waves' arrays are joined in wave order and left in the workspace, one
// row per workgroup; attn_dtable_kernel sums each bucket's run of positions.
//
// Measured (traced, box to box): causal 2 x 4,096, 32 query over 8 key heads, D = 128
// bf16 dq 426-445 us (930-970 TFLOP/s), dk/dv 602-624 us (880-910); over 8,192 keys in
// full 374-396 and 542-569 us (970-1,100). Both hold two waves per SIMD (accumulators
// and fragments fill the registers; the 16-bit dk/dv instances of D over 96 spill
// 28 bytes a lane without the bias, 100-148 with it, single row groups 76-216) and
// have matrix cores and vector unit busy one after the other, 36-38% and 22-30% of
// the time. With the bias at D = 128, 8 x 16 heads of 1,024: 131 and 278-287 us,
// without it 118 and 179-187. 8 x 16 ragged heads of up to 1,024, D = 64 with the
// bias: 59 and 105-107 us, where the empty key blocks leave 1.1 rounds of
// workgroups. Head dimensions off 16 bytes: D = 100 1,170 and 1,920 us where 104
// takes 127 and 197.
#pragma once

#include "attn_tile.hpp"

namespace dytb {

template <typename T, int DP, int NW, int SL, bool BIAS, bool VEC>
__global__ __launch_bounds__(NW * SL * 64, attn_waves(sizeof(T))) void attn_dq_kernel(AttnArgs a) {
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
    int end = w.len;   // keys that the block's rows see
    if (a.causal) end = min(end, w.start + (min((w.block + 1) * NW * 32, rows) - 1) / a.pack + 1);
    const bool refine = sizeof(T) == 2 && end <= min(kRefineKeys, a.per_split);
    end = min(end, (w.split + 1) * a.per_split);
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

    Frag<T> q[DP / 16], dout[DP / 16];
    float delta = 0.0f;
    {
        const int64_t hd = w.head + g;
        const char* pq = a.q + w.b * a.qs.b + (int64_t)pos_i * a.qs.s + hd * a.qs.h;
        const char* po = a.o + w.b * a.os.b + (int64_t)pos_i * a.os.s + hd * a.os.h;
        const char* pd = a.dout + w.b * a.dos.b + (int64_t)pos_i * a.dos.s + hd * a.dos.h;
#pragma unroll
        for (int ds = 0; ds < DP / 16; ++ds) {
            q[ds] = global_frag<T, VEC>(pq, ds * 16 + 8 * h, a.D, there);
            dout[ds] = global_frag<T, VEC>(pd, ds * 16 + 8 * h, a.D, there);
            delta += frag_dot<T>(dout[ds], global_frag<T, VEC>(po, ds * 16 + 8 * h, a.D, there));
        }
    }
    delta = swap32_other_sum(delta);
    if (a.causal && pos < 0) delta = 0.0f;   // sees no key: its do may hold anything
    float lse = INFINITY;   // a row that sees no key: every p is 2^-inf
    if (there) {
        const int64_t at = ((int64_t)w.b * a.Hq + w.head + g) * a.Sq + pos_i;
        const float s = a.stats[at];
        if (s != -INFINITY) lse = s * kLog2e;
    }
    float rest = 0.0f;   // this lane's part of the sum of dS over its row
    f32x16 dq[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[dt][i] = 0.0f;

    // one pass over the keys; the second: see below
    const auto walk = [&](auto pass) __attribute__((always_inline)) {
        constexpr bool AGAIN = decltype(pass)::value != 0;
        alternate(begin, end, KT, [&](auto which, int j0) __attribute__((always_inline)) {
            constexpr int buf = decltype(which)::value;
            loads_landed();
            __syncthreads();
            if (j0 + KT < end) {
                ks.fetch((buf ^ 1) * KB, kr, end - j0 - KT, KT, a.D, wave, lane);
                if constexpr (!AGAIN) vs.fetch(2 * KB + (buf ^ 1) * KB, vr, end - j0 - KT, KT, a.D, wave, lane);
            }
            constexpr int kt = buf * KB, vt = kt + 2 * KB;
            const int first = j0 + sl * 32;
            // (a branch around a single sub-tile would have the accumulators copied)
            if (row0 >= rows || (SL > 1 && first >= end) || (a.causal && first > w.start + imax)) return;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int js = first + n * 32;
                f32x16 s, dp;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
                for (int ds = 0; ds < DP / 16; ++ds) {
                    s = mma<T>(TL::row_frag(row_at, kt, n, ds), q[ds], s);
                    if constexpr (!AGAIN) dp = mma<T>(TL::row_frag(row_at, vt, n, ds), dout[ds], dp);
                }
                const int reach = a.borders.reach, after = a.borders.bidirectional ? reach : 0;
                const bool far_after = js - (w.start + imax) >= after;
                const bool near = js + 31 - (w.start + imin) > -reach && !far_after;
                float p[16];
                if constexpr (BIAS) {
                    if (near) {
                        const float* at = bias + (js - pos + reach + kPad + 4 * h);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, at[8 * (i / 4) + (i % 4)]) - lse);
                    } else {
                        const float one = bias[far_after ? 2 * (reach + kPad) - 1 : 0];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, one) - lse);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse));
                }
                if (js + 32 > end || (a.causal && js + 31 > w.start + imin)) {
                    const int last = a.causal ? min(end - 1, pos) : end - 1;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool in = js + acc_row(i, h) <= last;
                        p[i] = in ? p[i] : 0.0f;
                        if constexpr (!AGAIN) dp[i] = in ? dp[i] : 0.0f;   // NaN of a row that sees no key
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if constexpr (AGAIN) {
                        p[i] *= -rest;
                    } else {
                        p[i] *= dp[i] - delta;
                        rest += p[i];
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const Frag<T> pf = pack_frag<T>(p + 8 * k);
#pragma unroll
                    for (int dt = 0; dt < DP / 32; ++dt)
                        dq[dt] = mma<T>(TL::col_frag(col_at, col_at8, kt, n * 32 + k * 16, dt), pf, dq[dt]);
                }
            }
        });
    };
    walk(Int<0>{});
    // rest is what delta is too small by (rounded o): the dkv kernel takes the sum
    rest = swap32_other_sum(rest);
    if constexpr (SL > 1) {
        float* stat = (float*)smem;   // [SL][32 rows]
        __syncthreads();
        if (h == 0) stat[sl * 32 + lane] = rest;
        __syncthreads();
        rest = 0.0f;
#pragma unroll
        for (int k = 0; k < SL; ++k) rest += stat[k * 32 + (lane & 31)];
    }
    if constexpr (sizeof(T) == 2) {
        if (refine) {
            // dq is too large by rest * sum_j p_j k_j
            __syncthreads();
            ks.start(kr, begin, KT, a.D, wave, lane);
            if (begin < end) ks.fetch(0, kr, end - begin, KT, a.D, wave, lane);
            walk(Int<1>{});
        }
    }
    if constexpr (SL > 1) {
        join_slices<DP, 1, SL>(dq, 0, sl, 0, lane);
        if (sl) return;
    }
    if (row0 < rows) {
        if (a.nsplit == 1) {
            char* out = a.dq + w.b * a.dqs.b + (int64_t)pos_i * a.dqs.s + (int64_t)(w.head + g) * a.dqs.h;
            store_acc<T, DP, VEC>(out, dq, a.scale, a.D, there, h);
        } else {
            const int64_t at = ((int64_t)w.split * a.units + w.u) * rows + row;
            store_part<DP>(a.part + at * DP, dq, a.scale, there, h);
        }
    }
    if (there && h == 0) {
        const int64_t at = ((int64_t)w.b * a.Hq + w.head + g) * a.Sq + pos_i, all = (int64_t)a.B * a.Hq * a.Sq;
        if (w.split == 0) {
            a.rows[at] = lse;
            a.rows[all + at] = a.nsplit == 1 ? delta + rest : delta;
        }
        if (a.nsplit > 1) a.rest[w.split * all + at] = rest;
    }
}

template <typename T, int DP, int NW, int SL, bool BIAS, bool VEC>
__global__ __launch_bounds__(NW * SL * 64, attn_waves(sizeof(T))) void attn_dkv_kernel(AttnArgs a) {
    typedef Tile<T, DP> TL;
    constexpr int RT = attn_dkv_tile_rows(sizeof(T), DP, NW, SL), SR = RT > 64 ? RT : 64;
    constexpr bool VLDS = dkv_vals_in_lds(sizeof(T), DP);
    constexpr int NS = RT / 32 / SL, RB = TL::bytes(RT), W = NW * SL;
    Work w;
    if (!find_work(a, w, false)) return;
    const int lane = (int)threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int rows = a.Sq * a.pack;
    const int kw = W == NW ? wave : wave % NW;   // this wave's keys of the workgroup's
    const int sl = W == NW ? 0 : wave / NW;      // and its slice of each tile's rows
    const int key0 = (w.block * NW + kw) * 32;
    const int key = key0 + (lane & 31);
    // keys that some row sees: those behind them may hold anything and are never read
    const int seen = a.causal ? min(w.len, w.start + a.Sq) : w.len;
    const bool there = key < seen;
    const float c = a.scale * kLog2e;

    // rows that see a key of this workgroup, in tiles of whole positions
    const int take = RT / a.pack * a.pack;
    int begin = w.split * a.per_split, end = min(rows, (w.split + 1) * a.per_split);
    if (a.causal) {
        const int first = max(w.block * NW * 32 - w.start, 0);   // position
        if (first >= a.Sq) begin = end;
        else begin = max(begin, first * a.pack / take * take);
    }
    if (w.block * NW * 32 >= seen) begin = end;

    const Rows qr = {a.q + w.b * a.qs.b + w.head * a.qs.h, a.qs.s, a.qs.h, a.pack};
    const Rows dr = {a.dout + w.b * a.dos.b + w.head * a.dos.h, a.dos.s, a.dos.h, a.pack};
    const int64_t row_at = ((int64_t)w.b * a.Hq + w.head) * a.Sq;
    const int64_t rows_all = (int64_t)a.B * a.Hq * a.Sq;
    constexpr int kStat = 4 * RB;   // [2 buffers][lse, delta][SR]
    const int entries = BIAS ? bias_entries(a.borders) : 0;
    constexpr int kVals = kStat + SR * 16;   // [NW][DP / 16][64 lanes] fragments
    float* bias = (float*)(smem + attn_dkv_lds_bytes(sizeof(T), DP, NW, SL));
    float* diag = bias + entries + wave * kDiagFloats;
    float* sums = bias + entries + W * kDiagFloats;   // [W][entries]
    float far_before = 0.0f, far_behind = 0.0f;
    if constexpr (BIAS) {
        fill_bias(bias, a, w.head);
        for (int x = lane; x < entries; x += 64) sums[wave * entries + x] = 0.0f;
    }

    Stream<T, DP, RT, W, VEC> qs, dos;
    int at_pos = begin / a.pack;   // position of the tile being fetched, then of the one worked on
    qs.start(qr, at_pos, take, a.D, wave, lane);
    dos.start(dr, at_pos, take, a.D, wave, lane);
    const int mine = sl * NS * 32 * TL::pitch;
    const int row_lane = TL::row_lane(lane) + mine, col_at = TL::col_lane(lane, 0) + mine;
    const int col_at8 = TL::col_lane(lane, 8) + mine;
    // log sums and delta of a tile: rows that are not there get 0, as do
    // their dO and q
    const int stat_row = (W > 1 ? (wave >> 1) * 64 : 0) + lane, stat_pos = stat_row / a.pack;
    const uint32_t stat_off =
        stat_row < take ? (uint32_t)((stat_row - stat_pos * a.pack) * a.Sq + stat_pos) * 4u : kOutside;
    // rows at negative positions see no key and are left out, whatever they hold
    const int blind = a.causal ? min(max(-w.start, 0), a.Sq) * a.pack : 0;
    const auto bring = [&](int r0, int pos0, int to) __attribute__((always_inline)) {
        qs.template fetch<true>(to * RB, qr, end - r0, take, a.D, wave, lane, blind - r0);
        dos.template fetch<true>(2 * RB + to * RB, dr, end - r0, take, a.D, wave, lane, blind - r0);
        // 64 rows of one of the two to a wave (both to a single wave)
        if (W == 1 || wave < SR / 32) {
            for (int k = wave & 1; k < 2; k += W == 1 ? 1 : 2)
                load_to_lds4(a.rows + k * rows_all + row_at + pos0, kStat + (to * 2 + k) * SR * 4 + (wave >> 1) * 256,
                             r0 + stat_row < end ? stat_off : kOutside);
        }
    };
    if (begin < end) bring(begin, at_pos, 0);

    Frag<T> kf[DP / 16], vf[VLDS ? 1 : DP / 16];
    {
        const int kk = min(key, a.Sk - 1);
        const char* pk = a.k + w.b * a.ks.b + (int64_t)kk * a.ks.s + w.kv * a.ks.h;
        const char* pv = a.v + w.b * a.vs.b + (int64_t)kk * a.vs.s + w.kv * a.vs.h;
#pragma unroll
        for (int ds = 0; ds < DP / 16; ++ds) {
            kf[ds] = global_frag<T, VEC>(pk, ds * 16 + 8 * h, a.D, there);
            const Frag<T> f = global_frag<T, VEC>(pv, ds * 16 + 8 * h, a.D, there);
            if constexpr (VLDS) {
                if (sl == 0) *(Frag<T>*)(smem + kVals + (kw * (DP / 16) + ds) * 1024 + lane * 16) = f;
            } else {
                vf[ds] = f;
            }
        }
    }
    f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[dt][i] = dv[dt][i] = 0.0f;

    // positions of the sub-tiles' first and last rows within a tile
    int sub_first[NS], sub_last[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        sub_first[n] = (sl * NS + n) * 32 / a.pack;
        sub_last[n] = min((sl * NS + n) * 32 + 31, take - 1) / a.pack;
    }
    const int last_pos = end / a.pack - 1;
    alternate(begin, end, take, [&](auto which, int r0) __attribute__((always_inline)) {
        constexpr int buf = decltype(which)::value;
        loads_landed();
        __syncthreads();
        const int pos0 = at_pos;
        at_pos += take / a.pack;
        if (r0 + take < end) bring(r0 + take, at_pos, buf ^ 1);
        constexpr int qt = buf * RB, ot = qt + 2 * RB;
        // (a branch around a single sub-tile would have the accumulators copied)
        if (key0 >= seen || (a.causal && key0 > w.start + min(pos0 + sub_last[NS - 1], last_pos))) return;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int rs = r0 + (sl * NS + n) * 32;
            const int imin = w.start + pos0 + sub_first[n];   // positions
            const int imax = w.start + max(min(pos0 + sub_last[n], last_pos), pos0 + sub_first[n]);
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int ds = 0; ds < DP / 16; ++ds) {
                s = mma<T>(TL::row_frag(row_lane, qt, n, ds), kf[ds], s);
                const Frag<T> vd = VLDS ? *(const Frag<T>*)(smem + kVals + (kw * (DP / 16) + ds) * 1024 + lane * 16)
                                        : vf[VLDS ? 0 : ds];
                dp = mma<T>(TL::row_frag(row_lane, ot, n, ds), vd, dp);
            }
            const float* st = (const float*)(smem + kStat + buf * SR * 8) + (sl * NS + n) * 32 + 4 * h;
            float p[16];
            const int reach = a.borders.reach, after = a.borders.bidirectional ? reach : 0;
            const bool far_after = key0 - imax >= after;
            const bool near = key0 + 31 - imin > -reach && !far_after;
            if constexpr (BIAS) {
                if (near) {
                    // pack = 1: the row of register i is acc_row(i, h) positions on
                    const float* at = bias + (key - w.start - rs + reach + kPad - 4 * h);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = 8 * (i / 4) + (i % 4);
                        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, at[-k]) - st[k]);
                    }
                } else {
                    const float one = bias[far_after ? entries - 1 : 0];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, one) - st[8 * (i / 4) + (i % 4)]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -st[8 * (i / 4) + (i % 4)]));
            }
            if (key0 + 32 > seen || (a.causal && key0 + 31 > imin) || rs + 32 > end) {
                // rows that see the key: `count` from `first` on. Rows past the end have
                // s = 0 and log sum 0, so with the bias e^bias as p: zeros of dO would
                // meet an infinity where that passes the type's range.
                const int first = a.causal ? min(max(key - w.start, 0), a.Sq) * a.pack : 0;
                const uint32_t count = there ? (uint32_t)max(end - first, 0) : 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = (uint32_t)(rs + acc_row(i, h) - first) < count ? p[i] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Frag<T> pf = pack_frag<T>(p + 8 * k);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt)
                    dv[dt] = mma<T>(TL::col_frag(col_at, col_at8, ot, n * 32 + k * 16, dt), pf, dv[dt]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] *= dp[i] - st[SR + 8 * (i / 4) + (i % 4)];
            if constexpr (BIAS) {
                // rows past the end have p = 0 and finite dP - delta: dS = 0
                if (near) {
                    // diagonal t = key - query + 31 has its elements in columns (keys)
                    // 0 .. t, diagonal t + 32 in t + 1 .. 31: they share row t
                    const int t0 = 31 - 4 * h + (lane & 31);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        diag[((t0 - 8 * (i / 4) - (i % 4)) & 31) * kDiagPitch + (lane & 31)] = p[i];
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    float d = 0.0f;
                    const uint32_t low = (2u << (lane & 31)) - 1u, mask = h ? ~low : low;   // its columns
                    const float* from = diag + (lane & 31) * kDiagPitch;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        d += __uint_as_float(__float_as_uint(from[x]) & (uint32_t)__builtin_amdgcn_sbfe((int)mask, x, 1));
                    // lane 63 has no diagonal: d = 0
                    float* to = sums + wave * entries + (key0 - (w.start + rs) + reach + kPad - 31 + lane);
                    if (lane < 63) *to += d;
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                } else {
                    float d = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) d += p[i];
                    if (far_after) far_behind += d;
                    else far_before += d;
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Frag<T> pf = pack_frag<T>(p + 8 * k);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt)
                    dk[dt] = mma<T>(TL::col_frag(col_at, col_at8, qt, n * 32 + k * 16, dt), pf, dk[dt]);
            }
        }
    });
    if constexpr (BIAS) {
        far_before = lanes_sum<64>(far_before);
        far_behind = lanes_sum<64>(far_behind);
        if (lane == 0) {
            sums[wave * entries] += far_before;             // farther than the reach: the outermost entries
            sums[wave * entries + entries - 1] += far_behind;
        }
        __syncthreads();
        for (int x = (int)threadIdx.x; x < entries; x += W * 64) {
            float s = sums[x];
            for (int k = 1; k < W; ++k) s += sums[k * entries + x];
            a.tpart[w.flat * entries + x] = s;
        }
    }
    if constexpr (SL > 1) {
        join_slices<DP, NW, SL>(dk, kw, sl, 0, lane);
        join_slices<DP, NW, SL>(dv, kw, sl, 1, lane);
        if (sl > 1) return;
    }
    if (key0 >= a.Sk) return;
    const bool in = key < a.Sk;
    // (of several slices, the first holds dk and the second dv)
    const bool has_dk = SL == 1 || sl == 0, has_dv = SL == 1 || sl == 1;
    const int parts = a.nsplit * (a.G / a.pack);   // float32 parts of each key head
    if (parts == 1) {
        const int64_t kk = min(key, a.Sk - 1);
        if (has_dk) store_acc<T, DP, VEC>(a.dk + w.b * a.dks.b + kk * a.dks.s + w.kv * a.dks.h, dk, a.scale, a.D, in, h);
        if (has_dv) store_acc<T, DP, VEC>(a.dv + w.b * a.dvs.b + kk * a.dvs.s + w.kv * a.dvs.h, dv, 1.0f, a.D, in, h);
    } else {
        // [part][dk, dv][B, Hkv, Sk, DP]
        const int64_t heads = (int64_t)a.B * a.Hkv, part = (w.head % a.G) / a.pack + (int64_t)(a.G / a.pack) * w.split;
        const int64_t at = ((part * 2 * heads + (int64_t)w.b * a.Hkv + w.kv) * a.Sk + min(key, a.Sk - 1)) * DP;
        if (has_dk) store_part<DP>(a.part + at, dk, a.scale, in, h);
        if (has_dv) store_part<DP>(a.part + at + heads * a.Sk * DP, dv, 1.0f, in, h);
    }
}

// Sums float32 parts in order and rounds once: out[b, s, h] = sum_p part[p]
// [(b, hu)][row][DP] with row = s * pack + g and h = hu * pack + g. One part
// lies `stride` floats after the other. DP / 4 threads per row. With `delta`
// (dq's sum) the parts of `rest` [part][b, head, i] are added to it.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attn_sum_kernel(SumArgs x) {
    constexpr int TPR = DP / 4, PER = 256 / TPR;
    if ((int)threadIdx.x >= PER * TPR) return;
    const int d = ((int)threadIdx.x % TPR) * 4;
    // workgroups past the first sum's rows make the second
    const int64_t first = (x.total + PER - 1) / PER;
    for (int64_t group = blockIdx.x; group < (x.out2 ? 2 : 1) * first; group += gridDim.x) {
        const bool second = group >= first;
        const int64_t at = (second ? group - first : group) * PER + (int)threadIdx.x / TPR;
        const float* part = second ? x.part2 : x.part;
        if (at >= x.total) continue;
        float o[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int p = 0; p < x.parts; ++p) {
            const f32x4 v = *(const f32x4*)(part + p * x.stride + at * DP + d);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] += v[k];
        }
        const int u = (int)(at / x.rows), r = (int)(at - (int64_t)u * x.rows);
        const int b = u / x.hu, i = r / x.pack, head = (u - b * x.hu) * x.pack + (r - i * x.pack);
        const Strides os = second ? x.os2 : x.os;
        T* to = (T*)((second ? x.out2 : x.out) + b * os.b + (int64_t)i * os.s + (int64_t)head * os.h);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (d + k < x.D) to[d + k] = dyt::from_f32<T>(o[k]);
        if (x.delta && d == 0) {
            const int64_t n = ((int64_t)b * x.hu * x.pack + head) * (x.rows / x.pack) + i;
            float s = 0.0f;
            for (int p = 0; p < x.parts; ++p) s += x.rest[p * x.total + n];
            x.delta[n] += s;
        }
    }
}

}  // namespace dytb
