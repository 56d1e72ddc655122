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
//
// Both take a split of their long axis where there are few blocks; the
// splits' float32 parts are summed in split order by attn_sum_kernel.
//
// Bias gradient (dkv kernel): tiles beyond the reach of the last bucket add
// to one sum per lane. In the others the pairs of one relative position form
// a diagonal: each lane writes its 16 values of dS into a wave's scratch at
// [key - query + 31][key] (the positions are the same for every tile, the
// rest of the scratch stays zero), then lane t adds up diagonal t - 31 and
// adds the sum to the wave's array of sums by relative position. At the end
// the waves' arrays are joined in wave order and left in the workspace, one
// row per workgroup; attn_dtable_kernel sums each bucket's run of positions.
#pragma once

#include "attn_tile.hpp"

namespace dytb {

constexpr int kDiagPitch = 33;
constexpr int kDiagFloats = 64 * kDiagPitch;

template <typename T, int NW> struct BwdTile { static constexpr int rows = sizeof(T) == 2 && NW > 1 ? 64 : 32; };

// The dk/dv kernel holds 4 DP / 32 accumulators and its keys' and values'
// fragments. Above D = 64 that leaves room for one wave per SIMD; with the
// values' fragments in LDS (which has bandwidth to spare) two fit, and hide
// each other's waits. Tiles of 32 rows then keep two workgroups' LDS in a CU.
template <typename T, int DP, int NW>
constexpr bool dkv_vals_in_lds() { return sizeof(T) == 2 && DP > 64; }
template <typename T, int DP, int NW> struct DkvTile {
    static constexpr int rows = dkv_vals_in_lds<T, DP, NW>() ? 32 : BwdTile<T, NW>::rows;
};
template <typename T, int DP, int NW>
constexpr int dkv_lds_bytes() {
    return 2 * 2 * Tile<T, DP>::bytes(DkvTile<T, DP, NW>::rows) + 1024 +
           (dkv_vals_in_lds<T, DP, NW>() ? NW * (DP / 16) * 1024 : 0);
}

template <typename T, int DP, int NW>
constexpr int bwd_lds_bytes() { return 2 * 2 * Tile<T, DP>::bytes(BwdTile<T, NW>::rows); }

// LDS floats of the bias gradient.
inline __host__ __device__ int dbias_floats(int entries, int nw) { return nw * (kDiagFloats + entries); }

template <typename T, int DP, int NW, bool BIAS, bool VEC>
__global__ __launch_bounds__(NW * 64, (sizeof(T) == 2 ? 2 : 1)) void attn_dq_kernel(AttnArgs a) {
    typedef Tile<T, DP> TL;
    constexpr int KT = BwdTile<T, NW>::rows;
    constexpr int NS = KT / 32, KB = TL::bytes(KT);
    Work w;
    if (!find_work(a, w, a.causal != 0, false)) return;
    const int lane = (int)threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int rows = a.Sq * a.pack;
    const int row0 = (w.block * NW + wave) * 32;
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

    Stream<T, DP, KT, NW, VEC> ks, vs;
    ks.start(kr, begin, KT, a.D, wave, lane);
    vs.start(vr, begin, KT, a.D, wave, lane);
    if (begin < end) {
        ks.fetch(0, kr, end - begin, KT, a.D, wave, lane);
        vs.fetch(2 * KB, vr, end - begin, KT, a.D, wave, lane);
    }
    const int row_at = TL::row_lane(lane), col_at = TL::col_lane(lane, 0), col_at8 = TL::col_lane(lane, 8);
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

    alternate(begin, end, KT, [&](auto which, int j0) __attribute__((always_inline)) {
        constexpr int buf = decltype(which)::value;
        loads_landed();
        __syncthreads();
        if (j0 + KT < end) {
            ks.fetch((buf ^ 1) * KB, kr, end - j0 - KT, KT, a.D, wave, lane);
            vs.fetch(2 * KB + (buf ^ 1) * KB, vr, end - j0 - KT, KT, a.D, wave, lane);
        }
        constexpr int kt = buf * KB, vt = kt + 2 * KB;
        // (a branch around a single sub-tile would have the accumulators copied)
        if (row0 >= rows || (a.causal && j0 > w.start + imax)) return;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int js = j0 + n * 32;
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int ds = 0; ds < DP / 16; ++ds) {
                s = mma<T>(TL::row_frag(row_at, kt, n, ds), q[ds], s);
                dp = mma<T>(TL::row_frag(row_at, vt, n, ds), dout[ds], dp);
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
                for (int i = 0; i < 16; ++i) p[i] = js + acc_row(i, h) <= last ? p[i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] *= dp[i] - delta;
                rest += p[i];
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
    if (row0 < rows) {
        if (a.nsplit == 1) {
            char* out = a.dq + w.b * a.dqs.b + (int64_t)pos_i * a.dqs.s + (int64_t)(w.head + g) * a.dqs.h;
            store_acc<T, DP, VEC>(out, dq, a.scale, a.D, there, h);
        } else {
            const int64_t at = ((int64_t)w.split * a.units + w.u) * rows + row;
            store_part<DP>(a.part + at * DP, dq, a.scale, there, h);
        }
    }
    // rest is what delta is too small by (rounded o): the dkv kernel takes the sum
    rest = swap32_other_sum(rest);
    if (there && h == 0) {
        const int64_t at = ((int64_t)w.b * a.Hq + w.head + g) * a.Sq + pos_i, all = (int64_t)a.B * a.Hq * a.Sq;
        if (w.split == 0) {
            a.rows[at] = lse;
            a.rows[all + at] = a.nsplit == 1 ? delta + rest : delta;
        }
        if (a.nsplit > 1) a.rest[w.split * all + at] = rest;
    }
}

template <typename T, int DP, int NW, bool BIAS, bool VEC>
__global__ __launch_bounds__(NW * 64, (sizeof(T) == 2 ? 2 : 1)) void attn_dkv_kernel(AttnArgs a) {
    typedef Tile<T, DP> TL;
    constexpr int RT = DkvTile<T, DP, NW>::rows;
    constexpr bool VLDS = dkv_vals_in_lds<T, DP, NW>();
    constexpr int NS = RT / 32, RB = TL::bytes(RT);
    Work w;
    if (!find_work(a, w, false, a.causal != 0)) return;
    const int lane = (int)threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int rows = a.Sq * a.pack;
    const int key0 = (w.block * NW + wave) * 32;
    const int key = key0 + (lane & 31);
    const bool there = key < w.len;
    const float c = a.scale * kLog2e;

    // rows that see a key of this workgroup, in tiles of whole positions
    const int take = RT / a.pack * a.pack;
    int begin = w.split * a.per_split, end = min(rows, (w.split + 1) * a.per_split);
    if (a.causal) {
        const int first = max(w.block * NW * 32 - w.start, 0);   // position
        if (first >= a.Sq) begin = end;
        else begin = max(begin, first * a.pack / take * take);
    }
    if (w.block * NW * 32 >= w.len) begin = end;

    const Rows qr = {a.q + w.b * a.qs.b + w.head * a.qs.h, a.qs.s, a.qs.h, a.pack};
    const Rows dr = {a.dout + w.b * a.dos.b + w.head * a.dos.h, a.dos.s, a.dos.h, a.pack};
    const int64_t row_at = ((int64_t)w.b * a.Hq + w.head) * a.Sq;
    const int64_t rows_all = (int64_t)a.B * a.Hq * a.Sq;
    constexpr int kStat = 4 * RB;   // [2 buffers][lse, delta][64]
    const int entries = BIAS ? bias_entries(a.borders) : 0;
    constexpr int kVals = kStat + 1024;   // [NW][DP / 16][64 lanes] fragments
    float* bias = (float*)(smem + dkv_lds_bytes<T, DP, NW>());
    float* diag = bias + entries + wave * kDiagFloats;
    float* sums = bias + entries + NW * kDiagFloats;   // [NW][entries]
    float far_before = 0.0f, far_behind = 0.0f;
    if constexpr (BIAS) {
        fill_bias(bias, a, w.head);
        for (int x = lane; x < kDiagFloats; x += 64) diag[x] = 0.0f;
        for (int x = lane; x < entries; x += 64) sums[wave * entries + x] = 0.0f;
    }

    Stream<T, DP, RT, NW, VEC> qs, dos;
    int at_pos = begin / a.pack;   // position of the tile being fetched, then of the one worked on
    qs.start(qr, at_pos, take, a.D, wave, lane);
    dos.start(dr, at_pos, take, a.D, wave, lane);
    const int row_lane = TL::row_lane(lane), col_at = TL::col_lane(lane, 0), col_at8 = TL::col_lane(lane, 8);
    // log sums and delta of a tile: rows that are not there get 0, and as
    // their dO and q are zeros they add nothing
    const int lane_pos = lane / a.pack;
    const uint32_t stat_off = lane < take ? (uint32_t)((lane - lane_pos * a.pack) * a.Sq + lane_pos) * 4u : kOutside;
    const auto bring = [&](int r0, int pos0, int to) __attribute__((always_inline)) {
        qs.fetch(to * RB, qr, end - r0, take, a.D, wave, lane);
        dos.fetch(2 * RB + to * RB, dr, end - r0, take, a.D, wave, lane);
        if (wave < 2) {
            for (int k = wave; k < 2; k += NW < 2 ? 1 : 2)
                load_to_lds4(a.rows + k * rows_all + row_at + pos0, kStat + to * 512 + k * 256,
                             r0 + lane < end ? stat_off : kOutside);
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
            if constexpr (VLDS) *(Frag<T>*)(smem + kVals + (wave * (DP / 16) + ds) * 1024 + lane * 16) = f;
            else vf[ds] = f;
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
        sub_first[n] = n * 32 / a.pack;
        sub_last[n] = min(n * 32 + 31, take - 1) / a.pack;
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
        if (key0 >= w.len || (a.causal && key0 > w.start + min(pos0 + sub_last[NS - 1], last_pos))) return;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int rs = r0 + n * 32;
            const int imin = w.start + pos0 + sub_first[n];   // positions
            const int imax = w.start + max(min(pos0 + sub_last[n], last_pos), pos0 + sub_first[n]);
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int ds = 0; ds < DP / 16; ++ds) {
                s = mma<T>(TL::row_frag(row_lane, qt, n, ds), kf[ds], s);
                const Frag<T> vd = VLDS ? *(const Frag<T>*)(smem + kVals + (wave * (DP / 16) + ds) * 1024 + lane * 16) : vf[VLDS ? 0 : ds];
                dp = mma<T>(TL::row_frag(row_lane, ot, n, ds), vd, dp);
            }
            const float* st = (const float*)(smem + kStat + buf * 512) + n * 32 + 4 * h;
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
            if (key0 + 32 > w.len || (a.causal && key0 + 31 > imin)) {
                // first row that sees the key
                const int first = there ? (a.causal ? min(max(key - w.start, 0), a.Sq) * a.pack : 0) : 0x7fffffff;
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = rs + acc_row(i, h) >= first ? p[i] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Frag<T> pf = pack_frag<T>(p + 8 * k);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt)
                    dv[dt] = mma<T>(TL::col_frag(col_at, col_at8, ot, n * 32 + k * 16, dt), pf, dv[dt]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] *= dp[i] - st[64 + 8 * (i / 4) + (i % 4)];
            if constexpr (BIAS) {
                // rows past the end have q = dO = 0 and delta = 0: dS = 0
                if (near) {
                    float* at = diag + (31 - 4 * h + (lane & 31)) * kDiagPitch + (lane & 31);
#pragma unroll
                    for (int i = 0; i < 16; ++i) at[-(8 * (i / 4) + (i % 4)) * kDiagPitch] = p[i];
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    float d = 0.0f;
#pragma unroll
                    for (int x = 0; x < 32; ++x) d += diag[lane * kDiagPitch + x];
                    // lane 63 has no diagonal: its row of the scratch is never written
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
        for (int x = (int)threadIdx.x; x < entries; x += NW * 64) {
            float s = sums[x];
            for (int k = 1; k < NW; ++k) s += sums[k * entries + x];
            a.tpart[w.flat * entries + x] = s;
        }
    }
    if (key0 >= a.Sk) return;
    const bool in = key < a.Sk;
    const int parts = a.nsplit * (a.G / a.pack);   // float32 parts of each key head
    if (parts == 1) {
        const int64_t kk = min(key, a.Sk - 1);
        store_acc<T, DP, VEC>(a.dk + w.b * a.dks.b + kk * a.dks.s + w.kv * a.dks.h, dk, a.scale, a.D, in, h);
        store_acc<T, DP, VEC>(a.dv + w.b * a.dvs.b + kk * a.dvs.s + w.kv * a.dvs.h, dv, 1.0f, a.D, in, h);
    } else {
        // [part][dk, dv][B, Hkv, Sk, DP]
        const int64_t heads = (int64_t)a.B * a.Hkv, part = (w.head % a.G) / a.pack + (int64_t)(a.G / a.pack) * w.split;
        const int64_t at = ((part * 2 * heads + (int64_t)w.b * a.Hkv + w.kv) * a.Sk + min(key, a.Sk - 1)) * DP;
        store_part<DP>(a.part + at, dk, a.scale, in, h);
        store_part<DP>(a.part + at + heads * a.Sk * DP, dv, 1.0f, in, h);
    }
}

// Sums float32 parts in order and rounds once: out[b, s, h] = sum_p part[p]
// [(b, hu)][row][DP] with row = s * pack + g and h = hu * pack + g. One part
// lies `stride` floats after the other. DP / 4 threads per row. With `delta`
// (dq's sum) the parts of `rest` [part][b, head, i] are added to it.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attn_sum_kernel(SumArgs x) {
    constexpr int TPR = DP / 4, PER = 256 / TPR;
    int64_t at = (int64_t)blockIdx.x * PER + (int)threadIdx.x / TPR;
    const int d = ((int)threadIdx.x % TPR) * 4;
    // workgroups past the first sum's rows make the second
    const int64_t first = (x.total + PER - 1) / PER;
    const bool second = (int64_t)blockIdx.x >= first;
    if (second) at -= first * PER;
    const float* part = second ? x.part2 : x.part;
    if ((int)threadIdx.x >= PER * TPR || at >= x.total) return;
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

}  // namespace dytb
