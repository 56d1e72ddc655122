// attn_api.hip - C ABI of attention (include/dyt_block.h): argument checks,
// the split of the work, and the bias gradient's last sum.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "attn_launch.hpp"
#include "block_host.hpp"
#include "dyt_block.h"

namespace dytb {

// dtable[t, head]: bucket t's run of positions in the rows of the head's
// workgroups, batch entry by batch entry. A workgroup per (head, bucket); the
// order of the sum depends on the shape alone. Bound by the loads' latency:
// sixteen waves take 5.8 us for 512 runs over 64 rows, four took 10.5.
constexpr int kTableThreads = 1024;

__global__ __launch_bounds__(kTableThreads) void attn_dtable_kernel(const float* part, int B, int Hq, int per_unit,
                                                                    int buckets, Borders o, void* dtable, int dt) {
    __shared__ float red[kTableThreads / 64];
    const int head = (int)blockIdx.x / buckets, t = (int)blockIdx.x - head * buckets;
    int lo, hi;
    bucket_range(o, t, lo, hi);
    const int entries = bias_entries(o), run = max(hi - lo, 0);
    float s = 0.0f;
    // rows of the head: a wave (or a part of one) along each row's run
    const int width = run <= 8 ? 8 : run <= 32 ? 32 : 64;
    const int lane = (int)threadIdx.x % width, side = kTableThreads / width;
#pragma unroll 4
    for (int x = (int)threadIdx.x / width; x < B * per_unit; x += side) {
        const int b = x / per_unit, k = x - b * per_unit;
        const float* row = part + (((int64_t)b * Hq + head) * per_unit + k) * entries + lo;
        for (int i = lane; i < run; i += width) s += row[i];
    }
    s = lanes_sum<64>(s);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kTableThreads / 64; ++k) s += red[k];
        store_param(dtable, (int64_t)t * Hq + head, dt, s);
    }
}

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 28;   // Sq * G, Sk: 32-bit row arithmetic in the kernels

int fill_borders(int num_buckets, int max_distance, int bidirectional, Borders& o) {
    if (num_buckets < 2 || num_buckets > DYT_ATTN_MAX_BUCKETS || max_distance < 1 ||
        max_distance > DYT_ATTN_MAX_DISTANCE || (bidirectional && num_buckets % 2))
        return DYT_ERR_INVALID_ARG;
    o.bidirectional = bidirectional;
    o.n = bidirectional ? num_buckets / 2 : num_buckets;
    o.e = o.n / 2;
    if (o.n < 2 || max_distance <= o.e) return DYT_ERR_INVALID_ARG;
    const int t_all = o.n - o.e;
    for (int d = 0; d < o.e; ++d) o.at[d] = d;
    // bucket e + t starts at the smallest d >= e (distance / e)^(t / (n - e)); the
    // powers are off by 1e-17 relative, and where one is a whole number d is it
    const long double ratio = expl(logl((long double)max_distance / o.e) / t_all);
    long double at = o.e;
    for (int t = 0; t < t_all; ++t, at *= ratio) o.at[o.e + t] = (int)ceill(at * (1 - 1e-13L));
    o.reach = o.at[o.n - 1];
    return DYT_OK;
}

struct Tensor {
    int64_t S, H;
    const dyt_attn_strides* st;
};

// Byte strides for the kernels (0 along dimensions of one element or none)
// and the span of the tensor in bytes; false where they overflow.
bool view(const dyt_attn_desc& d, const Tensor& t, bool out, Strides& s, int64_t& span) {
    const int64_t es = dtype_size(d.dtype);
    const int64_t size[3] = {d.B, t.S, t.H}, stride[3] = {t.st->b, t.st->s, t.st->h};
    int64_t bytes[3];
    s = Strides{0, 0, 0};
    span = 0;
    if (!size[0] || !size[1] || !size[2]) return true;
    span = d.D * es;
    for (int i = 0; i < 3; ++i) {
        bytes[i] = 0;
        if (size[i] <= 1) continue;
        if (stride[i] < 0 || stride[i] > (((int64_t)1 << 60) / es) / size[i]) return false;
        bytes[i] = stride[i] * es;
        span += bytes[i] * (size[i] - 1);
        if (span > ((int64_t)1 << 61)) return false;
    }
    if (out) {
        // no two elements of an output share memory: every dimension steps
        // over all of the faster ones
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [&](int x, int y) { return bytes[x] < bytes[y]; });
        int64_t covered = d.D * es;
        for (int i : order) {
            if (size[i] <= 1) continue;
            if (bytes[i] < covered) return false;
            covered = bytes[i] * (size[i] - 1) + covered;
        }
    }
    s = Strides{bytes[0], bytes[1], bytes[2]};
    return true;
}

// One output's rows: up to three dimensions that step over each other, the
// largest stride first, and the bytes of a row.
struct Layout {
    struct { int64_t n, stride; } dim[3];
    int dims;
    int64_t row;
    Layout(const int64_t (&size)[3], const Strides& s, int64_t row_bytes) : dims(0), row(row_bytes) {
        const int64_t stride[3] = {s.b, s.s, s.h};
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1) dim[dims++] = {size[i], stride[i]};
        std::sort(dim, dim + dims, [](const auto& x, const auto& y) { return x.stride > y.stride; });
    }
    int64_t extent(int from) const {
        int64_t n = row;
        for (int i = from; i < dims; ++i) n += (dim[i].n - 1) * dim[i].stride;
        return n;
    }
};

// Whether x from its dimension i on and y from j on, `delta` bytes behind it,
// share a byte. The larger stride (or both, where they are the same) is taken
// out, and only those of its multiples are tried at which what is left can
// meet: two or three for slices of one tensor. Layouts that need more than
// `tries` in all count as sharing.
bool share(const Layout& x, int i, const Layout& y, int j, int64_t delta, int& tries) {
    const int64_t ex = x.extent(i), ey = y.extent(j);
    if (delta >= ex || delta <= -ey) return false;
    if (--tries < 0 || (i == x.dims && j == y.dims)) return true;
    const int64_t sx = i < x.dims ? x.dim[i].stride : 0, sy = j < y.dims ? y.dim[j].stride : 0, step = std::max(sx, sy);
    const int64_t nx = sx == step ? x.dim[i].n - 1 : 0, ny = sy == step ? y.dim[j].n - 1 : 0;
    const int ii = i + (sx == step), jj = j + (sy == step);
    // delta + k step within (-rest of y, rest of x)
    const int64_t rx = ex - nx * step, ry = ey - ny * step;
    const auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const int64_t lo = std::max(-nx, floor_div(-ry - delta, step) + 1), hi = std::min(ny, -floor_div(delta - rx, step) - 1);
    for (int64_t k = lo; k <= hi; ++k)
        if (share(x, ii, y, jj, delta + k * step, tries)) return true;
    return false;
}

// Whether a tensor takes 16-byte accesses: aligned base, strides and rows.
bool vec_ok(const void* p, const Strides& s, int64_t row_bytes) {
    return (uintptr_t)p % 16 == 0 && s.b % 16 == 0 && s.s % 16 == 0 && s.h % 16 == 0 && row_bytes % 16 == 0;
}

// Whether the rows of a tile, up to 128 of `pack` heads to a position, lie
// within the 31-bit offsets of the direct-to-LDS loads. Keys and values (pack
// 1) go head by head: how far apart their heads are does not matter.
bool tile_ok(const Strides& s, int pack, int64_t row_bytes) {
    constexpr int64_t limit = (int64_t)1 << 31;
    if (s.s >= limit || (pack > 1 && s.h >= limit)) return false;
    return 127 / pack * s.s + (pack > 1 ? (pack - 1) * s.h : 0) + row_bytes < limit;
}

// The rows of a unit: all heads of a group (or a 32-row tile's worth, the
// largest divisor), unless each needs its own column of the table.
int pack_of(const dyt_attn_desc& d) {
    int pack = 1;
    const int64_t G = d.Hq / d.Hkv;
    if (!d.table)
        for (int n = 2; n <= 32 && n <= G; ++n)
            if (G % n == 0) pack = n;
    return pack;
}

struct Plan {
    int64_t rows;
    AttnPick fwd, dq, dkv;
    int pack, units;
    int fwd_blocks, fwd_split, fwd_per;
    int dq_blocks, dq_split, dq_per;
    int dkv_blocks, dkv_split, dkv_per, dkv_parts;
    int fwd_lds, dq_lds, dkv_lds;
    int per_unit;   // dkv workgroups of a head
    size_t fwd_bytes, bwd_bytes;
    size_t off_rest, off_tpart, off_part;   // backward workspace: rows, rest, tpart, part
    bool nothing_out, nothing_keys;
    Borders borders{};
};

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// How a kernel's work is cut. Workgroups of four row groups share each tile
// of the long axis; smaller ones each bring their own, which the L2 only
// keeps up with while they are few. So four wherever their workgroups, with
// the long axis cut into runs of 1,024, would fill the 256 CUs, and one
// below (and for up to 32 rows, one group's).
//
// Those of one row group may have 2 or 4 slices, and the long axis may be
// cut into a power of two of splits; the pair is taken that minimises
//   rounds * steps * max(lat, waves per SIMD * busy) + join,
// steps of 32 per slice, rounds of the workgroups that the LDS of 256 CUs
// holds (several slices: all of a workgroup's waves end together). A wave
// alone on its SIMD takes `lat` for a step (the chain of loads, products and
// exponentials), and a SIMD is `busy` with it. Slices join in LDS (0.5 us a
// pair), splits in a launch of its own (6 us, 0.1 us for each part it reads).
struct Shape {
    int es, dp, pack;
    int extra, extra_wave;   // LDS of the bias: of a workgroup, of each wave
    bool dkv, whole;         // whole: no splits
    double lat, busy;
    int tile(int nw, int sl) const {
        return (dkv ? attn_dkv_tile_rows(es, dp, nw, sl) : attn_tile_rows(es, nw, sl)) / pack * pack;   // whole positions
    }
    int lds(int nw, int sl) const {
        return (dkv ? attn_dkv_lds_bytes(es, dp, nw, sl) : attn_lds_bytes(es, dp, nw, sl)) + extra + extra_wave * nw * sl;
    }
};

int choose(const Shape& h, int64_t units, int64_t rows, int64_t len, AttnPick& pick, int& blocks, int& split, int& per) {
    const int64_t b4 = units * ((rows + 127) / 128);
    pick.nw = pick.vec && rows > 32 && b4 * std::max<int64_t>(1, len / 1024) >= 256 ? 4 : 1;
    const int nw = pick.nw;
    blocks = ceil_div(rows, 32 * nw);
    const double groups = (double)units * blocks;
    double best = 0.0;
    int64_t parts = 1;
    pick.sl = 1;
    // dk/dv above dp = 64, where a CU holds eight waves: all on one block of keys
    // at a time, so that under a causal mask the next block goes to whichever CU
    // is free (2 x 8 key heads of 4,096, D = 128: 842 -> 655 us)
    const int lo = nw == 4 && h.dkv && dkv_vals_in_lds(h.es, h.dp) && h.lds(4, 2) <= kMaxLds ? 2 : 1;
    const int hi = nw == 4 ? lo : pick.vec ? 4 : 1;
    for (int sl = lo; sl <= hi; sl *= 2) {
        if (h.lds(nw, sl) > kMaxLds || (sl == 4 && attn_lds_bytes(h.es, h.dp, 1, 4) > kMaxLds)) break;
        const int tile = h.tile(nw, sl), steps = (tile + 32 * sl - 1) / (32 * sl);
        const int64_t tiles = std::max<int64_t>(1, ceil_div(len, tile));
        const double resident = 256.0 * (kMaxLds / h.lds(nw, sl));
        for (int64_t n = 1; n == 1 || (!h.whole && n <= 64 && n * 4 <= tiles); n *= 2) {
            double at_once = groups * n, rounds = 1.0;
            if (nw == 1 && sl > 1 && at_once > resident) {
                rounds = std::ceil(at_once / resident);
                at_once = resident;
            }
            const double t = rounds * ceil_div(tiles, n) * steps * std::max(h.lat, at_once * nw * sl / 1024.0 * h.busy) +
                             0.5 * (sl - 1) + (n > 1 ? 6.0 + 0.1 * n : 0.0);
            if (best == 0.0 || t < best) {
                best = t;
                parts = n;
                pick.sl = sl;
            }
        }
    }
    const int tile = h.tile(nw, pick.sl);
    // One block of rows (single tokens): every key is read once, and what counts
    // are the loads in flight. Once the keys are split, they are split until
    // every CU has all the workgroups it holds (16 x 16 heads over 4,096 keys, D =
    // 64: 45 us with 2,048 workgroups, 41 with 4,096; where 1,280 are held, D =
    // 128, 73 us with 2,048 and 76 with 4,096).
    if (!h.dkv && rows <= 32 && pick.sl == 1 && parts > 1) {
        const double held = 256.0 * (kMaxLds / h.lds(nw, 1));
        while (groups * parts < held && parts < 64 && parts * 8 <= ceil_div(len, tile)) parts *= 2;
    }
    per = ceil_div(ceil_div(len, tile), parts) * tile;
    per = std::max(per, tile);
    split = std::max(1, ceil_div(len, per));
    return h.lds(nw, pick.sl);
}

// The order of the work under a causal mask (find_work): an XCD takes as many
// units at a time as give each of its 32 CUs four workgroups; a CU holds what
// its LDS (`lds` bytes a workgroup) and registers allow.
void set_order(AttnArgs& a, const AttnPick& pick, int lds, int es) {
    const int per_cu = std::min(kMaxLds / lds, 4 * attn_waves(es) / (pick.nw * pick.sl));
    a.together = a.causal ? std::max(1, std::min(a.units / 8, 128 / (a.blocks * a.nsplit))) : 1;
    a.zigzag = a.causal && per_cu > 1;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

int check(const dyt_attn_desc& d, Borders& borders) {
    if (d.B < 0 || d.Sq < 0 || d.Sk < 0 || d.Hq < 0 || d.Hkv < 1 || d.D < 1 || d.D > DYT_ATTN_MAX_D)
        return DYT_ERR_INVALID_ARG;
    if (d.Hq % d.Hkv || (d.causal & ~1) || (d.bidirectional & ~1) || d.reserved) return DYT_ERR_INVALID_ARG;
    if (!(d.scale > 0.0f) || std::isinf(d.scale)) return DYT_ERR_INVALID_ARG;
    const int64_t G = d.Hq / d.Hkv;
    if (d.Sk > kMaxRows || d.Sq > kMaxRows || G > kMaxRows || d.Sq * std::max<int64_t>(G, 1) > kMaxRows)
        return DYT_ERR_INVALID_ARG;
    if (d.Hq > (1 << 20) || d.Hkv > (1 << 20) || d.B > (1 << 24) || d.B * d.Hq > (1 << 24) || d.B * d.Hkv > (1 << 24))
        return DYT_ERR_INVALID_ARG;
    if (!dtype_ok(d.dtype) || (d.table && !dtype_ok(d.table_dtype))) return DYT_ERR_UNSUPPORTED_DTYPE;
    return d.table ? fill_borders(d.num_buckets, d.max_distance, d.bidirectional, borders) : DYT_OK;
}

// vec: whether every tensor takes 16-byte accesses (single waves otherwise).
Plan make_plan(const dyt_attn_desc& d, const Borders& borders, bool backward, bool vec) {
    Plan p{};
    const int64_t G = d.Hq / d.Hkv;
    p.borders = borders;
    p.nothing_out = d.B == 0 || d.Sq == 0 || d.Hq == 0;
    p.nothing_keys = d.B == 0 || d.Sk == 0;
    p.pack = pack_of(d);
    p.units = (int)(d.B * (d.Hq / p.pack));
    p.rows = d.Sq * p.pack;
    const int dp = attn_dp(d.D), es = (int)dtype_size(d.dtype);
    p.fwd = p.dq = p.dkv = {dp, 1, 1, d.table != nullptr, vec};
    // us per 32 keys (rows), measured at D = 32 (float32: the matrix cores'
    // rate) and, 16-bit, much the same up to 128
    const double f = d.dtype == DYT_F32 ? 2.2 * dp / 32 : 0.0;
    const int bias = d.table ? bias_lds_bytes(p.borders) : 0, dbias = d.table ? dbias_lds_bytes(p.borders, 1) : 0;
    if (!p.nothing_out && !backward)
        p.fwd_lds = choose({es, dp, 1, bias, 0, false, false, std::max(f, 0.8), std::max(f, 0.4)}, p.units, p.rows, d.Sk, p.fwd,
                           p.fwd_blocks, p.fwd_split, p.fwd_per);
    if (!p.nothing_out && backward)
        p.dq_lds = choose({es, dp, 1, bias, 0, false, es == 2 && d.Sk <= kRefineKeys, std::max(1.2 * f, 0.9),
                           std::max(1.2 * f, 0.6)}, p.units, p.rows, d.Sk, p.dq, p.dq_blocks, p.dq_split, p.dq_per);
    if (!p.nothing_keys && d.Hq > 0 && backward)
        p.dkv_lds = choose({es, dp, p.pack, bias, dbias, true, false, std::max(1.7 * f, 1.2), std::max(1.7 * f, 0.9)}, p.units,
                           d.Sk, p.rows, p.dkv, p.dkv_blocks, p.dkv_split, p.dkv_per);
    const int64_t part_rows = p.units * p.rows * (int64_t)dp * 4;
    if (p.fwd_split > 1) p.fwd_bytes = round256((size_t)p.fwd_split * part_rows) + (size_t)p.fwd_split * p.units * p.rows * 8;
    p.per_unit = p.dkv_blocks * p.dkv_split;
    p.off_rest = round256((size_t)2 * d.B * d.Hq * d.Sq * 4);
    p.off_tpart = p.off_rest + (p.dq_split > 1 ? round256((size_t)p.dq_split * d.B * d.Hq * d.Sq * 4) : 0);
    p.off_part = p.off_tpart + (d.table ? round256((size_t)p.units * p.per_unit * 2 * (p.borders.reach + kPad) * 4) : 0);
    p.dkv_parts = p.dkv_split * (int)(d.Hq > 0 ? G / p.pack : 1);
    size_t part = p.dq_split > 1 ? (size_t)p.dq_split * part_rows : 0;
    if (p.dkv_parts > 1) part = std::max(part, (size_t)p.dkv_parts * 2 * d.B * d.Hkv * d.Sk * dp * 4);
    p.bwd_bytes = p.off_part + part;
    return p;
}

// A launch has fewer than 2^32 threads. (The sums of float32 parts walk.)
bool launches_fit(const dyt_attn_desc& d, const Plan& p, bool backward) {
    const auto fit = [](int64_t groups, int threads) { return groups * threads < ((int64_t)1 << 32); };
    const auto main = [&](const AttnPick& pick, int blocks, int split) {
        return fit((int64_t)p.units * blocks * split, pick.nw * pick.sl * 64);
    };
    if (!backward)
        return main(p.fwd, p.fwd_blocks, p.fwd_split) && (p.fwd_split == 1 || fit(p.units * p.rows, p.fwd.dp / 4 * 8));
    return main(p.dq, p.dq_blocks, p.dq_split) && main(p.dkv, p.dkv_blocks, p.dkv_split) &&
           (!d.table || fit(d.Hq * d.num_buckets, kTableThreads));
}

template <typename F>
int with_type(int dt, F&& f) {
    if (dt == DYT_F32) return f((float*)nullptr);
    if (dt == DYT_BF16) return f((bf16_t*)nullptr);
    return f((f16_t*)nullptr);
}

void fill_args(const dyt_attn_desc& d, const Plan& p, AttnArgs& a) {
    a.lens = d.seqlens_k;
    a.starts = d.q_start;
    a.table = d.table;
    a.B = (int)d.B; a.Sq = (int)d.Sq; a.Sk = (int)d.Sk; a.Hq = (int)d.Hq; a.Hkv = (int)d.Hkv; a.D = (int)d.D;
    a.G = (int)std::max<int64_t>(d.Hq / d.Hkv, 1);
    a.pack = p.pack;
    a.units = p.units;
    a.causal = d.causal;
    a.table_dt = d.table_dtype;
    a.buckets = d.num_buckets;
    a.scale = d.scale;
    a.borders = p.borders;
}

struct Spans {
    int64_t q, k, v, o, dout, dq, dk, dv;
};

bool lists_aligned(const dyt_attn_desc& d) {
    return aligned({d.seqlens_k, d.q_start}, 4) && (!d.table || aligned({d.table}, dtype_size(d.table_dtype)));
}

}  // namespace
}  // namespace dytb

using namespace dytb;

extern "C" {

int dyt_attn_bucket_borders(int num_buckets, int max_distance, int bidirectional, int32_t* borders) {
    Borders o;
    if (!borders || (bidirectional & ~1) || fill_borders(num_buckets, max_distance, bidirectional, o)) return 0;
    for (int i = 0; i < o.n; ++i) borders[i] = o.at[i];
    return o.n;
}

size_t dyt_attn_forward_workspace_size(const dyt_attn_desc* desc) {
    if (!desc) return 0;
    Borders borders{};
    if (check(*desc, borders)) return 0;
    const Plan p = make_plan(*desc, borders, false, true), each = make_plan(*desc, borders, false, false);
    if (p.nothing_out || !launches_fit(*desc, p, false) || !launches_fit(*desc, each, false)) return 0;
    return std::max(p.fwd_bytes, each.fwd_bytes);
}

size_t dyt_attn_backward_workspace_size(const dyt_attn_desc* desc) {
    if (!desc) return 0;
    Borders borders{};
    if (check(*desc, borders)) return 0;
    const Plan p = make_plan(*desc, borders, true, true), each = make_plan(*desc, borders, true, false);
    if (!launches_fit(*desc, p, true) || !launches_fit(*desc, each, true)) return 0;
    return std::max(p.bwd_bytes, each.bwd_bytes);
}

int dyt_attn_forward(const dyt_attn_desc* desc, const void* q, const void* k, const void* v, void* o, float* stats,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!desc) return DYT_ERR_INVALID_ARG;
    const dyt_attn_desc& d = *desc;
    Borders borders{};
    if (int st = check(d, borders)) return st;
    AttnArgs a{};
    Spans n{};
    if (!view(d, {d.Sq, d.Hq, &d.q}, false, a.qs, n.q) || !view(d, {d.Sk, d.Hkv, &d.k}, false, a.ks, n.k) ||
        !view(d, {d.Sk, d.Hkv, &d.v}, false, a.vs, n.v) || !view(d, {d.Sq, d.Hq, &d.o}, true, a.os, n.o))
        return DYT_ERR_INVALID_ARG;
    const int64_t es = dtype_size(d.dtype), row = d.D * es;
    const Plan p = make_plan(d, borders, false, vec_ok(q, a.qs, row) && vec_ok(k, a.ks, row) && vec_ok(v, a.vs, row) &&
                                                    vec_ok(o, a.os, row) && tile_ok(a.ks, 1, row) && tile_ok(a.vs, 1, row));
    if (p.nothing_out) return DYT_OK;
    if (!launches_fit(d, p, false)) return DYT_ERR_INVALID_ARG;
    if (!q || !o || !stats || (d.Sk > 0 && (!k || !v))) return DYT_ERR_INVALID_ARG;
    if (d.Sk == 0) n.k = n.v = 0;
    if (!aligned({q, k, v, o}, es) || !aligned({stats}, 4) || !lists_aligned(d)) return DYT_ERR_MISALIGNED;
    if (p.fwd_bytes && (!workspace || workspace_bytes < p.fwd_bytes)) return DYT_ERR_WORKSPACE_TOO_SMALL;
    if (p.fwd_bytes && !aligned({workspace}, 16)) return DYT_ERR_MISALIGNED;
    const Range in[] = {{q, n.q}, {k, n.k}, {v, n.v}, {d.seqlens_k, d.B * 4}, {d.q_start, d.B * 4},
                        {d.table, d.table ? d.num_buckets * d.Hq * dtype_size(d.table_dtype) : 0}};
    const Range out[] = {{o, n.o}, {stats, d.B * d.Hq * d.Sq * 4}, {workspace, (int64_t)p.fwd_bytes}};
    if (!disjoint(in, 6, out, 3)) return DYT_ERR_INVALID_ARG;
    fill_args(d, p, a);
    a.q = (const char*)q; a.k = (const char*)k; a.v = (const char*)v; a.out = (char*)o; a.stats = stats;
    a.blocks = p.fwd_blocks; a.nsplit = p.fwd_split; a.per_split = p.fwd_per;
    set_order(a, p.fwd, p.fwd_lds, (int)es);
    a.part = (float*)workspace;
    a.part_ml = (float*)((char*)workspace + round256((size_t)p.fwd_split * p.units * p.rows * p.fwd.dp * 4));
    return with_type(d.dtype, [&](auto* t) {
        return attn_launch_fwd<std::remove_pointer_t<decltype(t)>>(p.fwd, a, (hipStream_t)stream);
    });
}

int dyt_attn_backward(const dyt_attn_desc* desc, const void* q, const void* k, const void* v, const void* o,
                      const void* dout, const float* stats, void* dq, void* dk, void* dv, void* dtable,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!desc) return DYT_ERR_INVALID_ARG;
    const dyt_attn_desc& d = *desc;
    Borders borders{};
    if (int st = check(d, borders)) return st;
    AttnArgs a{};
    Spans n{};
    if (!view(d, {d.Sq, d.Hq, &d.q}, false, a.qs, n.q) || !view(d, {d.Sk, d.Hkv, &d.k}, false, a.ks, n.k) ||
        !view(d, {d.Sk, d.Hkv, &d.v}, false, a.vs, n.v) || !view(d, {d.Sq, d.Hq, &d.o}, false, a.os, n.o) ||
        !view(d, {d.Sq, d.Hq, &d.dout}, false, a.dos, n.dout) || !view(d, {d.Sq, d.Hq, &d.dq}, true, a.dqs, n.dq) ||
        !view(d, {d.Sk, d.Hkv, &d.dk}, true, a.dks, n.dk) || !view(d, {d.Sk, d.Hkv, &d.dv}, true, a.dvs, n.dv))
        return DYT_ERR_INVALID_ARG;
    const int64_t es = dtype_size(d.dtype), row = d.D * es, ts = d.table ? dtype_size(d.table_dtype) : 1;
    const int pack = pack_of(d);
    const Plan p = make_plan(d, borders, true, vec_ok(q, a.qs, row) && vec_ok(k, a.ks, row) && vec_ok(v, a.vs, row) &&
                                    vec_ok(o, a.os, row) && vec_ok(dout, a.dos, row) && vec_ok(dq, a.dqs, row) &&
                                    vec_ok(dk, a.dks, row) && vec_ok(dv, a.dvs, row) &&
                                    tile_ok(a.ks, 1, row) && tile_ok(a.vs, 1, row) && tile_ok(a.qs, pack, row) &&
                                    tile_ok(a.dos, pack, row));
    if (!launches_fit(d, p, true)) return DYT_ERR_INVALID_ARG;
    if (p.nothing_out) n.q = n.o = n.dout = n.dq = 0;
    if (p.nothing_keys) n.k = n.v = n.dk = n.dv = 0;
    if (!p.nothing_out && (!q || !o || !dout || !stats || !dq)) return DYT_ERR_INVALID_ARG;
    if (!p.nothing_keys && (!k || !v || !dk || !dv)) return DYT_ERR_INVALID_ARG;
    if (d.table && !dtable) return DYT_ERR_INVALID_ARG;
    if (!aligned({q, k, v, o, dout, dq, dk, dv}, es) || !aligned({stats}, 4) || !lists_aligned(d) ||
        (d.table && !aligned({dtable}, ts)))
        return DYT_ERR_MISALIGNED;
    const int64_t tb = d.table ? d.num_buckets * d.Hq * ts : 0;
    const Range in[] = {{q, n.q}, {k, n.k}, {v, n.v}, {o, n.o}, {dout, n.dout},
                        {stats, p.nothing_out ? 0 : d.B * d.Hq * d.Sq * 4},
                        {d.seqlens_k, d.B * 4}, {d.q_start, d.B * 4}, {d.table, tb}};
    // dq, dk and dv may be interleaved slices of one tensor: each is held
    // against the inputs, the workspace and dtable as a range, against each
    // other element by element
    const Range outs[] = {{dq, n.dq}, {dk, n.dk}, {dv, n.dv}};
    const Range rest[] = {{dtable, tb}, {workspace, (int64_t)p.bwd_bytes}};
    const int64_t of_q[] = {d.B, d.Sq, d.Hq}, of_k[] = {d.B, d.Sk, d.Hkv};
    const Layout layouts[] = {{of_q, a.dqs, row}, {of_k, a.dks, row}, {of_k, a.dvs, row}};
    for (int i = 0; i < 3; ++i) {
        if (!disjoint(in, 9, outs + i, 1) || !disjoint(rest, 2, outs + i, 1)) return DYT_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j) {
            int tries = 4096;
            if (meet(outs[i], outs[j]) && share(layouts[i], 0, layouts[j], 0, (const char*)outs[j].p - (const char*)outs[i].p, tries))
                return DYT_ERR_INVALID_ARG;
        }
    }
    if (!disjoint(in, 9, rest, 2)) return DYT_ERR_INVALID_ARG;
    if (p.bwd_bytes && (!workspace || workspace_bytes < p.bwd_bytes)) return DYT_ERR_WORKSPACE_TOO_SMALL;
    if (p.bwd_bytes && !aligned({workspace}, 16)) return DYT_ERR_MISALIGNED;
    if (p.nothing_out && p.nothing_keys && !(d.table && d.Hq > 0)) return DYT_OK;

    const hipStream_t s = (hipStream_t)stream;
    fill_args(d, p, a);
    a.q = (const char*)q; a.k = (const char*)k; a.v = (const char*)v; a.o = (const char*)o;
    a.dout = (const char*)dout; a.dq = (char*)dq; a.dk = (char*)dk; a.dv = (char*)dv;
    a.stats = const_cast<float*>(stats);
    a.dtable = dtable;
    a.rows = (float*)workspace;
    a.rest = (float*)((char*)workspace + p.off_rest);
    a.tpart = (float*)((char*)workspace + p.off_tpart);
    a.part = (float*)((char*)workspace + p.off_part);
    return with_type(d.dtype, [&](auto* t) {
        typedef std::remove_pointer_t<decltype(t)> T;
        const int dp = p.dq.dp;
        if (!p.nothing_out) {
            a.blocks = p.dq_blocks; a.nsplit = p.dq_split; a.per_split = p.dq_per;
            set_order(a, p.dq, p.dq_lds, (int)es);
            if (int st = attn_launch_dq<T>(p.dq, a, s)) return st;
            if (p.dq_split > 1) {
                const int64_t total = (int64_t)p.units * p.rows;
                SumArgs sum{};
                sum.part = a.part; sum.stride = total * dp; sum.parts = p.dq_split;
                sum.out = (char*)dq; sum.os = a.dqs; sum.total = total; sum.rows = (int)p.rows; sum.pack = p.pack;
                sum.hu = (int)(d.Hq / p.pack); sum.D = (int)d.D;
                sum.delta = a.rows + (int64_t)d.B * d.Hq * d.Sq;
                sum.rest = a.rest;
                attn_launch_sum<T>(dp, sum, s);
            }
        }
        if (!p.nothing_keys) {
            const int64_t total = d.B * d.Hkv * d.Sk, stride = 2 * total * dp;
            SumArgs sums{};
            sums.part = a.part; sums.stride = stride; sums.parts = d.Hq ? p.dkv_parts : 0;   // no head: zeros
            sums.out = (char*)dk; sums.os = a.dks; sums.total = total; sums.rows = (int)d.Sk; sums.pack = 1;
            sums.hu = (int)d.Hkv; sums.D = (int)d.D;
            sums.part2 = a.part + total * dp; sums.out2 = (char*)dv; sums.os2 = a.dvs;
            if (d.Hq == 0) {
                attn_launch_sum<T>(dp, sums, s);
                return hip_status();
            }
            a.blocks = p.dkv_blocks; a.nsplit = p.dkv_split; a.per_split = p.dkv_per;
            set_order(a, p.dkv, p.dkv_lds, (int)es);
            if (int st = attn_launch_dkv<T>(p.dkv, a, s)) return st;
            if (p.dkv_parts > 1) attn_launch_sum<T>(dp, sums, s);
        }
        if (d.table && d.Hq > 0)
            attn_dtable_kernel<<<(unsigned)(d.Hq * d.num_buckets), kTableThreads, 0, s>>>(
                a.tpart, p.nothing_keys ? 0 : (int)d.B, (int)d.Hq, p.nothing_keys ? 1 : p.per_unit, d.num_buckets,
                p.borders, dtable, d.table_dtype);
        return hip_status();
    });
}

}  // extern "C"
