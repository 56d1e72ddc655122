"""Attention and its gradients on the GPU against the formulas in float64
(tests/block_ref.py: every tolerance is derived there from the roundings)."""
import math

import pytest
import torch

from block_ref import Attention, d

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


def make(seed, dt, B, Sq, Sk, Hq, Hkv, D, *, buckets=0, table_dt=None, lens=None, starts=None, causal=False,
         distance=128, bidirectional=True, scale=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()
    t = dict(q=r(B, Sq, Hq, D), k=r(B, Sk, Hkv, D), v=r(B, Sk, Hkv, D))
    do = r(B, Sq, Hq, D)
    kw = dict(causal=causal)
    if scale is not None:
        kw["scale"] = scale
    if lens is not None:
        kw["seqlens_k"] = torch.tensor(lens, dtype=torch.int32).cuda()
    if starts is not None:
        kw["q_start"] = torch.tensor(starts, dtype=torch.int32).cuda()
    if buckets:
        kw.update(table=torch.randn(buckets, Hq, generator=g).to(table_dt or dt).cuda(), max_distance=distance,
                  bidirectional=bidirectional)
    return t, do, kw


def run_and_check(dyt, t, do, kw, backward=True):
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    ref = Attention(t["q"], t["k"], t["v"], **kw)
    ref.check_forward(o, stats)
    if not backward:
        return (o, stats)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    ref.check_backward(do, *grads)
    return (o, stats, *grads)


# B, Sq, Sk, Hq, Hkv, D
SIZES = [
    (1, 1, 1, 1, 1, 1), (2, 1, 33, 2, 1, 8), (1, 31, 32, 1, 1, 16), (3, 33, 65, 2, 2, 32), (2, 64, 64, 3, 3, 40),
    (1, 129, 127, 6, 2, 64), (2, 100, 257, 5, 1, 80), (1, 200, 200, 7, 1, 96), (1, 70, 300, 12, 3, 100),
    (2, 130, 130, 4, 2, 128), (1, 65, 40, 8, 1, 127), (1, 3, 700, 33, 1, 24), (1, 2, 90, 64, 1, 48),
    (4, 1, 1500, 8, 2, 128), (1, 1, 5000, 4, 4, 64), (1, 300, 16, 2, 1, 7),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_sizes(dyt, dt, size, causal):
    t, do, kw = make(hash(size) % 1000, DTYPES[dt], *size, causal=causal)
    run_and_check(dyt, t, do, kw)


BIAS = [
    # size, buckets, distance, bidirectional, table type
    ((1, 1, 1, 1, 1, 8), 4, 3, True, "f32"), ((2, 65, 65, 2, 1, 32), 32, 128, True, "f32"),
    ((1, 129, 200, 4, 4, 64), 16, 64, True, "bf16"), ((3, 90, 50, 6, 2, 80), 33, 100, False, "f16"),
    ((1, 260, 260, 2, 2, 128), 64, 256, False, "f32"), ((1, 40, 300, 3, 1, 33), 2, 2, False, "f32"),
    ((1, 130, 1200, 1, 1, 16), 128, 1024, True, "f32"), ((2, 1, 700, 8, 2, 64), 32, 128, False, "f16"),
    ((1, 700, 33, 2, 1, 96), 32, 20, True, "bf16"), ((2, 500, 500, 3, 3, 48), 8, 6, True, "f32"),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", BIAS, ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_bias(dyt, dt, case, causal):
    size, buckets, distance, bidi, tdt = case
    t, do, kw = make(7, DTYPES[dt], *size, buckets=buckets, distance=distance, bidirectional=bidi,
                     table_dt=DTYPES[tdt], causal=causal)
    run_and_check(dyt, t, do, kw)


@pytest.mark.parametrize("buckets", [0, 16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt", DTYPES)
def test_rows_and_keys_that_nothing_meets(dyt, dt, causal, buckets):
    """Empty sequences, lengths past the end, positions before the first key
    and far past the last one; the memory of keys nobody sees is NaN, and
    that of masked rows' neighbours infinite."""
    B, Sq, Sk = 6, 70, 150
    lens, starts = [0, 1, 64, 150, 400, 97], [0, -30, -200, 80, 1000, 27]
    t, do, kw = make(3, DTYPES[dt], B, Sq, Sk, 4, 2, 72, lens=lens, starts=starts, causal=causal, buckets=buckets)
    for b in range(B):
        end = min(max(lens[b], 0), Sk)
        if causal:
            end = max(0, min(end, starts[b] + Sq))
        t["k"][b, end:] = math.nan
        t["v"][b, end:] = math.inf if b % 2 else math.nan
    o, stats, dq, dk, dv, *_ = run_and_check(dyt, t, do, kw)
    assert (o[0] == 0).all() and (dq[0] == 0).all() and (dk[0] == 0).all() and (dv[0] == 0).all()
    assert (dk[5, 97:] == 0).all() and (dv[5, 97:] == 0).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("Sq,Sk,Hq", [(0, 5, 2), (5, 0, 2), (0, 0, 2), (3, 4, 0)])
def test_nothing_there(dyt, dt, Sq, Sk, Hq):
    Hkv = 1 if Hq else 2
    t, do, kw = make(1, DTYPES[dt], 2, Sq, Sk, Hq, Hkv, 16, buckets=8)
    kw["table"] = kw["table"].reshape(8, Hq)
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    dq, dk, dv, dtab = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    for x in (o, dq, dk, dv, dtab):
        assert (x == 0).all()
    assert (stats == -math.inf).all()
    e, s = dyt.dyt_attn_forward(t["q"][:0], t["k"][:0], t["v"][:0])
    assert e.shape[0] == 0 and s.shape[0] == 0


@pytest.mark.parametrize("dt", DTYPES)
def test_large_scores_and_offsets(dyt, dt):
    """Scores of a few hundred (one key takes all), and a common offset of
    the keys that the softmax takes out again."""
    t, do, kw = make(5, DTYPES[dt], 2, 90, 300, 4, 2, 64, scale=4.0)
    run_and_check(dyt, t, do, kw)
    t, do, kw = make(6, DTYPES[dt], 1, 64, 200, 2, 2, 32)
    t["q"].abs_().add_(0.5)
    t["k"].sub_(6)
    run_and_check(dyt, t, do, kw)


def test_scores_that_grow_along_the_keys(dyt):
    """Every tile raises the running maximum."""
    t, do, kw = make(8, torch.float32, 1, 40, 640, 2, 1, 32)
    t["q"].fill_(0.5)
    t["k"].mul_(0.05).add_(torch.arange(640).cuda().view(1, -1, 1, 1) * 0.02)
    run_and_check(dyt, t, do, kw)


def test_one_bucket_of_every_pair(dyt):
    """q = 0: the probabilities are those of the bias alone, so every pair's
    bucket shows in them."""
    for causal, bidi in ((False, True), (False, False), (True, False)):
        t, do, kw = make(9, torch.float32, 1, 300, 300, 1, 1, 32, buckets=32, distance=77, bidirectional=bidi,
                         causal=causal)
        t["q"].zero_()
        run_and_check(dyt, t, do, kw)


def test_table_entries_of_minus_infinity_hide_their_buckets(dyt):
    t, do, kw = make(10, torch.float32, 2, 100, 100, 2, 2, 32, buckets=16, distance=30)
    kw["table"][3] = -math.inf
    kw["table"][15] = -math.inf
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    kw["table"] = kw["table"].clamp(min=-1e4)   # exp(-1e4) = 0 as well
    ref = Attention(t["q"], t["k"], t["v"], **kw)
    ref.rho = ref.rho.clamp(max=1e-4)
    ref.check_forward(o, stats)
    for x in grads:
        assert torch.isfinite(x).all()
    assert (grads[3][3] == 0).all() and (grads[3][15] == 0).all()


def _copy_into(t, like):
    like.copy_(t)
    return like


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("layout", ["fused", "heads_first", "offset_one", "odd_pitch", "expanded"])
def test_strides(dyt, dt, layout):
    """Slices of one fused projection, [B, H, S, D] caches, bases and pitches
    off the 16-byte grid, heads that share memory. The results must not
    depend on the layout's kernel beyond their bounds, and nothing outside the
    outputs' elements may be written."""
    B, S, Hq, Hkv, D = 2, 140, 4, 2, 64
    T = DTYPES[dt]
    t, do, kw = make(11, T, B, S, S, Hq, Hkv, D, causal=True, buckets=16)
    if layout == "expanded":
        t["k"] = t["k"][:, :, :1].expand(B, S, Hkv, D)
        t["v"] = t["v"][:1].expand(B, S, Hkv, D)
        run_and_check(dyt, t, do, kw)
        return

    def buffers(H):
        if layout == "heads_first":
            b = torch.full((B, H, S, D), 7.0, dtype=T, device="cuda")
            return b, b.transpose(1, 2)
        if layout == "offset_one":
            b = torch.full((B * S * H * D + 1,), 7.0, dtype=T, device="cuda")
            return b, b[1:].view(B, S, H, D)
        if layout == "odd_pitch":
            b = torch.full((B, S, H, D + 3), 7.0, dtype=T, device="cuda")
            return b, b[..., :D]
        raise AssertionError

    if layout == "fused":
        n = Hq + 2 * Hkv
        x = torch.full((B, S, n, D), 7.0, dtype=T, device="cuda")
        parts = lambda y: (y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:])
        q, k, v = (_copy_into(t[c], w) for c, w in zip("qkv", parts(x)))
        g = torch.full((B, S, n + 1, D), 7.0, dtype=T, device="cuda")
        outs = parts(g[:, :, :n])
        o = torch.empty(B, S, Hq + 1, D, dtype=T, device="cuda").fill_(7.0)[:, :, :Hq]
    else:
        q, k, v = (_copy_into(t[c], buffers(t[c].shape[2])[1]) for c in "qkv")
        o_all, o = buffers(Hq)
        outs_all = [buffers(h) for h in (Hq, Hkv, Hkv)]
        outs = [b for _, b in outs_all]
    stats = torch.empty(B, Hq, S, device="cuda")
    dyt.dyt_attn_forward(q, k, v, o=o, stats=stats, **kw)
    ref = Attention(q, k, v, **kw)
    ref.check_forward(o, stats)
    dq, dk, dv, dtab = dyt.dyt_attn_backward(q, k, v, o, do, stats, dq=outs[0], dk=outs[1], dv=outs[2], **kw)
    assert dq.data_ptr() == outs[0].data_ptr()
    ref.check_backward(do, dq, dk, dv, dtab)
    if layout == "fused":
        assert (g[:, :, n] == 7).all()
    elif layout == "odd_pitch":
        assert (o_all[..., D:] == 7).all() and all((b[..., D:] == 7).all() for b, _ in outs_all)
    elif layout == "offset_one":
        assert o_all[0] == 7 and all(b[0] == 7 for b, _ in outs_all)


@pytest.mark.parametrize("pitch", [1 << 19, 1 << 24], ids=["tile_in_31_bits", "tile_over_31_bits"])
def test_cache_offsets_past_32_bits(dyt, pitch):
    """A cache whose last keys lie over 2^32 elements from its first: rows of
    a wide buffer, with the 16-byte loads' range and past it."""
    S = (5 << 32) // 4 // pitch + 3   # the last row starts past 2^32 elements (10.7 GB of bf16)
    D, Hkv = 64, 2
    big = torch.empty((S - 1) * pitch + Hkv * 2 * D, dtype=torch.bfloat16, device="cuda")
    kv = big.as_strided((1, S, 2 * Hkv, D), (0, pitch, D, 1))
    t, do, kw = make(13, torch.bfloat16, 1, 40, S, 4, Hkv, D)
    kv[:, :, :Hkv] = t["k"]
    kv[:, :, Hkv:] = t["v"]
    t["k"], t["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
    run_and_check(dyt, t, do, kw)
    t1, do1, kw1 = make(14, torch.bfloat16, 1, 1, S, 4, Hkv, D)
    t1["k"], t1["v"] = t["k"], t["v"]
    run_and_check(dyt, t1, do1, kw1, backward=False)


@pytest.mark.parametrize("dt", DTYPES)
def test_single_tokens_over_a_ragged_cache(dyt, dt):
    lens = [1, 17, 4000, 2049, 64, 3999]
    for buckets in (0, 32):
        t, do, kw = make(15, DTYPES[dt], 6, 1, 4000, 8, 2, 128, lens=lens, starts=[n - 1 for n in lens],
                         causal=True, buckets=buckets, bidirectional=False)
        for b, n in enumerate(lens):
            t["k"][b, n:] = math.nan
            t["v"][b, n:] = math.nan
        run_and_check(dyt, t, do, kw)


# large enough for four waves to a workgroup and for the split of the keys
LARGE = [
    (dict(B=8, Sq=512, Sk=1024, Hq=16, Hkv=4, D=128), {}), (dict(B=8, Sq=700, Sk=700, Hq=8, Hkv=8, D=64), {}),
    (dict(B=16, Sq=257, Sk=513, Hq=8, Hkv=8, D=96), {}), (dict(B=2, Sq=1100, Sk=2200, Hq=16, Hkv=16, D=32), {}),
    (dict(B=8, Sq=600, Sk=700, Hq=12, Hkv=4, D=64), dict(buckets=32)),
    (dict(B=8, Sq=520, Sk=1040, Hq=16, Hkv=16, D=128), dict(buckets=64, distance=256)),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", LARGE, ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_large(dyt, dt, case, causal):
    """One batch entry of the first, a middle and the last against the
    formula; dtable, a sum over all of them, by linearity: the upstream
    gradient is zero elsewhere."""
    size, more = case
    B = size["B"]
    lens = [size["Sk"] - 3 * b for b in range(B)]
    t, do, kw = make(17, DTYPES[dt], **size, causal=causal, lens=lens, **more)
    b = B - 1
    only = torch.zeros_like(do)
    only[b] = do[b]
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, only, stats, **kw)
    one = {n: x[b:b + 1] for n, x in t.items()}
    kw1 = dict(kw, seqlens_k=kw["seqlens_k"][b:])
    ref = Attention(**one, **kw1)
    ref.check_forward(o[b:], stats[b:])
    ref.check_backward(do[b:], *(g[b:] for g in grads[:3]), *grads[3:])
    for g in grads[:3]:
        assert (g[:b] == 0).all()


@pytest.mark.parametrize("size", [(8, 300, 1030, 16, 16, 128), (2, 40, 1200, 2, 2, 128), (1, 90, 2300, 3, 3, 64)], ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_the_widest_table(dyt, dt, size):
    """Every bucket and the longest reach: the most LDS each kernel takes."""
    t, do, kw = make(18, DTYPES[dt], *size, buckets=128, distance=1024, causal=False)
    b = size[0] - 1
    only = torch.zeros_like(do)
    only[b] = do[b]
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, only, stats, **kw)
    ref = Attention(*(t[n][b:] for n in "qkv"), **kw)
    ref.check_forward(o[b:], stats[b:])
    ref.check_backward(do[b:], *(g[b:] for g in grads[:3]), *grads[3:])


@pytest.mark.parametrize("buckets", [0, 16])
def test_gradients_against_differences(dyt, buckets):
    """f = sum(w o): its change along a direction, from the float32 forward."""
    t, do, kw = make(19, torch.float32, 2, 60, 90, 4, 2, 32, causal=True, buckets=buckets)
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    names = ["q", "k", "v"] + (["table"] if buckets else [])
    g = torch.Generator().manual_seed(23)
    for i, name in enumerate(names):
        x = kw["table"] if name == "table" else t[name]
        w = torch.randn(x.shape, generator=g).cuda()
        w /= w.norm()
        eps = 0.25

        def f(step):
            y = x + step * w
            args = dict(t, **({} if name == "table" else {name: y}))
            opts = dict(kw, **({"table": y} if name == "table" else {}))
            return (d(do) * d(dyt.dyt_attn_forward(args["q"], args["k"], args["v"], **opts)[0])).sum().item()

        # two central differences, extrapolated: error of order eps^4
        d1, d2 = (f(eps) - f(-eps)) / (2 * eps), (f(eps / 2) - f(-eps / 2)) / eps
        want = (d(grads[i]) * d(w)).sum().item()
        # each f sums do.o with errors of about 2^-20 |do||o| at random signs
        noise = 8 * 2.0 ** -20 * (d(do).norm() * d(o).abs().max()).item() / eps
        assert abs((4 * d2 - d1) / 3 - want) <= noise + abs(d2 - d1) / 3 + 1e-4 * abs(want), (name, d1, d2, want)


def test_same_bits_every_time(dyt):
    for dt, buckets in ((torch.bfloat16, 32), (torch.float32, 0), (torch.float16, 0)):
        t, do, kw = make(29, dt, 4, 300, 600, 8, 2, 64, causal=True, buckets=buckets)
        first = None
        for _ in range(3):
            o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
            r = (o, stats, *dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw))
            if first is None:
                first = r
            assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_captured_in_a_graph(dyt):
    t, do, kw = make(31, torch.bfloat16, 2, 200, 400, 8, 2, 64, causal=True, buckets=16)

    def step():
        o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
        return (o, stats, *dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        t["q"].copy_(torch.randn(t["q"].shape, generator=torch.Generator().manual_seed(i)).cuda())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_on_another_stream(dyt):
    t, do, kw = make(37, torch.float16, 2, 150, 300, 4, 4, 64)
    want = run_and_check(dyt, t, do, kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], stream=s, **kw)
    got = (o, stats, *dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, stream=s, **kw))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_random_problems(dyt):
    """Forty problems over the whole range of sizes and options."""
    import random
    rng = random.Random(4)
    for i in range(40):
        D = rng.randint(1, 128)
        Hkv = rng.choice([1, 1, 2, 3])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 6])
        Sq, Sk = (int(math.exp(rng.uniform(0, math.log(600)))) for _ in range(2))
        B = rng.randint(1, 4)
        causal = rng.random() < 0.5
        lens = [rng.randint(0, Sk + 5) for _ in range(B)] if rng.random() < 0.4 else None
        starts = [rng.randint(-Sq, Sk + 5) for _ in range(B)] if rng.random() < 0.4 else None
        more = {}
        if rng.random() < 0.5:
            bidi = rng.random() < 0.5
            buckets = rng.choice([4, 10, 32, 64])
            more = dict(buckets=buckets, bidirectional=bidi, distance=rng.randint(buckets // 2 + 1, 300),
                        table_dt=rng.choice(list(DTYPES.values())))
        dt = rng.choice(list(DTYPES))
        print(i, dt, (B, Sq, Sk, Hq, Hkv, D), causal, lens, starts, more, flush=True)
        t, do, kw = make(i, DTYPES[dt], B, Sq, Sk, Hq, Hkv, D, causal=causal, lens=lens, starts=starts, **more)
        run_and_check(dyt, t, do, kw)
