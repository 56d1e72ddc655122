"""Attention's gradients where a masked place could leak into a sum: padding
rows of the last tile under a large bias, keys that the causal mask hides
from every row, and rows that see no key, against the formulas in float64
(tests/block_ref.py) and against the same problem with whole tiles."""
import math
import random

import pytest
import torch

from block_ref import Attention
from test_gpu_block_attn import DTYPES, LARGE, dyt, make, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu

# row tiles of 32 and 64 that end before the tile does, one wave and four to
# a workgroup, slices, splits, each padded head dimension
SIZES = [(2, 33, 70, 2, 1, 32), (1, 70, 40, 2, 2, 64), (1, 96, 96, 1, 1, 24), (2, 129, 129, 2, 2, 80),
         (1, 700, 40, 1, 1, 64), (16, 160, 130, 16, 16, 64), (16, 100, 130, 16, 16, 128), (1, 37, 50, 2, 1, 33)]


def table_problem(dt, causal, size, shift, every):
    t, do, kw = make(41, DTYPES[dt], *size, buckets=16, distance=40, causal=causal, bidirectional=not causal,
                     table_dt=torch.float32)
    kw["table"][::every] += shift
    return t, do, kw


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("entry", [12.0, 30.0])
def test_entries_whose_exponential_passes_float16(dyt, entry, causal, size):  # noqa: F811
    """exp(11.09) is float16's largest value."""
    run_and_check(dyt, *table_problem("f16", causal, size, entry, 3))


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt,shift", [("f16", 30.0), ("bf16", 100.0), ("f32", 100.0)])
def test_an_offset_of_the_whole_table(dyt, dt, shift, causal, size):  # noqa: F811
    """The softmax takes it out again; exp(88.72) is float32's largest value."""
    run_and_check(dyt, *table_problem(dt, causal, size, shift, 1))


@pytest.mark.parametrize("size", [s for s in SIZES if s[1] % 32], ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt,entry", [("f16", 12.0), ("f16", 30.0), ("bf16", 90.0), ("f32", 100.0)])
def test_rows_of_zero_gradient_change_no_bit(dyt, dt, entry, causal, size):  # noqa: F811
    """The rows that complete a block of 32 (so every launch stays the same)
    have do = 0: they add exact zeros."""
    B, Sq, Sk, Hq, Hkv, D = size
    full = (B, (Sq + 31) // 32 * 32, Sk, Hq, Hkv, D)
    t, do, kw = table_problem(dt, causal, full, entry, 3)
    kw["q_start"] = torch.full((B,), Sk - Sq, dtype=torch.int32, device="cuda")
    do[:, Sq:] = 0
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    want = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    q, o, do = (x[:, :Sq].contiguous() for x in (t["q"], o, do))
    got = dyt.dyt_attn_backward(q, t["k"], t["v"], o, do, stats[:, :, :Sq].contiguous(), **kw)
    for name, a, b in zip(("dq", "dk", "dv", "dtable"), got, (want[0][:, :Sq], *want[1:])):
        assert torch.isfinite(a).all() and torch.equal(a, b), name


# where start + Sq falls inside a block of 32 keys below the length: q_start,
# size, lengths (None: all keys)
HIDDEN = [([10], (1, 70, 150, 2, 1, 64), None), ([0, 3, 40], (3, 64, 200, 4, 2, 72), [200, 90, 130]),
          ([5, -20], (2, 33, 100, 6, 2, 32), None), ([100, 7], (2, 32, 1200, 1, 1, 128), [1200, 50]),
          ([17] * 16, (16, 160, 300, 16, 16, 64), None), ([9] * 8, (8, 130, 260, 32, 8, 128), None),
          ([1], (1, 1, 40, 8, 1, 64), None), ([2], (1, 40, 77, 3, 1, 33), None)]


@pytest.mark.parametrize("buckets", [0, 16])
@pytest.mark.parametrize("case", HIDDEN, ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_keys_past_the_last_causal_position(dyt, dt, case, buckets):  # noqa: F811
    """A cache's tail that no row sees yet: its memory may hold anything, and
    its gradients are zeros."""
    starts, size, lens = case
    B, Sq, Sk = size[:3]
    t, do, kw = make(43, DTYPES[dt], *size, starts=starts, lens=lens, causal=True, buckets=buckets, bidirectional=False)
    ends = [max(0, min(n, s + Sq)) for s, n in zip(starts, lens or [Sk] * B)]
    for b, end in enumerate(ends):
        t["k"][b, end:] = math.inf if b % 3 == 1 else math.nan
        t["v"][b, end:] = math.inf if b % 2 else math.nan
    _, _, _, dk, dv, *_ = run_and_check(dyt, t, do, kw)
    for b, end in enumerate(ends):
        assert (dk[b, end:] == 0).all() and (dv[b, end:] == 0).all()


@pytest.mark.parametrize("buckets", [0, 16])
@pytest.mark.parametrize("size", [(3, 70, 90, 4, 2, 64), (2, 130, 200, 6, 2, 40), (16, 160, 300, 16, 16, 128),
                                  (2, 40, 900, 2, 2, 33), (8, 300, 256, 16, 4, 64)], ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_rows_before_the_first_key(dyt, dt, size, buckets):  # noqa: F811
    """Left-padded sequences: rows at negative positions see no key under the
    causal mask, and neither their q nor their do may reach a gradient."""
    B, Sq = size[:2]
    starts = [-((7 + 13 * b) % (Sq + 5)) for b in range(B)]
    t, do, kw = make(47, DTYPES[dt], *size, starts=starts, causal=True, buckets=buckets, bidirectional=False)
    clean, do_clean = t["q"].clone(), do.clone()
    for b, s in enumerate(starts):
        clean[b, :-s] = 0
        do_clean[b, :-s] = 0
        t["q"][b, :-s] = math.nan if b % 2 else math.inf
        do[b, :-s] = math.inf if b % 3 else math.nan
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    ref = Attention(clean, t["k"], t["v"], **kw)
    ref.check_forward(o, stats)
    ref.check_backward(do_clean, *grads)
    for b, s in enumerate(starts):
        assert (o[b, :-s] == 0).all() and (grads[0][b, :-s] == 0).all()


def test_layer_norm_of_a_row_of_2_to_the_27(dyt):  # noqa: F811
    """The parameters' gradients of more columns than one launch has threads
    for: the second pass walks. One row, so dbeta is dy and dgamma is one
    product."""
    N = (1 << 27) + 3
    g = torch.Generator(device="cuda").manual_seed(53)
    x, dy = (torch.randn(1, N, device="cuda", generator=g, dtype=torch.float16) for _ in range(2))
    gamma = torch.ones(N, device="cuda", dtype=torch.float16)
    y, mean, rstd = dyt.dyt_ln_forward(x, gamma, torch.zeros_like(gamma))
    dx, dgamma, dbeta = dyt.dyt_ln_backward(x, dy, mean, rstd, gamma)
    assert torch.equal(dbeta, dy[0])
    n = (x[0].double() - mean.double()) * rstd.double()
    want = n * dy[0].double()
    # n is rounded twice and the product once in float32, the result to float16
    bound = want.abs() * (2.0 ** -11 + 4 * 2.0 ** -24) + 2.0 ** -24
    assert ((dgamma.double() - want).abs() <= bound).all()
    assert torch.isfinite(dx).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("size", [(1, 200, 300, 4, 2, 64), (2, 1, 3000, 4, 2, 128), (1, 257, 130, 2, 2, 72),
                                  (8, 160, 300, 16, 16, 64)], ids=str)
def test_head_strides_of_long_caches(dyt, size):  # noqa: F811
    """[B, H, S, D] tensors whose heads lie 2^25 bytes and more apart (131,072
    positions of D = 128) take the same kernels as contiguous ones: equal bits."""
    B, Sq, Sk, Hq, Hkv, D = size
    t, do, kw = make(59, torch.bfloat16, *size, causal=True)
    apart = (1 << 24) + 64

    def far(x):
        S, H = x.shape[1:3]
        y = torch.zeros((B * H - 1) * apart + S * D, dtype=x.dtype, device="cuda").as_strided(x.shape, (H * apart, D, apart, 1))
        return y.copy_(x)

    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    want = (o, stats, *dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw))
    q, k, v = (far(t[n]) for n in "qkv")
    o2 = far(torch.zeros_like(o))
    o2, stats = dyt.dyt_attn_forward(q, k, v, o=o2, **kw)
    outs = {n: far(torch.zeros_like(x)) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    got = (o2, stats, *dyt.dyt_attn_backward(q, k, v, o2, far(do), stats, **outs, **kw))
    for name, a, b in zip(("o", "stats", "dq", "dk", "dv"), got, want):
        assert torch.equal(a, b), name


def test_a_captured_append_replayed_past_the_end(dyt):  # noqa: F811
    """A decoding step as a graph: each replay is the next token, checked
    against the whole sequence; past the end it changes nothing, and an eager
    append sees that the cache is full."""
    torch.manual_seed(61)
    B, prompt, room = 2, 5, 11
    m = dyt.Attention(64, 4, 2, num_buckets=16, max_distance=40, device="cuda")
    torch.nn.init.normal_(m.table)
    x = torch.randn(B, room, 64, device="cuda")
    token = x[:, prompt:prompt + 1].clone()
    with torch.no_grad():
        want = m(x)
        warm = dyt.KVCache(B, room, 2, 16, torch.float32)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                m(token, cache=warm)
        torch.cuda.current_stream().wait_stream(side)
        cache = dyt.KVCache(B, room, 2, 16, torch.float32)
        m(x[:, :prompt], cache=cache)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = m(token, cache=cache)
        for i in range(prompt, room):
            token.copy_(x[:, i:i + 1])
            graph.replay()
            torch.cuda.synchronize()
            # the same 64 and room terms of order one in other orders
            assert (out - want[:, i:i + 1]).abs().max() <= 200 * 2.0 ** -24 * 4, i
            assert cache.length.tolist() == [i + 1] * B
            m(token, cache=dyt.KVCache(B, 1, 2, 16, torch.float32))   # eager work in between
        k, v = cache.k.clone(), cache.v.clone()
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(cache.k, k) and torch.equal(cache.v, v) and cache.length.tolist() == [room] * B
        with pytest.raises(ValueError, match="no room"):
            m(token, cache=cache)


def test_gradients_through_a_cache(dyt):  # noqa: F811
    """A prompt's gradients are those without a cache; the next token's call
    takes the prompt's keys and values as they are, and holds no graph of it."""
    torch.manual_seed(67)
    m = dyt.Attention(64, 4, 2, num_buckets=16, max_distance=40, device="cuda")
    torch.nn.init.normal_(m.table)
    x = torch.randn(2, 40, 64, device="cuda")
    w = torch.randn(2, 40, 64, device="cuda")

    def gradients(out, w):
        m.zero_grad()
        (out * w).sum().backward()
        return [p.grad.clone() for p in m.parameters()]

    want = gradients(m(x), w)
    cache = dyt.KVCache(2, 42, 2, 16, torch.float32)
    got = gradients(m(x, cache=cache), w)
    for a, b in zip(got, want):
        # sums of 80 rows' and 64 columns' float32 terms, a few operators deep
        assert (a - b).norm() <= 500 * 2.0 ** -24 * b.norm()
    for _ in range(2):
        before = cache.k.clone(), cache.v.clone()
        assert not cache.k.requires_grad and not cache.v.requires_grad
        token = torch.randn(2, 1, 64, device="cuda")
        out = m(token, cache=cache)
        got = gradients(out, w[:, :1])
        # the same in float64: the keys before are constants
        n = int(cache.length[0])
        p = [t.detach().double().requires_grad_() for t in (m.table, m.qkv.weight, m.out.weight)]
        q, k, v = (token.double() @ p[1].t()).view(2, 1, 8, 16).split([4, 2, 2], 2)
        k, v = (torch.cat([b[:, :n - 1].double(), t], 1).repeat_interleave(2, 2) for b, t in zip(before, (k, v)))
        far = torch.arange(n - 1, -1, -1, device="cuda")
        bucket = torch.searchsorted(torch.tensor(dyt.dyt_attn_bucket_borders(16, 40, False), device="cuda"), far, right=True) - 1
        s = (q * k).sum(-1) / 4 + p[0][bucket]
        o = (torch.softmax(s, 1).unsqueeze(-1) * v).sum(1, keepdim=True).reshape(2, 1, 64) @ p[2].t()
        (o * w[:, :1].double()).sum().backward()
        names = [x for x, _ in m.named_parameters()]
        for a, b in ((got[names.index("table")], p[0].grad), (got[names.index("qkv.weight")], p[1].grad),
                     (got[names.index("out.weight")], p[2].grad)):
            assert (a - b).norm() <= 500 * 2.0 ** -24 * b.norm()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", LARGE, ids=str)
@pytest.mark.parametrize("dt", DTYPES)
def test_batch_entries_of_the_large_sizes(dyt, dt, case, causal):  # noqa: F811
    """The first and a middle batch entry of the sizes with four waves to a
    workgroup (the last is test_large's): their outputs from the one forward,
    their gradients with the others' upstream gradient zero."""
    size, more = case
    B = size["B"]
    t, do, kw = make(71, DTYPES[dt], **size, causal=causal, lens=[size["Sk"] - 3 * b for b in range(B)], **more)
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    for b in (0, B // 2):
        only = torch.zeros_like(do)
        only[b] = do[b]
        grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, only, stats, **kw)
        one = slice(b, b + 1)
        ref = Attention(*(t[n][one] for n in "qkv"), **dict(kw, seqlens_k=kw["seqlens_k"][one]))
        ref.check_forward(o[one], stats[one])
        ref.check_backward(do[one], *(g[one] for g in grads[:3]), *grads[3:])
        others = [i for i in range(B) if i != b]
        assert all((g[others] == 0).all() for g in grads[:3])


def test_random_problems_whose_unseen_places_are_nan(dyt):  # noqa: F811
    """Forty problems with lengths, positions and the causal mask drawn, and
    everything that no pair reaches filled with NaN: keys that no row sees,
    rows at negative positions, and all of a batch entry without keys."""
    rng = random.Random(73)
    for i in range(40):
        D = rng.randint(1, 128)
        Hkv = rng.choice([1, 1, 2, 3])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 6])
        Sq, Sk = (int(math.exp(rng.uniform(0, math.log(600)))) for _ in range(2))
        B = rng.randint(1, 4)
        causal = rng.random() < 0.7
        lens = [rng.randint(0, Sk + 5) for _ in range(B)]
        starts = [rng.randint(-Sq, max(0, Sk - Sq // 2)) for _ in range(B)]
        more = {}
        if rng.random() < 0.5:
            bidi = rng.random() < 0.5
            buckets = rng.choice([4, 10, 32, 64])
            more = dict(buckets=buckets, bidirectional=bidi, distance=rng.randint(buckets // 2 + 1, 300))
        dt = rng.choice(list(DTYPES))
        print(i, dt, (B, Sq, Sk, Hq, Hkv, D), causal, lens, starts, more, flush=True)
        t, do, kw = make(i, DTYPES[dt], B, Sq, Sk, Hq, Hkv, D, causal=causal, lens=lens, starts=starts, **more)
        q, clean_do = t["q"].clone(), do.clone()
        for b in range(B):
            end = max(0, min(lens[b], Sk, starts[b] + Sq if causal else Sk))
            t["k"][b, end:] = t["v"][b, end:] = math.nan
            blind = Sq if end == 0 else max(0, -starts[b]) if causal else 0
            q[b, :blind] = clean_do[b, :blind] = 0
            t["q"][b, :blind] = do[b, :blind] = math.nan
        o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
        grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
        ref = Attention(q, t["k"], t["v"], **kw)
        ref.check_forward(o, stats)
        ref.check_backward(clean_do, *grads)


@pytest.mark.parametrize("size", [(3, 160, 160, 2, 2, 64), (3, 90, 200, 4, 2, 40)], ids=str)
@pytest.mark.parametrize("hide", [-1e4, -1e8, -1e9, -3e38, -math.inf])
@pytest.mark.parametrize("dt", DTYPES)
def test_rows_that_see_hidden_buckets_only(dyt, dt, hide, size):  # noqa: F811
    """A window made by hiding the farthest buckets, over a padded batch: rows
    of the padding see only hidden keys. Their log sums are too large for a
    float32 probability to mean anything; with an upstream gradient of zero
    they must add nothing all the same."""
    B, S, Sk = size[:3]
    lens = [[Sk, 40, 7][b % 3] for b in range(B)]
    t, do, kw = make(79, DTYPES[dt], *size, buckets=16, distance=30, lens=lens, starts=[0] * B, table_dt=torch.float32)
    for b, n in enumerate(lens):
        do[b, n:] = 0
    kw["table"][7] = kw["table"][15] = hide
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    grads = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    kw["table"] = kw["table"].clamp(min=-1e4)   # exp(-1e4) = 0 as well
    ref = Attention(t["q"], t["k"], t["v"], **kw)
    # the rows before the padding, which see an ordinary key each: what their
    # hidden pairs' size adds to rho is no error of theirs
    ref.rho = ref.rho.clamp(max=1e-4)
    for b, n in enumerate(lens):
        n = min(n, S)
        err = (o[b, :n].double().cpu().transpose(0, 1) - ref.o[b, :, :n]).abs()
        half = {"f32": 0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
        pv = ref.p[b, :, :n] @ ref.v[b].abs()
        assert (err <= 1.05 * (2 * half + 1e-4) * pv + 2.0 ** -24).all()
        ref.p[b, :, n:] = 0
        ref.o[b, :, n:] = 0
    for x in grads:
        assert torch.isfinite(x).all()
    ref.check_backward(do, *grads)


def test_prompts_of_unequal_lengths_in_a_cache(dyt):  # noqa: F811
    """Appended padded, then the lengths set: the next tokens see each
    sequence as if it stood alone, whatever the padding held."""
    torch.manual_seed(83)
    m = dyt.Attention(64, 4, 2, num_buckets=16, max_distance=40, device="cuda")
    torch.nn.init.normal_(m.table)
    lens = [9, 3, 6]
    x = torch.randn(3, 13, 64, device="cuda")
    padded = torch.full((3, 9, 64), 1e3, device="cuda")
    for b, n in enumerate(lens):
        padded[b, :n] = x[b, :n]
    with torch.no_grad():
        cache = dyt.KVCache(3, 13, 2, 16, torch.float32)
        m(padded, cache=cache)
        cache.length.copy_(torch.tensor(lens))
        for i in range(4):
            got = m(torch.stack([x[b, n + i:n + i + 1] for b, n in enumerate(lens)]), cache=cache)
            for b, n in enumerate(lens):
                want = m(x[b:b + 1, :n + i + 1])[:, -1]
                # both sides sum the same 64 and 13 terms of order one in other orders
                assert (got[b] - want).abs().max() <= 200 * 2.0 ** -24 * 4, (b, i)
    assert cache.length.tolist() == [n + 4 for n in lens]
