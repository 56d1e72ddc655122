"""Embedding lookup and its gradient on the GPU against float64
(tests/lm_ref.py)."""
import math

import pytest
import torch

from block_ref import d
from lm_ref import check_embed_backward, check_embed_forward

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


def make(seed, T, V, D, wdt, ydt, spread=None, ignored=0.1, token=torch.int64):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(V, D, generator=g).to(wdt).cuda()
    dy = torch.randn(T, D, generator=g).to(ydt).cuda()
    t = torch.randint(0, spread or max(V, 1), (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = -1
    return w, t.to(token).cuda(), dy


def run(dyt, w, t, dy, scale, ydt, gdt):
    y = dyt.dyt_embed_forward(w, t, scale, dtype=ydt)
    check_embed_forward(w, t, scale, y)
    dw = dyt.dyt_embed_backward(dy, t, w.shape[0], scale, dtype=gdt)
    check_embed_backward(dy, t, w.shape[0], scale, dw)
    before = torch.randn(dw.shape, device="cuda").to(gdt)
    after = before.clone()
    assert dyt.dyt_embed_backward(dy, t, w.shape[0], scale, dweight=after, accumulate=True) is after
    check_embed_backward(dy, t, w.shape[0], scale, after, before=before)
    absent = torch.ones(w.shape[0], dtype=torch.bool)
    absent[t.cpu()[(t >= 0).cpu() & (t < w.shape[0]).cpu()].long()] = False
    assert torch.equal(after[absent.cuda()], before[absent.cuda()])
    return y, dw


@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 9, 16, 33, 100, 128, 255, 1000, 2048, 2049, 4104])
@pytest.mark.parametrize("wdt,ydt,gdt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "f32"),
                                         ("f16", "f32", "f16"), ("bf16", "f16", "f32"), ("f16", "f16", "bf16")])
def test_widths(dyt, D, wdt, ydt, gdt):
    for T, V in ((1, 1), (1, 5), (70, 9), (300, 1000)):
        w, t, dy = make(D + T, T, V, D, DTYPES[wdt], DTYPES[ydt])
        run(dyt, w, t, dy, math.sqrt(D), DTYPES[ydt], DTYPES[gdt])


# one token for all, runs that pass many chunks, none at all; several passes of
# the sort (V up to and past 2^9, 2^18), one and many workgroups
@pytest.mark.parametrize("T,V,D,spread", [(5000, 40, 64, 1), (5000, 511, 64, 511), (5000, 512, 24, 512), (4096, 513, 64, 3),
                                          (65536, 300000, 16, 300000), (65537, 300000, 16, 300000), (65537, 50, 8, 2),
                                          (200001, 262143, 8, 262143), (200001, 262144, 16, 7), (100000, 1000, 40, 1),
                                          (20000, 70, 2056, 70), (3, 600000, 8, 600000)])
@pytest.mark.parametrize("token", [torch.int32, torch.int64])
def test_runs(dyt, T, V, D, spread, token):
    w, t, dy = make(T, T, V, D, torch.float32, torch.float32, spread, token=token)
    run(dyt, w, t, dy, 1.0, torch.float32, torch.float32)


# around the border of one launch (2,048 tokens): even, and with one token for most places
@pytest.mark.parametrize("T,V,D,spread", [(2048, 700, 24, 700), (2049, 700, 24, 700), (2048, 1, 130, 1), (2049, 1, 130, 1),
                                          (2047, 65536, 8, 65536), (2048, 65537, 8, 65537), (2048, 3, 257, 2), (1, 65536, 9, 9),
                                          (2048, 3000, 129, 40), (1000, 4099, 300, 4099), (9, 100, 1, 1), (8, 1, 1, 1),
                                          (2048, 8191, 2048, 8191), (2048, 8193, 2048, 8193)])
@pytest.mark.parametrize("dt", DTYPES)
def test_around_the_border_of_one_launch(dyt, T, V, D, spread, dt):
    w, t, dy = make(T + V, T, V, D, DTYPES[dt], DTYPES[dt], spread, token=torch.int32)
    g = torch.Generator().manual_seed(T)
    t[(torch.rand(T, generator=g) < 0.4).cuda()] = V // 2   # as often as all others together
    _, dw = run(dyt, w, t, dy, -0.5, DTYPES[dt], DTYPES[dt])
    assert torch.equal(dw, dyt.dyt_embed_backward(dy, t, V, -0.5, dtype=DTYPES[dt]))


@pytest.mark.parametrize("D", [(1 << 20) - 1, (1 << 20) + 8, 1 << 23])
def test_wide_rows(dyt, D):
    w, t, dy = make(5, 5, 2, D, torch.bfloat16, torch.bfloat16)
    run(dyt, w, t, dy, 1.0, torch.bfloat16, torch.bfloat16)


@pytest.mark.parametrize("D", [1, 3, 8, 33, 128, 255, 1000])
@pytest.mark.parametrize("wdt,ydt,gdt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "f32"),
                                         ("f16", "f32", "f16"), ("bf16", "f16", "f32"), ("f16", "f16", "bf16")])
def test_widths_of_many_tokens(dyt, D, wdt, ydt, gdt):
    w, t, dy = make(D, 2100, 600, D, DTYPES[wdt], DTYPES[ydt])
    t[:500] = 17
    run(dyt, w, t, dy, math.sqrt(D), DTYPES[ydt], DTYPES[gdt])
    pitch = D + 3
    buf = torch.full((600 * pitch + 1,), math.nan, dtype=DTYPES[gdt], device="cuda")
    dys = torch.full((2100 * pitch + 1,), math.nan, dtype=DTYPES[ydt], device="cuda").as_strided((2100, D), (pitch, 1), 1)
    dys.copy_(dy)
    dys[t < 0] = math.nan
    dws = buf.as_strided((600, D), (pitch, 1), 1)
    dyt.dyt_embed_backward(dys, t, 600, 1.5, dweight=dws)
    check_embed_backward(dy, t, 600, 1.5, dws)
    assert int(torch.isnan(buf).sum()) == buf.numel() - 600 * D


def test_tokens_outside(dyt):
    w, t, dy = make(1, 200, 50, 24, torch.float32, torch.float32, ignored=0.0)
    t[::7] = torch.tensor([-1, 50, 51, -(1 << 40), 1 << 40, (1 << 32) + 3, -100]).cuda().repeat(29)[:len(t[::7])]
    run(dyt, w, t, dy, 2.0, torch.float32, torch.float32)
    t.fill_(-1)
    y, dw = run(dyt, w, t, dy, 2.0, torch.float32, torch.float32)
    assert (y == 0).all() and (dw == 0).all()
    # a place that is ignored may hold anything
    dy.fill_(math.nan)
    assert (dyt.dyt_embed_backward(dy, t, 50) == 0).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("D,pitch,at", [(64, 72, 0), (64, 67, 3), (101, 103, 1), (2050, 2051, 1), (1, 9, 2)])
def test_row_strides(dyt, dt, D, pitch, at):
    T, V, X = 83, 37, DTYPES[dt]
    w, t, dy = make(7, T, V, D, X, X)
    bufs = [torch.full((n * pitch + at,), math.nan, dtype=X, device="cuda") for n in (V, T, T, V)]
    ws, dys, ys, dws = (b.as_strided((n, D), (pitch, 1), at) for b, n in zip(bufs, (V, T, T, V)))
    ws.copy_(w)
    dys.copy_(dy)
    dyt.dyt_embed_forward(ws, t, 1.5, y=ys)
    check_embed_forward(w, t, 1.5, ys)
    dyt.dyt_embed_backward(dys, t, V, 1.5, dweight=dws)
    check_embed_backward(dy, t, V, 1.5, dws)
    for b, n in zip(bufs[2:], (T, V)):
        assert int(torch.isnan(b).sum()) == b.numel() - n * D


def test_more_rows_than_workgroups(dyt):
    """Zero rows of a launch that walks them (2^20 workgroups of 64 rows)."""
    V = (1 << 26) + 200
    t = torch.tensor([3, V - 1, 1 << 26, 3, (1 << 26) - 1], device="cuda")
    dy = torch.arange(1, 6, device="cuda", dtype=torch.float32).view(5, 1).expand(5, 2).contiguous()
    dw = torch.full((V, 2), 9.0, device="cuda")
    dyt.dyt_embed_backward(dy, t, V, dweight=dw)
    assert [dw[i].tolist() for i in (3, V - 1, 1 << 26, (1 << 26) - 1)] == [[5, 5], [2, 2], [3, 3], [5, 5]]
    assert int((dw != 0).sum()) == 8


def test_nothing_there(dyt):
    w, t, dy = make(1, 0, 30, 16, torch.bfloat16, torch.bfloat16)
    assert dyt.dyt_embed_forward(w, t).shape == (0, 16)
    dw = torch.full((30, 16), 3.0, device="cuda")
    dyt.dyt_embed_backward(dy, t, 30, dweight=dw)
    assert (dw == 0).all()
    dw.fill_(3.0)
    dyt.dyt_embed_backward(dy, t, 30, dweight=dw, accumulate=True)
    assert (dw == 3).all()
    w, t, dy = make(1, 5, 0, 16, torch.float32, torch.float32, ignored=1.0)
    assert (dyt.dyt_embed_forward(w, t) == 0).all()
    assert dyt.dyt_embed_backward(dy, t, 0).shape == (0, 16)
    w, t, dy = make(1, 5, 7, 0, torch.float32, torch.float32)
    assert dyt.dyt_embed_forward(w, t).shape == (5, 0) and dyt.dyt_embed_backward(dy, t, 7).shape == (7, 0)


def test_gradient_against_differences(dyt):
    w, t, dy = make(3, 60, 11, 24, torch.float32, torch.float32)
    dw = dyt.dyt_embed_backward(dy, t, 11, 3.0)
    v = torch.randn(w.shape, generator=torch.Generator().manual_seed(5)).cuda()

    def f(step):
        return (d(dy) * d(dyt.dyt_embed_forward(w + step * v, t, 3.0))).sum().item()

    # linear in the weight: a difference is exact but for the roundings of w + v and y
    got, want = (f(0.5) - f(-0.5)), (d(dw) * d(v)).sum().item()
    noise = 6 * 2.0 ** -24 * (d(dy).abs().sum() * (3 * d(w).abs().max() + 3 * d(v).abs().max())).item()
    assert abs(got - want) <= noise


def test_same_bits_every_time_and_in_a_graph(dyt):
    w, t, dy = make(19, 9000, 700, 200, torch.bfloat16, torch.bfloat16)
    big = make(20, 70000, 700, 16, torch.bfloat16, torch.bfloat16)

    def step():
        return (dyt.dyt_embed_forward(w, t, 2.0), dyt.dyt_embed_backward(dy, t, 700, 2.0),
                dyt.dyt_embed_backward(big[2], big[1], 700, dtype=torch.float32))

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        t.copy_(torch.randint(-1, 700, t.shape, generator=torch.Generator().manual_seed(i)).cuda())
        big[1].copy_(torch.randint(-1, 700, big[1].shape, generator=torch.Generator().manual_seed(i)).cuda())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_on_another_stream(dyt):
    w, t, dy = make(23, 700, 60, 100, torch.float16, torch.float16)
    want = run(dyt, w, t, dy, 1.0, torch.float16, torch.float16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (dyt.dyt_embed_forward(w, t, stream=s), dyt.dyt_embed_backward(dy, t, 60, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits(dyt):
    """A table of over 2^32 elements, and as many of dy."""
    V, D = (1 << 32) // 2048 + 300, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(V, D, generator=g, device="cuda", dtype=torch.bfloat16)
    t = torch.cat([torch.arange(40), torch.arange(V - 40, V), torch.randint(0, V, (400,))]).cuda()
    y = dyt.dyt_embed_forward(w, t, 2.0)
    assert torch.equal(y, w[t] * 2)
    dw = dyt.dyt_embed_backward(y, t, V, 1.0, dweight=w)
    rows = torch.unique(t)
    want = torch.zeros(rows.numel(), D, device="cuda", dtype=torch.float64)
    want.index_add_(0, torch.searchsorted(rows, t), y.double())
    assert ((dw[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() + 400 * 2.0 ** -24 * 400).all()
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[rows] = False
    at = rest.nonzero().squeeze(1)
    assert all((dw[part] == 0).all() for part in at.split(100000))
    del w, dw
    T = V
    t = torch.randint(0, 64, (T,), device="cuda", generator=g)
    dy = torch.ones(T, D, device="cuda", dtype=torch.bfloat16)
    dw = dyt.dyt_embed_backward(dy, t, 64, dtype=torch.float32)
    assert torch.equal(dw[:, ::97], torch.bincount(t, minlength=64).float().view(-1, 1).expand(-1, -(-D // 97)))
