"""Root-mean-square norm on the GPU against the formulas in float64
(tests/lm_ref.py: every tolerance is derived there from the roundings)."""
import math

import pytest
import torch

from block_ref import d
from lm_ref import check_rms_backward, check_rms_forward, check_rms_q8

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


def make(seed, M, N, dt, pdt, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (r(M, N) * 1.5 + shift).to(dt).cuda()
    return x, (r(N) * 0.1 + 1).to(pdt).cuda(), r(M, N).to(dt).cuda(), r(M, N).to(dt).cuda()


def run_plain(dyt, x, gm, dy, eps=EPS, **kw):
    y, rstd = dyt.dyt_rms_forward(x, gm, eps)
    check_rms_forward(x, gm, eps, y, rstd)
    dx, dg = dyt.dyt_rms_backward(x, dy, rstd, gm, **kw)
    check_rms_backward(x, dy, rstd, gm, dx, dg)
    return y, rstd, dx, dg


# around every border of the kernels' shapes, and rows that are no whole vectors
WIDTHS = [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 127, 128, 255, 256, 257, 500, 512, 513, 1000, 1024, 1025,
          2047, 2048, 2049, 4096, 4100, 8191, 8192, 8193, 16384, 16385, 20011, 32768, 32769, 65536, 65537, 70001]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dt,pdt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
def test_widths(dyt, dt, pdt, N):
    for M in (1, 5, 300) if N <= 4100 else (1, 21):
        x, gm, dy, r = make(N, M, N, DTYPES[dt], DTYPES[pdt])
        run_plain(dyt, x, gm, dy)
        h, y, rstd = dyt.dyt_rms_forward_residual(x, r, gm, EPS)
        assert torch.equal(h, x + r)
        check_rms_forward(h, gm, EPS, y, rstd)
        check_rms_backward(h, dy, rstd, gm, *dyt.dyt_rms_backward_residual(h, dy, r, rstd, gm), dres=r)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dt", DTYPES)
def test_8_bits(dyt, dt, N):
    for M in (1, 5, 300) if N <= 4100 else (1, 21):
        x, gm, _, r = make(N + 1, M, N, DTYPES[dt], torch.float32)
        x[:, ::61] *= 8
        for group in (0, 32, 64, 128):
            check_rms_q8(x, gm, EPS, group, *dyt.dyt_rms_forward_q8(x, gm, EPS, group))
            h, q, scales = dyt.dyt_rms_forward_residual_q8(x, r, gm, EPS, group)
            assert torch.equal(h, x + r)
            check_rms_q8(h, gm, EPS, group, q, scales)


@pytest.mark.parametrize("M,N", [(70000, 16), (200003, 5), (9000, 64), (40000, 255), (3000, 1024), (1500, 4096)])
@pytest.mark.parametrize("dt", DTYPES)
def test_many_rows(dyt, dt, M, N):
    """Several rounds of every workgroup, and the rows-at-a-time instances."""
    x, gm, dy, r = make(3, M, N, DTYPES[dt], torch.float32)
    run_plain(dyt, x, gm, dy)
    h, y, rstd = dyt.dyt_rms_forward_residual(x, r, gm, EPS)
    check_rms_forward(h, gm, EPS, y, rstd)
    check_rms_backward(h, dy, rstd, gm, *dyt.dyt_rms_backward_residual(h, dy, r, rstd, gm), dres=r)
    for group in (0, 64):
        check_rms_q8(x, gm, EPS, group, *dyt.dyt_rms_forward_q8(x, gm, EPS, group))


@pytest.mark.parametrize("M,N", [(1024, 512), (1024, 513), (1025, 1), (1025, 3), (1025, 17), (1025, 64), (1025, 127), (1025, 200),
                                 (1025, 500), (1100, 1000), (1030, 2047), (64, 8192), (64, 8193), (7, 70001), (1, 524288),
                                 (1, 524289), (1024, 4), (1000, 15)])
@pytest.mark.parametrize("dt,pdt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
def test_around_the_border_of_one_launch(dyt, dt, pdt, M, N):
    x, gm, dy, r = make(M + N, M, N, DTYPES[dt], DTYPES[pdt])
    run_plain(dyt, x, gm, dy)
    h, y, rstd = dyt.dyt_rms_forward_residual(x, r, gm, EPS)
    dx, dg = dyt.dyt_rms_backward_residual(h, dy, r, rstd, gm)
    check_rms_backward(h, dy, rstd, gm, dx, dg, dres=r)
    again = dyt.dyt_rms_backward_residual(h, dy, r, rstd, gm)
    assert torch.equal(dx, again[0]) and torch.equal(dg, again[1])


@pytest.mark.parametrize("M,N", [(9000, 8192), (600, 131072)])
def test_rows_of_large_tensors(dyt, M, N):
    """Nontemporal instances: 64 MB tensors and more; first and last rows."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, dy = (torch.randn(M, N, device="cuda", generator=g).bfloat16() for _ in range(3))
    gm = torch.randn(N, device="cuda", generator=g)
    at = [0, 1, M // 2, M - 2, M - 1]
    y, rstd = dyt.dyt_rms_forward(x, gm, EPS)
    check_rms_forward(x[at], gm, EPS, y[at], rstd[at])
    h, y, rstd = dyt.dyt_rms_forward_residual(x, r, gm, EPS)
    check_rms_forward(h[at], gm, EPS, y[at], rstd[at])
    dx, dg = dyt.dyt_rms_backward_residual(h, dy, r, rstd, gm)
    part, _ = dyt.dyt_rms_backward_residual(h[at].contiguous(), dy[at].contiguous(), r[at].contiguous(),
                                            rstd[at].contiguous(), gm)
    assert torch.equal(dx[at], part)
    want = (dy.double() * (h.double() * rstd.double().view(-1, 1))).sum(0)
    size = (dy.double() * (h.double() * rstd.double().view(-1, 1))).abs().sum(0)
    assert ((dg.double() - want).abs() <= (M / 256 + 356) * 2.0 ** -24 * 1.01 * size + 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("M,N,group", [(8300, 8192, 0), (33000, 2047, 32), (270000, 256, 128)])
def test_8_bits_of_large_tensors(dyt, M, N, group):
    """Nontemporal instances of the 8-bit output: first, middle and last rows."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x, r = (torch.randn(M, N, device="cuda", generator=g).bfloat16() for _ in range(2))
    gm = torch.randn(N, device="cuda", generator=g)
    at = [0, 1, M // 2, M - 2, M - 1]
    h, q, scales = dyt.dyt_rms_forward_residual_q8(x, r, gm, EPS, group)
    assert torch.equal(h, x + r)
    check_rms_q8(h[at], gm, EPS, group, q[at], scales[at])
    q, scales = dyt.dyt_rms_forward_q8(x, gm, EPS, group)
    check_rms_q8(x[at], gm, EPS, group, q[at], scales[at])
    few = dyt.dyt_rms_forward_q8(x[:100], gm, EPS, group)
    assert torch.equal(q[:100].view(torch.uint8), few[0].view(torch.uint8)) and torch.equal(scales[:100], few[1])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("N,pitch,at", [(64, 72, 0), (64, 67, 0), (100, 101, 3), (1000, 1032, 8), (2050, 2051, 1),
                                        (17000, 17003, 5), (70000, 70001, 3), (1, 9, 2)])
def test_row_strides(dyt, dt, N, pitch, at):
    """Rows sliced out of wider buffers, bases off the 16-byte grid; what lies
    between the rows is NaN and is neither read into a result nor written."""
    M, T = 41 if N < 50000 else 7, DTYPES[dt]
    x, gm, dy, _ = make(5, M, N, T, torch.float32)
    bufs = [torch.full((M * pitch + at,), math.nan, dtype=T, device="cuda") for _ in range(4)]
    xs, dys, ys, dxs = (b.as_strided((M, N), (pitch, 1), at) for b in bufs)
    xs.copy_(x)
    dys.copy_(dy)
    y, rstd = dyt.dyt_rms_forward(xs, gm, EPS, y=ys)
    check_rms_forward(x, gm, EPS, ys, rstd)
    dx, dg = dyt.dyt_rms_backward(xs, dys, rstd, gm, dx=dxs)
    check_rms_backward(x, dy, rstd, gm, dxs, dg)
    for b in bufs[2:]:
        assert int(torch.isnan(b).sum()) == b.numel() - M * N
    for group in (0, 32):
        check_rms_q8(x, gm, EPS, group, *dyt.dyt_rms_forward_q8(xs, gm, EPS, group))


def test_nothing_there(dyt):
    x, gm, dy, _ = make(1, 0, 40, torch.bfloat16, torch.float32)
    y, rstd = dyt.dyt_rms_forward(x, gm)
    assert y.shape == (0, 40)
    dg = torch.full((40,), 3.0, device="cuda")
    dyt.dyt_rms_backward(x, dy, rstd, gm, dgamma=dg)
    assert (dg == 0).all()
    q, scales = dyt.dyt_rms_forward_q8(x, gm, group=32)
    assert q.shape == (0, 40) and scales.shape == (0, 2)
    x, gm, dy, _ = make(1, 5, 0, torch.float32, torch.float32)
    assert dyt.dyt_rms_forward(x, gm)[0].shape == (5, 0)


def test_zero_rows_and_eps(dyt):
    x, gm, dy, _ = make(9, 6, 300, torch.float32, torch.float32)
    x[0] = 0.0
    x[1] = 2.0
    x[2] *= 1e-18
    for eps in (1e-12, 1e-5, 0.5):
        y, rstd, *_ = run_plain(dyt, x, gm, dy, eps=eps)
        assert (y[0] == 0).all()
        for group in (0, 128):
            q, scales = dyt.dyt_rms_forward_q8(x, gm, eps, group)
            assert (q[0].float() == 0).all() and (scales[0] == 2.0 ** -126).all()
            check_rms_q8(x, gm, eps, group, q, scales)


def test_nan_and_infinite_rows_stay_in_their_rows(dyt):
    x, gm, dy, _ = make(11, 70, 200, torch.float32, torch.float32)
    clean, _ = dyt.dyt_rms_forward(x, gm)
    q0, s0 = dyt.dyt_rms_forward_q8(x, gm, group=64)
    x[3, 5], x[40, 199], x[69, 0] = math.nan, math.inf, -math.inf
    y, rstd = dyt.dyt_rms_forward(x, gm)
    dx, _ = dyt.dyt_rms_backward(x, dy, rstd, gm)
    bad = [3, 40, 69]
    good = [i for i in range(70) if i not in bad]
    assert torch.equal(y[good], clean[good])
    assert torch.isnan(y[3]).all() and torch.isnan(y[40, 199]) and torch.isnan(y[69, 0])
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[good]).all()
    for group in (0, 64):
        q, s = dyt.dyt_rms_forward_q8(x, gm, group=group)
        assert torch.isnan(q[3].float()).all() and torch.isnan(q[40, 199].float()) and torch.isnan(q[69, 0].float())
        if group:
            assert torch.equal(q[good].float(), q0[good].float()) and torch.equal(s[good], s0[good])


def test_gradients_against_differences(dyt):
    x, gm, dy, _ = make(13, 30, 96, torch.float32, torch.float32)
    y, rstd = dyt.dyt_rms_forward(x, gm, EPS)
    grads = dyt.dyt_rms_backward(x, dy, rstd, gm)
    g = torch.Generator().manual_seed(17)
    for i, name in enumerate(("x", "gamma")):
        args = [x, gm]
        w = torch.randn(args[i].shape, generator=g).cuda()
        w /= w.norm()
        eps = 0.25

        def f(step):
            a = list(args)
            a[i] = a[i] + step * w
            return (d(dy) * d(dyt.dyt_rms_forward(*a, EPS)[0])).sum().item()

        d1, d2 = (f(eps) - f(-eps)) / (2 * eps), (f(eps / 2) - f(-eps / 2)) / eps
        want = (d(grads[i]) * d(w)).sum().item()
        noise = 8 * 2.0 ** -21 * (d(dy).norm() * d(y).abs().max()).item() / eps
        assert abs((4 * d2 - d1) / 3 - want) <= noise + abs(d2 - d1) / 3 + 1e-4 * abs(want), name


def test_same_bits_every_time_and_in_a_graph(dyt):
    x, gm, dy, r = make(19, 5000, 200, torch.bfloat16, torch.float32)

    def step():
        h, y, rstd = dyt.dyt_rms_forward_residual(x, r, gm)
        _, q, scales = dyt.dyt_rms_forward_residual_q8(x, r, gm, group=32)
        return (h, y, rstd, q.view(torch.uint8), scales, *dyt.dyt_rms_backward_residual(h, dy, r, rstd, gm))

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
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).cuda())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_on_another_stream(dyt):
    x, gm, dy, _ = make(23, 700, 333, torch.float16, torch.float16)
    want = (*run_plain(dyt, x, gm, dy), *dyt.dyt_rms_forward_q8(x, gm))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, rstd = dyt.dyt_rms_forward(x, gm, EPS, stream=s)
    got = (y, rstd, *dyt.dyt_rms_backward(x, dy, rstd, gm, stream=s), *dyt.dyt_rms_forward_q8(x, gm, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(want, got))


def test_offsets_past_32_bits(dyt):
    """Over 2^32 elements: rows at both ends and in between against the formula."""
    M, N = (1 << 32) // 64 + 5000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16)
    gm = torch.ones(N, device="cuda")
    y, rstd = dyt.dyt_rms_forward(x, gm, EPS)
    rows = torch.cat([torch.arange(64), torch.arange(M - 4000, M), torch.randint(0, M, (2000,))]).cuda()
    check_rms_forward(x[rows], gm, EPS, y[rows], rstd[rows])
    q, scales = dyt.dyt_rms_forward_q8(x, gm, EPS, 32)
    check_rms_q8(x[rows], gm, EPS, 32, q[rows], scales[rows])
    del q, scales
    dx, dg = dyt.dyt_rms_backward(x, y, rstd, gm)
    part, _ = dyt.dyt_rms_backward(x[rows], y[rows], rstd[rows], gm)
    assert torch.equal(dx[rows], part)
    assert dg.min().item() > 0.99 * M
