"""Layer norm on the GPU against the formulas in float64 (tests/block_ref.py:
every tolerance is derived there from the roundings)."""
import math

import pytest
import torch

from block_ref import check_ln_backward, check_ln_forward, d

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
    return x, (r(N) * 0.1 + 1).to(pdt).cuda(), (r(N) * 0.1).to(pdt).cuda(), r(M, N).to(dt).cuda(), r(M, N).to(dt).cuda()


def run_plain(dyt, x, gm, bt, dy, eps=EPS, **kw):
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt, eps)
    check_ln_forward(x, gm, bt, eps, y, mean, rstd)
    dx, dg, db = dyt.dyt_ln_backward(x, dy, mean, rstd, gm, **kw)
    check_ln_backward(x, dy, mean, rstd, gm, dx, dg, db)
    return y, mean, rstd, dx, dg, db


# around every border of the kernels' shapes, and rows that are no whole vectors
WIDTHS = [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 127, 128, 255, 256, 257, 500, 512, 513, 1000, 1024, 1025,
          2047, 2048, 2049, 4096, 4100, 8191, 8192, 8193, 16384, 16385, 20011, 33000]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dt,pdt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
def test_widths(dyt, dt, pdt, N):
    for M in (1, 5, 300) if N <= 4100 else (1, 37):
        x, gm, bt, dy, r = make(N, M, N, DTYPES[dt], DTYPES[pdt])
        run_plain(dyt, x, gm, bt, dy)
        h, y, mean, rstd = dyt.dyt_ln_forward_residual(x, r, gm, bt, EPS)
        assert torch.equal(h, x + r)
        check_ln_forward(h, gm, bt, EPS, y, mean, rstd)
        dx, dg, db = dyt.dyt_ln_backward_residual(h, dy, r, mean, rstd, gm)
        check_ln_backward(h, dy, mean, rstd, gm, dx, dg, db, dres=r)


@pytest.mark.parametrize("M,N", [(70000, 16), (200003, 5), (9000, 64), (40000, 255), (3000, 1024), (1500, 4096)])
@pytest.mark.parametrize("dt", DTYPES)
def test_many_rows(dyt, dt, M, N):
    """Several rounds of every workgroup, and the rows-at-a-time instances."""
    x, gm, bt, dy, r = make(3, M, N, DTYPES[dt], torch.float32)
    run_plain(dyt, x, gm, bt, dy)
    h, y, mean, rstd = dyt.dyt_ln_forward_residual(x, r, gm, bt, EPS)
    check_ln_forward(h, gm, bt, EPS, y, mean, rstd)
    check_ln_backward(h, dy, mean, rstd, gm, *dyt.dyt_ln_backward_residual(h, dy, r, mean, rstd, gm), dres=r)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("N,pitch,at", [(64, 72, 0), (64, 67, 0), (100, 101, 3), (1000, 1032, 8), (2050, 2051, 1),
                                        (17000, 17003, 5), (1, 9, 2)])
def test_row_strides(dyt, dt, N, pitch, at):
    """Rows sliced out of wider buffers, bases off the 16-byte grid; what lies
    between the rows is NaN and is neither read into a result nor written."""
    M, T = 41, DTYPES[dt]
    x, gm, bt, dy, _ = make(5, M, N, T, torch.float32)
    bufs = [torch.full((M * pitch + at,), math.nan, dtype=T, device="cuda") for _ in range(4)]
    xs, dys, ys, dxs = (b.as_strided((M, N), (pitch, 1), at) for b in bufs)
    xs.copy_(x)
    dys.copy_(dy)
    y, mean, rstd = dyt.dyt_ln_forward(xs, gm, bt, EPS, y=ys)
    check_ln_forward(x, gm, bt, EPS, ys, mean, rstd)
    dx, dg, db = dyt.dyt_ln_backward(xs, dys, mean, rstd, gm, dx=dxs)
    check_ln_backward(x, dy, mean, rstd, gm, dxs, dg, db)
    for b in bufs[2:]:
        assert int(torch.isnan(b).sum()) == b.numel() - M * N


def test_nothing_there(dyt):
    x, gm, bt, dy, _ = make(1, 0, 40, torch.bfloat16, torch.float32)
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt)
    assert y.shape == (0, 40)
    dg, db = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    dyt.dyt_ln_backward(x, dy, mean, rstd, gm, dgamma=dg, dbeta=db)
    assert (dg == 0).all() and (db == 0).all()
    x, gm, bt, dy, _ = make(1, 5, 0, torch.float32, torch.float32)
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt)
    assert y.shape == (5, 0)


@pytest.mark.parametrize("N", [48, 1000, 4096, 40000])
def test_offset_much_larger_than_the_spread(dyt, N):
    """The variance is taken around the mean: an offset of 4,000 costs a
    relative N-independent error, no cancellation of squares."""
    x, gm, bt, dy, _ = make(7, 20, N, torch.float32, torch.float32, shift=4000.0)
    run_plain(dyt, x, gm, bt, dy)


def test_constant_rows_and_eps(dyt):
    x, gm, bt, dy, _ = make(9, 6, 300, torch.float32, torch.float32)
    x[0] = 0.0
    x[1] = 2.0
    for eps in (1e-12, 1e-5, 0.5):
        y, mean, rstd, *_ = run_plain(dyt, x, gm, bt, dy, eps=eps)
        assert torch.equal(y[0], bt) and torch.equal(y[1], bt)
        assert abs(rstd[0].item() * math.sqrt(eps) - 1) < 1e-6


def test_nan_and_infinite_rows_stay_in_their_rows(dyt):
    x, gm, bt, dy, _ = make(11, 70, 200, torch.float32, torch.float32)
    clean, mean0, rstd0 = dyt.dyt_ln_forward(x, gm, bt)
    x[3, 5], x[40, 199], x[69, 0] = math.nan, math.inf, -math.inf
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt)
    dx, _, _ = dyt.dyt_ln_backward(x, dy, mean, rstd, gm)
    bad = [3, 40, 69]
    good = [i for i in range(70) if i not in bad]
    assert torch.equal(y[good], clean[good])
    assert torch.isnan(y[bad]).all() and torch.isnan(dx[bad]).all() and torch.isfinite(dx[good]).all()


def test_gradients_against_differences(dyt):
    x, gm, bt, dy, _ = make(13, 30, 96, torch.float32, torch.float32)
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt, EPS)
    grads = dyt.dyt_ln_backward(x, dy, mean, rstd, gm)
    g = torch.Generator().manual_seed(17)
    for i, name in enumerate(("x", "gamma", "beta")):
        args = [x, gm, bt]
        w = torch.randn(args[i].shape, generator=g).cuda()
        w /= w.norm()
        eps = 0.25

        def f(step):
            a = list(args)
            a[i] = a[i] + step * w
            return (d(dy) * d(dyt.dyt_ln_forward(*a, EPS)[0])).sum().item()

        d1, d2 = (f(eps) - f(-eps)) / (2 * eps), (f(eps / 2) - f(-eps / 2)) / eps
        want = (d(grads[i]) * d(w)).sum().item()
        noise = 8 * 2.0 ** -21 * (d(dy).norm() * d(y).abs().max()).item() / eps
        assert abs((4 * d2 - d1) / 3 - want) <= noise + abs(d2 - d1) / 3 + 1e-4 * abs(want), name


def test_same_bits_every_time_and_in_a_graph(dyt):
    x, gm, bt, dy, r = make(19, 5000, 200, torch.bfloat16, torch.float32)

    def step():
        h, y, mean, rstd = dyt.dyt_ln_forward_residual(x, r, gm, bt)
        return (h, y, mean, rstd, *dyt.dyt_ln_backward_residual(h, dy, r, mean, rstd, gm))

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
    x, gm, bt, dy, _ = make(23, 700, 333, torch.float16, torch.float16)
    want = run_plain(dyt, x, gm, bt, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt, EPS, stream=s)
    got = (y, mean, rstd, *dyt.dyt_ln_backward(x, dy, mean, rstd, gm, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits(dyt):
    """Over 2^32 elements: rows at both ends and in between against the formula."""
    M, N = (1 << 32) // 64 + 5000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16)
    gm, bt = torch.ones(N, device="cuda"), torch.zeros(N, device="cuda")
    y, mean, rstd = dyt.dyt_ln_forward(x, gm, bt, EPS)
    rows = torch.cat([torch.arange(64), torch.arange(M - 4000, M), torch.randint(0, M, (2000,))]).cuda()
    check_ln_forward(x[rows], gm, bt, EPS, y[rows], mean[rows], rstd[rows])
    dx, dg, db = dyt.dyt_ln_backward(x, y, mean, rstd, gm)
    n = (d(x[rows]) - d(mean[rows]).view(-1, 1)) * d(rstd[rows]).view(-1, 1)
    dy = d(y[rows])
    want = d(rstd[rows]).view(-1, 1) * (dy - dy.mean(1, keepdim=True) - n * (dy * n).mean(1, keepdim=True))
    # dy = y is n rounded, so dx is what the rounding left: absolute float32 error of terms near |n|
    assert ((d(dx[rows]) - want).abs() <= 2.0 ** -8 * want.abs() + 120 * 2.0 ** -24 * (n.abs() + 1) * (n.abs() + 2)).all()
    assert dg.min().item() > 0.99 * M and torch.isfinite(db).all()
