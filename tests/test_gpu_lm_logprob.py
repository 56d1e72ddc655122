"""Log probabilities of tokens on the GPU against float64 (tests/lm_ref.py)."""
import math

import pytest
import torch

from block_ref import d
from lm_ref import LogProb

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


def make(seed, T, V, dt, spread=3.0, ignored=0.1, token=torch.int64):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, V, generator=g) * spread).to(dt).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = -100
    return x, t.to(token).cuda(), torch.randn(T, generator=g).cuda(), torch.randn(T, generator=g).cuda() * 0.3


def run(dyt, x, t, up, ue, scale=1.0, top=0, ref=None):
    ref = ref or LogProb(x, t, scale)
    logp, entropy, lse, *best = dyt.dyt_logprob_forward(x, t, scale=scale, top=top)
    ref.check_forward(logp, entropy, lse)
    if top:
        ref.check_top(top, *best)
    out = [logp, entropy, lse, *best]
    for a, b in ((up, ue), (up, None), (None, ue)):
        dx = dyt.dyt_logprob_backward(x, t, entropy, lse, a, b, scale=scale)
        ref.check_backward(a, b, entropy, lse, dx)
        out.append(dx)
    return out


# around every border of the kernels' shapes, and rows that are no whole vectors
WIDTHS = [1, 2, 3, 5, 8, 9, 16, 31, 32, 33, 64, 65, 100, 127, 128, 129, 255, 256, 500, 512, 513, 1000, 1023, 1024, 1025, 2048,
          2049, 4100, 8192, 10007, 50257]


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("dt", DTYPES)
def test_widths(dyt, dt, V):
    for T in (1, 6, 700) if V <= 2049 else (1, 6):
        x, t, up, ue = make(V + T, T, V, DTYPES[dt])
        run(dyt, x, t, up, ue, top=0)
        for top in {1, min(5, V), min(20, V), min(64, V)}:
            ref = LogProb(x, t)
            logp, entropy, lse, *best = dyt.dyt_logprob_forward(x, t, top=top)
            ref.check_forward(logp, entropy, lse)
            ref.check_top(top, *best)


@pytest.mark.parametrize("T,V", [(1, 300001), (3, 128000), (40, 70000), (513, 9000), (600, 9001), (2, 1100000)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_in_parts(dyt, dt, T, V):
    x, t, up, ue = make(V, T, V, DTYPES[dt], token=torch.int32)
    run(dyt, x, t, up, ue, scale=1.25, top=20)


@pytest.mark.parametrize("scale", [1e-3, 0.7, 1.0, 2.0, 50.0])
def test_scales(dyt, scale):
    x, t, up, ue = make(3, 50, 1000, torch.float32)
    run(dyt, x, t, up, ue, scale=scale, top=7)


@pytest.mark.parametrize("V,T", [(40, 30), (3000, 20), (70000, 3)])
@pytest.mark.parametrize("dt", DTYPES)
def test_equal_and_masked_logits(dyt, dt, V, T):
    """Ties everywhere; rows with few places left, one, none; masks of -inf
    and of the type's lowest value; negative and positive zeros."""
    X = DTYPES[dt]
    x, t, up, ue = make(5, T, V, X, ignored=0.0)
    low = torch.finfo(X).min
    x[0] = 1.5
    x[1] = 0.0
    x[1, ::2] = -0.0
    x[2] = -math.inf
    x[2, V - 3] = 0.5
    x[2, 4] = -2.0
    t[2] = V - 3
    if T > 3:
        x[3] = -math.inf
        x[4] = low
        x[5] = low
        x[5, V // 2:] = 1.0
        x[6, 3:] = -math.inf
        x[7] = x[7].round()
        x[8] = -math.inf
        x[8, ::5] = low
        x[9] = 60.0
        x[9, 7] = -60.0
    run(dyt, x, t, up, ue, top=min(V, 20))
    run(dyt, x, t, up, ue, top=1)
    if T > 3:
        logp, entropy, lse = dyt.dyt_logprob_forward(x, t)
        assert logp[3] == -math.inf and lse[3] == -math.inf and entropy[3] == 0
        assert (dyt.dyt_logprob_backward(x, t, entropy, lse, up, ue)[3] == 0).all()


@pytest.mark.parametrize("V", [50, 5000, 80000])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_sorted_logits(dyt, V, order):
    x, t, up, ue = make(6, 3, V, torch.float32)
    x = torch.sort(x, 1, descending=order == "falling").values.contiguous()
    run(dyt, x, t, up, ue, top=32)


def test_nan_and_infinite_rows_stay_in_their_rows(dyt):
    for V in (60, 6000):
        x, t, up, ue = make(11, 70, V, torch.float32, ignored=0.0)
        clean = dyt.dyt_logprob_forward(x, t, top=5)
        dclean = dyt.dyt_logprob_backward(x, t, clean[1], clean[2], up, ue)
        x[3, 5], x[40, V - 1] = math.nan, math.inf
        got = dyt.dyt_logprob_forward(x, t, top=5)
        dx = dyt.dyt_logprob_backward(x, t, got[1], got[2], up, ue)
        good = [i for i in range(70) if i not in (3, 40)]
        assert all(torch.equal(a[good], b[good]) for a, b in zip(clean, got)) and torch.equal(dx[good], dclean[good])
        for a in got[:4]:
            assert torch.isnan(a[[3, 40]]).all()
        assert torch.isnan(dx[[3, 40]]).all()
        places = got[4][[3, 40]]
        assert ((places >= 0) & (places < V)).all() and all(len(set(p.tolist())) == 5 for p in places)
        # nothing flows back into them
        up[[3, 40]] = 0
        ue[[3, 40]] = 0
        assert (dyt.dyt_logprob_backward(x, t, got[1], got[2], up, ue)[[3, 40]] == 0).all()


def test_tokens_outside(dyt):
    x, t, up, ue = make(1, 200, 50, torch.float32, ignored=0.0)
    t[::7] = torch.tensor([-1, 50, 51, -(1 << 40), 1 << 40, (1 << 32) + 3, -100]).cuda().repeat(29)[:len(t[::7])]
    logp, entropy, lse, *_ = run(dyt, x, t, up, ue)
    assert (logp[::7] == 0).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V,pitch,at", [(64, 72, 0), (50, 67, 3), (5001, 5003, 1), (1, 9, 2)])
def test_row_strides(dyt, dt, V, pitch, at):
    """A vocabulary padded to its pitch: the padding holds NaN, is not read
    into a result and not written."""
    T, X = 29, DTYPES[dt]
    x, t, up, ue = make(9, T, V, X)
    bufs = [torch.full((T * pitch + at,), math.nan, dtype=X, device="cuda") for _ in range(2)]
    xs, dxs = (b.as_strided((T, V), (pitch, 1), at) for b in bufs)
    xs.copy_(x)
    ref = LogProb(x, t)
    logp, entropy, lse, *best = dyt.dyt_logprob_forward(xs, t, top=min(V, 3))
    ref.check_forward(logp, entropy, lse)
    ref.check_top(min(V, 3), *best)
    dyt.dyt_logprob_backward(xs, t, entropy, lse, up, ue, dlogits=dxs)
    ref.check_backward(up, ue, entropy, lse, dxs)
    assert int(torch.isnan(bufs[1]).sum()) == bufs[1].numel() - T * V
    want = dxs.clone()
    assert dyt.dyt_logprob_backward(xs, t, entropy, lse, up, ue, dlogits=xs) is xs   # in place
    assert torch.equal(xs, want) and int(torch.isnan(bufs[0]).sum()) == bufs[0].numel() - T * V


@pytest.mark.parametrize("T,V", [(900, 301), (30, 50257), (2, 130001)])
def test_in_place(dyt, T, V):
    x, t, up, ue = make(21, T, V, torch.bfloat16)
    logp, entropy, lse = dyt.dyt_logprob_forward(x, t)
    want = dyt.dyt_logprob_backward(x, t, entropy, lse, up, ue)
    got = dyt.dyt_logprob_backward(x, t, entropy, lse, up, ue, dlogits=x)
    assert got is x and torch.equal(got, want)


def test_nothing_there(dyt):
    x, t, up, ue = make(1, 0, 40, torch.bfloat16)
    out = dyt.dyt_logprob_forward(x, t, top=3)
    assert [tuple(o.shape) for o in out] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    assert dyt.dyt_logprob_backward(x, t, out[1], out[2], up, ue).shape == (0, 40)


def test_gradients_against_differences(dyt):
    x, t, up, ue = make(13, 20, 60, torch.float32, spread=1.0)
    logp, entropy, lse = dyt.dyt_logprob_forward(x, t, scale=1.5)
    dx = dyt.dyt_logprob_backward(x, t, entropy, lse, up, ue, scale=1.5)
    w = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).cuda()
    w /= w.norm()

    def f(step):
        a, b, _ = dyt.dyt_logprob_forward(x + step * w, t, scale=1.5)
        return (d(up) * d(a) + d(ue) * d(b)).sum().item()

    eps = 0.25
    d1, d2 = (f(eps) - f(-eps)) / (2 * eps), (f(eps / 2) - f(-eps / 2)) / eps
    want = (d(dx) * d(w)).sum().item()
    noise = 8 * 2.0 ** -20 * (d(up).abs().sum() + d(ue).abs().sum()).item() * 8 / eps
    assert abs((4 * d2 - d1) / 3 - want) <= noise + abs(d2 - d1) / 3 + 1e-4 * abs(want)


def test_same_bits_every_time_and_in_a_graph(dyt):
    x, t, up, ue = make(19, 900, 300, torch.bfloat16)
    y, s, *_ = make(20, 4, 60000, torch.bfloat16)

    def step():
        logp, entropy, lse = dyt.dyt_logprob_forward(x, t)
        return (logp, entropy, lse, dyt.dyt_logprob_backward(x, t, entropy, lse, up, ue),
                *dyt.dyt_logprob_forward(y, s, top=20))

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
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(x.shape, generator=g).cuda())
        y.copy_(torch.randn(y.shape, generator=g).cuda())
        t.copy_(torch.randint(-1, 300, t.shape, generator=g).cuda())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_on_another_stream(dyt):
    x, t, up, ue = make(23, 7, 33000, torch.float16)
    want = run(dyt, x, t, up, ue, top=4)[:6]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = list(dyt.dyt_logprob_forward(x, t, top=4, stream=s))
    got.append(dyt.dyt_logprob_backward(x, t, got[1], got[2], up, ue, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits(dyt):
    """Over 2^32 logits: rows at both ends and in between."""
    V = 50000
    T = (1 << 32) // V + 300
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, V, generator=g, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    up, ue = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    rows = [0, 1, T // 2, T - 300, T - 2, T - 1]
    out = dyt.dyt_logprob_forward(x, t, top=3)
    ref = LogProb(x[rows], t[rows])
    ref.check_forward(*(o[rows] for o in out[:3]))
    ref.check_top(3, *(o[rows] for o in out[3:]))
    dyt.dyt_logprob_backward(x, t, out[1], out[2], up, ue, dlogits=x)
    ref.check_backward(up[rows], ue[rows], out[1][rows], out[2][rows], x[rows])
