"""Calls of the decoder operators that the documentation allows at the edges of
their ranges, on the GPU against float64."""
import math

import numpy as np
import pytest
import torch
from torch import nn

from block_ref import HALF, TINY, U, check, d
from lm_ref import EXP2, LogProb, avg_values, check_embed_backward

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


# ---------------------------------------------------- root-mean-square norm
@pytest.mark.parametrize("M,N", [(64, 8192), (700, 96), (5, 70001)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_codes_are_the_rounded_quotients(dyt, M, N, group):
    """q is y / scale, a float32 quotient, rounded to e4m3. Elements of 8 bits
    make many quotients lie next to the middle between two codes."""
    g = torch.Generator().manual_seed(N)
    x = (torch.randn(M, N, generator=g) * 1.5).bfloat16().float().cuda()
    gamma = (torch.randn(N, generator=g) * 0.1 + 1).bfloat16().float().cuda()
    x[:, ::61] *= 8
    x[:, 5::97] = 0.0
    x[:, 6::97] = -0.0
    y, _ = dyt.dyt_rms_forward(x, gamma)
    q, scales = dyt.dyt_rms_forward_q8(x, gamma, group=group)
    s = scales.cpu().repeat_interleave(group or N, 1)[:, :N]
    want = (y.cpu() / s).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 300, 5000, 70001])
def test_squares_below_the_normal_range(dyt, dt, N):
    """Elements of 3e-20 without an eps: their squares are subnormal."""
    x = torch.full((3, N), 3e-20).to(DTYPES[dt]).cuda()
    x[1] = 3e-19
    x[2, ::2] = -x[2, ::2]
    gamma, beta = torch.ones(N, device="cuda"), torch.zeros(N, device="cuda")
    y, rstd = dyt.dyt_rms_forward(x, gamma, 0.0)
    # a square of 9e-40 is rounded by up to 2^-150, as is each sum, and the mean once more
    # by its factor: 3 in 9e-40 / 2^-150, half of it in the root
    bound = 2 * 2.0 ** -150 / 8.9e-40 + 8 * U + N / 256 * U
    want = 1 / d(x).square().mean(1).sqrt()
    check("rstd", rstd, want, (bound + (80 + N / 256) * U) * want)
    n = d(x) * want.view(-1, 1)
    check("y", y, n, (bound + HALF[y.dtype] + (80 + N / 256) * U) * n.abs())
    if N % 2 == 0:   # a mean of zero
        _, mean, r = dyt.dyt_ln_forward(x[2:], gamma, beta, 0.0)
        check("layer norm's rstd", r, want[2:], (bound + (80 + N / 256) * U) * want[2:])


# --------------------------------------------------------------- embedding
@pytest.mark.parametrize("T", [5119, 5120, 5121, 6000])
@pytest.mark.parametrize("V", [300, 70000, 300000])
def test_both_sorts_of_the_embedding(dyt, T, V):
    """Around the number of tokens from which many workgroups sort."""
    g = torch.Generator().manual_seed(T)
    t = (torch.rand(T, generator=g) ** 4 * (V + 9)).long() - 4
    dy = torch.randn(T, 33, generator=g).bfloat16().cuda()
    dw = dyt.dyt_embed_backward(dy, t.cuda(), V, 3.0, dtype=torch.float32)
    check_embed_backward(dy, t, V, 3.0, dw)


# ------------------------------------------------- token log probabilities
def make(seed, T, V, dt=torch.float32, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, V, generator=g) * spread).to(dt)
    t = torch.randint(0, V, (T,), generator=g)
    t[::9] = -1
    return x, t.cuda(), torch.randn(T, generator=g).cuda(), torch.randn(T, generator=g).cuda() * 0.3


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V", [40, 3000, 70000])
def test_masked_places_under_large_gradients(dyt, dt, V):
    """A masked place's gradient is 0, however large the upstream gradients are."""
    x, t, up, ue = make(1, 4, V, DTYPES[dt])
    t[:] = 1
    x[:, 3::2] = -math.inf
    x[1, 3::2] = torch.finfo(DTYPES[dt]).min
    x = x.cuda()
    hidden = d(x) < -1e4
    _, entropy, lse = dyt.dyt_logprob_forward(x, t)
    for big in (1e9, 1e30, 3e38):
        for a, b in ((up, ue * big / 3), (up * big / 4, None), (up * big / 4, ue * big / 3)):
            dx = d(dyt.dyt_logprob_backward(x, t, entropy, lse, a, b))
            assert (dx[hidden] == 0).all(), (big, b is None)


@pytest.mark.parametrize("V,T", [(32, 200), (3000, 20), (70000, 3)])
@pytest.mark.parametrize("dt", DTYPES)
def test_a_masked_token_keeps_its_gradient(dyt, dt, V, T):
    """The row's own token at a masked place: log probability -inf, gradient scale dlogp
    there; 0 at the other masked places, and 0 everywhere in a row of nothing else."""
    X = DTYPES[dt]
    x, t, up, _ = make(2, T, V, X)
    t[:] = 5
    x[:, 4:9] = -math.inf
    x[1, 4:9] = -math.inf if dt == "f16" else torch.finfo(X).min   # (float16's lowest is far from float32's)
    x[2] = -math.inf
    x = x.cuda()
    logp, entropy, lse = dyt.dyt_logprob_forward(x, t, scale=1.5)
    assert (logp == -math.inf).all()
    dx = d(dyt.dyt_logprob_backward(x, t, entropy, lse, up, scale=1.5))
    want = 1.5 * d(up)
    want[2] = 0
    check("at the token", dx[:, 5], want, (U + HALF[X]) * want.abs() + 2.0 ** -24)
    assert (dx[:, [4, 6, 7, 8]] == 0).all() and (dx[2] == 0).all()


def check_gradient(ref, up, ue, scale, dx):
    """dlogits against the gradient of the logits themselves, in float64."""
    up = d(up).masked_fill(~ref.real, 0).view(-1, 1)
    ue = d(ue).view(-1, 1)
    none = ref.none.view(-1, 1)
    lp = (ref.x - ref.top) * ref.scale - ref.log_s.masked_fill(ref.none, 0).view(-1, 1)
    p, h = lp.exp(), ref.entropy.view(-1, 1)
    lp = lp.masked_fill(lp == -math.inf, 0)
    hit = torch.zeros_like(p)
    hit[ref.real, ref.t[ref.real]] = 1
    want = (scale * (up * (hit - p) - ue * p * (lp + h))).masked_fill(none, 0)
    away, ls, rel = (v.view(-1, 1) for v in (ref.away, ref.log_s.masked_fill(ref.none, 0).abs(), ref.rel))
    # p: of its argument the distance to the maximum (two roundings and the factor's
    # error, 4 U, which counts against the row's mean distance), log s (its sum and its
    # own error) and their difference; then the exponential
    rel_p = 8 * U * (lp.abs() + away + ls) + rel + 2 * EXP2
    # the entropy (as in LogProb.check_forward), z - lse + h and three products
    off_h = rel * (1 + 2 * away) + 6 * U * (ls + away)
    size = up.abs() + (ue * h).abs() + (ue * lp).abs()
    bound = scale * (p * (rel_p + 6 * U) * size + p * ue.abs() * (off_h + rel_p) + 2 * U * (up * hit).abs())
    # an exponential below float32's normal range counts as 0
    bound += scale * size * torch.where(p < 2.0 ** -125, 2.0 ** -126, 0.0) + U * want.abs() + 2.0 ** -149
    check("dlogits", dx, want, 1.02 * bound + HALF[dx.dtype] * want.abs() + TINY[dx.dtype])


@pytest.mark.parametrize("T,V", [(300, 32), (50, 1000), (20, 9001), (3, 70001)])
@pytest.mark.parametrize("offset", [0.0, 30.0, 1000.0, -1000.0, 30000.0])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_an_offset_of_the_logits_costs_the_gradient_nothing(dyt, T, V, offset, scale):
    x, t, up, ue = make(V, T, V)
    x = (x + offset).cuda().requires_grad_()
    logp, entropy = dyt.token_log_probs(x, t, scale)
    torch.autograd.backward([logp, entropy], [up, ue])
    check_gradient(LogProb(x, t, scale), up, ue, scale, x.grad)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,V", [(700, 50), (600, 2049), (30, 9001), (2, 130001)])
def test_the_sums_in_two_numbers(dyt, dt, T, V):
    """The kernels' own calls: the same results beside norm, its two numbers, strides,
    in place, masked rows and places, parts of a row, alternatives."""
    x, t, up, ue = make(V, T, V, DTYPES[dt])
    x[0, 1::3] = -math.inf
    if T > 2:
        x[2] = -math.inf
    t[0] = 0
    x = x.cuda()
    buf = torch.full((T, V + 3), math.nan, dtype=x.dtype, device="cuda")
    xs = buf[:, 2:2 + V]
    xs.copy_(x)
    norm = torch.full((T, 3), math.nan, device="cuda")
    top = min(V, 5)
    plain = dyt.dyt_logprob_forward(xs, t, scale=0.7, top=top)
    got = dyt.dyt_logprob_forward(xs, t, scale=0.7, top=top, norm=norm)
    assert all(torch.equal(a, b) for a, b in zip(plain, got))
    ref = LogProb(x, t, 0.7)
    real = ~ref.none
    assert (norm.cpu()[ref.none, 1] == -math.inf).all()
    # (m + log2 s) ln 2 is the lse: the factor k is off by 2 U of the maximum, the rest as in the forward
    assert torch.equal(norm[:, 2], got[1])
    lse = d(norm)[:, :2].sum(1)[real] * math.log(2)
    check("norm", lse, ref.lse[real], ref.rel[real] + 4 * U * (ref.log_s[real].abs() + ref.m[real].abs()))
    for a, b in ((up, ue), (up, None), (None, ue)):
        dx = dyt.dyt_logprob_backward(xs, t, None, None, a, b, scale=0.7, norm=norm)
        check_gradient(ref, up if a is not None else 0 * up, ue if b is not None else 0 * ue, 0.7, dx)
    again = dyt.dyt_logprob_backward(xs, t, dentropy=ue, scale=0.7, norm=norm, dlogits=xs)
    assert again is xs and torch.equal(xs, dx) and torch.isnan(buf[:, :2]).all() and torch.isnan(buf[:, 2 + V:]).all()
    with pytest.raises(ValueError, match="norm"):
        dyt.dyt_logprob_forward(x, t, norm=norm[:, 0])


@pytest.mark.parametrize("V", [16, 700, 5000, 70000])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1.3])
def test_the_log_sum_is_rounded_once(dyt, V, scale):
    """Rows of one finite logit and of two equal ones: lse is scale x (and ln 2), logp 0
    (and -ln 2), top_logp too."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((40, V), -math.inf)
    at = torch.randint(0, V - 1, (40,), generator=g)
    value = torch.randn(40, generator=g) * torch.exp(torch.randn(40, generator=g) * 3)
    x[torch.arange(40), at] = value
    x[20:][torch.arange(20), at[20:] + 1] = value[20:]
    two = (torch.arange(40) >= 20).double()
    scale = float(np.float32(scale))
    logp, entropy, lse, top_logp, _ = dyt.dyt_logprob_forward(x.cuda(), at.cuda(), scale=scale, top=2)
    want = scale * value.double() + two * math.log(2)
    # one rounding, and what s is off by: it is 2^d or twice that, where d is what m, the
    # rounded k x, leaves of k x. The hardware's exponential of that is off by EXP2 of
    # it, and its logarithm, where 2^d is not exactly 1, by a rounding.
    s_off = EXP2 + 2 * U
    check("lse", lse, want, 1.001 * U * want.abs() + s_off)
    check("logp", logp, -two * math.log(2), 1.001 * U * two + s_off)
    check("top_logp", top_logp[:, 0], -two * math.log(2), 1.001 * U * two + s_off)
    assert (top_logp[:20, 1] == -math.inf).all() and torch.equal(top_logp[20:, 0], top_logp[20:, 1])


@pytest.mark.parametrize("back", [False, True])
def test_more_rows_than_a_launch_has_workgroups(dyt, back):
    """2^24 rows of a workgroup each and a few more: the last rows as in a call of
    their own, the first too. With alternatives a row takes a workgroup however
    short it is, else one of more than 128 vectors does."""
    T, V, top = (1 << 24) + 37, 1030 if back else 16, 0 if back else 2
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, V, generator=g, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(-1, V, (T,), generator=g, device="cuda")
    out = dyt.dyt_logprob_forward(x, t, top=top)
    parts = [slice(0, 600), slice((1 << 24) - 700, T)]
    for part in parts:
        assert all(torch.equal(a[part], b) for a, b in zip(out, dyt.dyt_logprob_forward(x[part], t[part], top=top)))
    if back:
        up = torch.randn(T, generator=g, device="cuda")
        want = [dyt.dyt_logprob_backward(x[s], t[s], out[1][s], out[2][s], up[s]) for s in parts]
        dyt.dyt_logprob_backward(x, t, out[1], out[2], up, dlogits=x)
        assert all(torch.equal(x[s], w) for s, w in zip(parts, want))


# ------------------------------------------------------------------- AdamW
def nearest_avg_codes(m, scale):
    """Codes of float32 moments m [blocks, 128], rounded to the nearest, and
    where the rounding is sure."""
    y = m.abs() / scale.view(-1, 1) * 127.0 ** 2
    low = y.sqrt().floor().clamp(max=126)
    middle = low.square() + low + 0.5
    # the scale's reciprocal (2 U), two products, 1/4 and 1/2 of the rounding's square
    # and sum; the root (2 U) counts twice in y
    slack = 16 * U * y + 1e-4
    sure = (y - middle).abs() > slack
    return torch.where(y > middle, low + 1, low) * m.sign(), sure


def test_first_moments_of_small_blocks(dyt):
    """Blocks whose largest first moment is next to the least scale, 2^-126:
    every moment gets its own code."""
    most = torch.tensor([1.2e-38, 1e-37, 1e-36, 4e-35, 5e-35, 1e-30, 1e-3])
    g = torch.Generator().manual_seed(3)
    part = torch.rand(len(most), 128, generator=g) * torch.exp(-4 * torch.rand(len(most), 128, generator=g))
    part[:, 0], part[:, 1], part[:, 2], part[:, 3:6] = 1.0, 0.25, 1e-3, 0.0
    grad = (part * most.view(-1, 1)) * torch.where(torch.rand(part.shape, generator=g) < 0.5, -10.0, 10.0)
    n = grad.numel()
    p = torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sm, sv = (torch.zeros(len(most), device="cuda") for _ in range(2))
    dyt.dyt_adamw_step([p], [grad.view(-1).cuda()], [m], [v], lr=1e-3, step=1, avg_scales=[sm], sq_scales=[sv])
    moment = torch.from_numpy(grad.numpy() * np.float32(1 - 0.9)).double()   # a float32 product
    scale = moment.abs().amax(1).clamp(min=2.0 ** -126)
    assert torch.equal(d(sm), scale)
    want, sure = nearest_avg_codes(moment, scale)
    got = d(m).view(-1, 128)
    assert (got[sure] == want[sure]).all() and sure.double().mean() > 0.98
    assert ((got - want).abs() <= 1).all()


def test_small_first_moments_keep_their_digits(dyt):
    """A step without a gradient: beta1 times what the codes stand for, in blocks
    with scales down to the least."""
    scale = torch.tensor([2.0 ** -126, 1.3e-38, 1e-37, 1e-36, 3e-34, 1e-20])
    g = torch.Generator().manual_seed(4)
    codes = torch.randint(-126, 127, (len(scale), 128), generator=g).to(torch.int8)
    codes[:, 0] = 127
    n = codes.numel()
    p, grad = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = codes.view(-1).cuda(), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sm, sv = scale.cuda(), torch.zeros(len(scale), device="cuda")
    before = avg_values(m, sm).view(-1, 128)
    dyt.dyt_adamw_step([p], [grad], [m], [v], lr=1e-3, step=5, avg_scales=[sm], sq_scales=[sv])
    want = (0.9 * before[:, 0]).clamp(min=2.0 ** -126)
    # 1 / 127^2, its product, beta1 and beta1's with the scale, the moment; a subnormal
    # product is off by half its step, which 127^2 codes multiply no further
    check("scales", sm, want, 6 * U * want + 2 * 2.0 ** -150)
    codes_after, sure = nearest_avg_codes(0.9 * before, want)
    # subnormal moments are rounded to multiples of 2^-149 (beta1 times the scale too)
    y = (0.9 * before).abs() / want.view(-1, 1) * 127.0 ** 2
    low = y.sqrt().floor()
    coarse = 3 * 2.0 ** -150 / want.view(-1, 1) * 127.0 ** 2
    sure &= ((y - (low.square() + low + 0.5)).abs() > coarse)
    assert (d(m).view(-1, 128)[sure] == codes_after[sure]).all() and sure.double().mean() > 0.95


@pytest.mark.parametrize("master", [False, True])
def test_second_moments_below_the_normal_range(dyt, master):
    """Gradients of 1e-18 to 3e-20 without an eps: the second moments are subnormal, and
    the first step is lr wide all the same."""
    g = torch.tensor([1e-18, 1e-19, 3e-20, 3e-20], device="cuda").repeat_interleave(300)
    g[-300:] *= -1
    n = g.numel()
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16 if master else torch.float32)
    m, v, copy = (torch.zeros(n, device="cuda") for _ in range(3))
    dyt.dyt_adamw_step([p], [g], [m], [v], lr=0.5, betas=(0.9, 0.99), eps=0.0, weight_decay=0.0, step=1,
                       masters=[copy] if master else None)
    # v: the gradient's square and its product with 1 - beta2 are rounded to multiples of 2^-149,
    # half of which counts in the root; else some ten roundings
    bound = 0.5 * ((2.0 ** -150 / (0.01 * d(g).square()) + 2.0 ** -150 / d(g).square()) / 2 + 10 * U + 2 * EXP2)
    check("step", copy if master else p, -0.5 * d(g).sign(), 1.01 * bound)


def test_second_moments_in_8_bits_below_the_normal_range(dyt):
    """They count as zero: code 0, the least scale, and the step that eps leaves."""
    g = torch.tensor([1e-18, 3e-20], device="cuda").repeat_interleave(128)
    p, m, v = torch.zeros(256, device="cuda"), torch.zeros(256, dtype=torch.int8, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    sm, sv = (torch.zeros(2, device="cuda") for _ in range(2))
    dyt.dyt_adamw_step([p], [g], [m], [v], lr=0.5, weight_decay=0.0, step=1, avg_scales=[sm], sq_scales=[sv])
    assert (m == 127).all() and (v == 0).all() and (sv == 2.0 ** -126).all()
    want = -0.5 * d(g) / 1e-8
    check("step", p, want, (10 * U + EXP2) * want.abs() + 1e-9 * want.abs())


def test_a_refused_step_moves_and_counts_nothing(dyt):
    """Two widths of states and two groups: the last call of the step is refused."""
    for capturable in (False, True):
        for second in (False, True):
            a, b, w = (nn.Parameter(torch.randn(64, 100, device="cuda")) for _ in range(3))
            small = nn.Parameter(torch.randn(40, device="cuda"))
            groups = [{"params": [small, a]}, {"params": [b, w]}] if second else [{"params": [small, a, b, w]}]
            opt = dyt.AdamW(groups, state_bits=8, capturable=capturable)
            params = [small, a, b, w]
            for x in params:
                x.grad = torch.ones_like(x)
            opt.step()
            before = [x.detach().clone() for x in params]
            states = [{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in opt.state[x].items()} for x in params]
            w.data = w.data.t()
            w.grad = torch.ones_like(w)
            with pytest.raises(ValueError):
                opt.step()
            w.data = w.data.t()
            w.grad = torch.ones_like(w)
            # memory that is written twice: found by the library
            keep = opt.state[w]["exp_avg_sq"]
            opt.state[w]["exp_avg_sq"] = opt.state[b]["exp_avg_sq"]
            with pytest.raises(RuntimeError):
                opt.step()
            opt.state[w]["exp_avg_sq"] = keep
            assert all(torch.equal(x, y) for x, y in zip(params, before))
            for x, s in zip(params, states):
                assert all(torch.equal(v, s[k]) if isinstance(v, torch.Tensor) else v == s[k] for k, v in opt.state[x].items())
            opt.step()
            assert all(int(opt.state[x]["step"]) == 2 and not torch.equal(x, y) for x, y in zip(params, before))


def test_states_loaded_from_the_host_can_be_stepped_and_captured(dyt):
    """A checkpoint read to the host, of counters and rate on the device: the loaded
    optimizer goes on as the saved one does, in a graph too."""
    def make():
        p = [nn.Parameter(torch.full((n,), 0.5, device="cuda")) for n in (700, 5000)]
        for x in p:
            x.grad = torch.linspace(-1, 1, x.numel(), device="cuda")
        return p, dyt.AdamW(p, lr=torch.tensor(1e-2, device="cuda"), capturable=True, state_bits=8)

    p, a = make()
    a.step()
    saved = a.state_dict()
    saved["state"] = {k: {n: v.cpu() for n, v in s.items()} for k, s in saved["state"].items()}
    saved["param_groups"] = [{**g, "lr": g["lr"].cpu()} for g in saved["param_groups"]]
    q, b = make()
    b.load_state_dict(saved)
    assert b.param_groups[0]["lr"].is_cuda and b.state[q[0]]["step"] is b.state[q[1]]["step"]
    with torch.no_grad():
        for x, y in zip(p, q):
            y.copy_(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.step()
    for i in range(4):
        b.param_groups[0]["lr"].fill_(1e-2 / (i + 1))
        a.param_groups[0]["lr"].fill_(1e-2 / (i + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        a.step()
        assert all(torch.equal(x, y) for x, y in zip(p, q)), i
    assert int(b.state[q[0]]["step"]) == 5
