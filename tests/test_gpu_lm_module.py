"""The decoder operators' modules and optimizer, and a run of them together."""
import math
import os
import sys

import pytest
import torch
from torch import nn

from block_ref import d

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


def near(name, got, want, steps=500):
    """Sums of some hundred float32 terms, a few operators deep."""
    err = ((d(got) - want).norm() / want.norm()).item()
    assert err <= steps * 2.0 ** -24, f"{name}: relative error {err:.3g}"


def test_a_run_of_all_of_them(dyt):
    """Embedding, residual norm, head, log probabilities and entropy, forward
    and backward in float32 against torch in float64."""
    torch.manual_seed(0)
    V, D, B, S = 50, 48, 3, 21
    emb = dyt.Embedding(V, D, scale=math.sqrt(D), device="cuda")
    first, norm = dyt.RMSNorm(D, device="cuda"), dyt.RMSNormResidual(D, device="cuda")
    head = nn.Linear(D, V, bias=False, device="cuda")
    nn.init.normal_(first.weight, 1.0, 0.1)
    nn.init.normal_(norm.weight, 1.0, 0.1)
    tokens = torch.randint(0, V, (B, S), device="cuda")
    targets = torch.randint(0, V, (B, S), device="cuda")
    targets[0, 5:] = -1
    tokens[1, :3] = -1
    x = emb(tokens)
    h, y = norm(x, first(x))
    logp, entropy = dyt.token_log_probs(head(y), targets, scale=0.9)
    (h.square().mean() - logp.sum() - 0.1 * entropy.sum()).backward()
    params = [emb.weight, first.weight, norm.weight, head.weight]
    we, g1, g2, wh = (p.detach().double().cpu().requires_grad_() for p in params)
    t, c = tokens.cpu(), targets.cpu()
    x64 = we[t.clamp(min=0)] * math.sqrt(D) * (t >= 0).unsqueeze(-1)

    def rms(v, g):
        return v * (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * g

    h64 = x64 + rms(x64, g1)
    lp = torch.log_softmax(rms(h64, g2) @ wh.t() * 0.9, -1)
    logp64 = lp.gather(-1, c.clamp(min=0).unsqueeze(-1)).squeeze(-1) * (c >= 0)
    ent64 = -(lp.exp() * lp).sum(-1)
    (h64.square().mean() - logp64.sum() - 0.1 * ent64.sum()).backward()
    for name, a, b in [("h", h, h64), ("logp", logp, logp64), ("entropy", entropy, ent64)] + [
            (n, p.grad, r.grad) for n, p, r in zip(("embedding", "first", "norm", "head"), params, (we, g1, g2, wh))]:
        near(name, a.detach(), b.detach())
    assert emb.weight.grad.shape == emb.weight.shape


def test_gradients_reach_only_what_asks(dyt):
    x = torch.randn(5, 7, 32, device="cuda", requires_grad=True)
    r = torch.randn(5, 7, 32, device="cuda", requires_grad=True)
    norm = dyt.RMSNormResidual(32, device="cuda")
    h, y = norm(x, r)
    h.sum().backward()
    assert (x.grad == 1).all() and (r.grad == 1).all() and norm.weight.grad is None
    x.grad += 1   # not one tensor with r's
    assert (r.grad == 1).all()
    x.grad = r.grad = None
    h, y = norm(x, r)
    y.sum().backward()
    assert torch.equal(x.grad, r.grad)
    logits = torch.randn(6, 40, device="cuda", requires_grad=True)
    t = torch.randint(0, 40, (6,), device="cuda")
    logp, entropy, best, places = dyt.token_log_probs(logits, t, top=3)
    assert not best.requires_grad and not places.requires_grad
    entropy.sum().backward()
    p = torch.softmax(logits.detach().double(), -1)
    want = -p * (p.log() - (p * p.log()).sum(-1, keepdim=True))
    near("entropy's gradient", logits.grad, want.cpu())
    logits.grad = None
    logp, _ = dyt.token_log_probs(logits, t)
    logp.sum().backward()
    near("logp's gradient", logits.grad, (nn.functional.one_hot(t, 40) - p).cpu())
    assert torch.equal(places.cpu(), torch.topk(logits.detach(), 3).indices.cpu())


def test_saved_tensors_are_guarded(dyt):
    emb = dyt.Embedding(10, 16, device="cuda")
    t = torch.randint(0, 10, (9,), device="cuda")
    y = emb(t)
    t.add_(0)
    with pytest.raises(RuntimeError):
        y.sum().backward()
    logits = torch.randn(6, 40, device="cuda", requires_grad=True)
    t = torch.randint(0, 40, (6,), device="cuda")
    logp, entropy = dyt.token_log_probs(logits, t)
    entropy.detach().mul_(2)   # the caller's own copy
    logp.sum().backward()
    logp, _ = dyt.token_log_probs(logits, t)
    t.add_(0)
    with pytest.raises(RuntimeError):
        logp.sum().backward()
    p = nn.Parameter(torch.randn(40, device="cuda"))
    y = (p * p).sum()
    p.grad = torch.ones_like(p)
    dyt.AdamW([p]).step()
    with pytest.raises(RuntimeError):
        y.backward()


def test_quantized_norm(dyt):
    norm, res = dyt.RMSNorm(200, device="cuda"), dyt.RMSNormResidual(200, device="cuda")
    x, r = torch.randn(3, 5, 200, device="cuda").bfloat16(), torch.randn(3, 5, 200, device="cuda").bfloat16()
    q, s = norm.quantized(x)
    assert q.shape == x.shape and s.shape == (3, 5, 1)
    y = norm(x).float()
    # half a step of four significant bits, and y's own rounding
    assert ((q.float() * s - y).abs() <= (2.0 ** -4 + 2.0 ** -7) * y.abs() + 2.0 ** -9 * s).all()
    h, q, s = res.quantized(x, r, group=64)
    assert s.shape == (3, 5, 4) and torch.equal(h, res(x, r)[0])
    q, s = norm.quantized(x.transpose(0, 1), 32)
    assert torch.equal(q.transpose(0, 1).float(), norm.quantized(x, 32)[0].float())


def _train(opt_of, dtype, steps=12):
    torch.manual_seed(1)
    net = nn.Sequential(nn.Linear(64, 96, dtype=dtype), nn.GELU(), nn.Linear(96, 10, dtype=dtype)).cuda()
    opt = opt_of(net.parameters())
    x = torch.randn(32, 64, device="cuda").to(dtype)
    y = torch.randn(32, 10, device="cuda").to(dtype)
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        (net(x) - y).float().square().mean().backward()
        opt.step()
    return net, opt


def test_optimizer_against_torch(dyt):
    """float32 states: torch's own AdamW in float64 on the same gradients."""
    torch.manual_seed(2)
    p = [nn.Parameter(torch.randn(n, device="cuda")) for n in (5, 130, 9000)]
    q = [nn.Parameter(x.detach().double().cpu()) for x in p]
    kw = dict(lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.05)
    groups = lambda ps: [{"params": ps[:1], "lr": 1e-2}, {"params": ps[1:]}]
    a, b = dyt.AdamW(groups(p), **kw), torch.optim.AdamW(groups(q), **kw)
    for step in range(10):
        for x, y in zip(p, q):
            y.grad = torch.randn(y.shape, generator=torch.Generator().manual_seed(step)).double()
            x.grad = y.grad.float().cuda()
            if step % 3 == 1 and x is p[1]:
                x.grad = y.grad = None   # no gradient in this step: its count stays
        a.step()
        b.step()
    for x, y in zip(p, q):
        near("parameter", x.detach(), y.detach(), 100)


@pytest.mark.parametrize("bits,master,dtype", [(32, False, torch.float32), (32, True, torch.bfloat16), (8, False, torch.bfloat16),
                                               (8, True, torch.float16), (8, False, torch.float32)])
def test_optimizer_states_survive_saving(dyt, bits, master, dtype):
    make = lambda ps: dyt.AdamW(ps, lr=1e-3, state_bits=bits, master=master, min_8bit=500, seed=4)
    net, opt = _train(make, dtype)
    saved = opt.state_dict()
    net2, _ = _train(make, dtype, steps=1)
    net2.load_state_dict(net.state_dict())
    opt2 = make(net2.parameters())
    opt2.load_state_dict(saved)
    for p, q in zip(net.parameters(), net2.parameters()):
        a, b = opt.state[p], opt2.state[q]
        assert a.keys() == b.keys()
        for k in a:
            assert type(a[k]) is type(b[k])
            if isinstance(a[k], torch.Tensor):
                assert a[k].dtype == b[k].dtype and torch.equal(a[k], b[k]) and a[k].data_ptr() != b[k].data_ptr()
        assert (opt.state[p]["exp_avg"].dtype == torch.int8) == (bits == 8 and p.numel() >= 500)
        p.grad = torch.ones_like(p)
        q.grad = torch.ones_like(q)
    opt.step()
    opt2.step()
    assert all(torch.equal(p, q) for p, q in zip(net.parameters(), net2.parameters()))


def test_optimizer_in_a_graph(dyt):
    """A captured step: its counter moves on with each replay."""
    torch.manual_seed(3)
    p, q = ([nn.Parameter(torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()) for n in (700, 33)] for _ in range(2))
    for x in p + q:
        x.grad = torch.zeros_like(x)
    a, b = dyt.AdamW(p, lr=1e-2, capturable=True), dyt.AdamW(q, lr=1e-2)
    grads = [torch.randn(6, x.numel(), device="cuda") for x in p]

    def feed(i):
        for x, y, g in zip(p, q, grads):
            x.grad.copy_(g[i])
            y.grad.copy_(g[i])

    feed(0)
    a.step()
    b.step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.step()
    for i in range(1, 6):
        feed(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.step()
        for x, y in zip(p, q):
            assert ((x - y).abs() <= 2.0 ** -20 * (y.abs() + 0.2)).all(), i
    assert a.state[p[0]]["step"].item() == 6
    del p[1].grad
    p[1].grad = None
    with pytest.raises(ValueError):
        a.step()


def test_optimizer_refusals(dyt):
    p = nn.Parameter(torch.randn(8, device="cuda"))
    with pytest.raises(ValueError):
        dyt.AdamW([p], state_bits=16)
    with pytest.raises(ValueError):
        dyt.AdamW([p], lr=torch.tensor(1e-3, device="cuda"))
    opt = dyt.AdamW([p])
    opt.step()   # no gradients: nothing
    assert not opt.state[p]
    w = nn.Parameter(torch.randn(4, 6, device="cuda").t())
    w.grad = torch.ones_like(w)
    with pytest.raises(ValueError):
        dyt.AdamW([w]).step()


def test_a_refused_step_does_not_count(dyt):
    p, w = nn.Parameter(torch.randn(8, device="cuda")), nn.Parameter(torch.randn(4, 6, device="cuda"))
    opt = dyt.AdamW([p, w])
    for x in (p, w):
        x.grad = torch.ones_like(x)
    opt.step()
    before, w.data = p.detach().clone(), w.data.t()
    w.grad = torch.ones_like(w)
    with pytest.raises(ValueError):
        opt.step()
    assert torch.equal(p, before) and opt.state[p]["step"] == opt.state[w]["step"] == 1


def test_nothing_there(dyt):
    """Modules over no tokens and no rows: empty results, zero gradients."""
    emb, norm, res = dyt.Embedding(7, 16, device="cuda"), dyt.RMSNorm(16, device="cuda"), dyt.RMSNormResidual(16, device="cuda")
    tokens = torch.zeros(2, 0, dtype=torch.int64, device="cuda")
    h, y = res(emb(tokens), norm(emb(tokens)))
    logits = y @ emb.weight.t()
    logp, entropy, best, places = dyt.token_log_probs(logits, tokens, top=2)
    assert logp.shape == entropy.shape == (2, 0) and best.shape == places.shape == (2, 0, 2)
    (logp.sum() + entropy.sum() + h.sum()).backward()
    assert (emb.weight.grad == 0).all() and (norm.weight.grad == 0).all() and (res.weight.grad == 0).all()
    q, s = norm.quantized(torch.zeros(0, 16, device="cuda"), group=32)
    assert q.shape == (0, 16) and s.shape == (0, 1)


@pytest.mark.parametrize("expand", [False, True])
def test_upstream_gradients_of_any_strides(dyt, expand):
    """Gradients that arrive expanded or transposed, as from sums and means."""
    emb, norm = dyt.Embedding(9, 24, device="cuda"), dyt.RMSNorm(24, device="cuda")
    tokens = torch.randint(0, 9, (4, 5), device="cuda")
    w = torch.randn(24, 5, 4, device="cuda")
    for back in (lambda y: y.sum(), lambda y: y.mean(0).sum()) if expand else (lambda y: (y.permute(2, 1, 0) * w).sum(),):
        got, want = [], []
        for contiguous in (False, True):
            y = norm(emb(tokens))
            if contiguous:
                y.register_hook(lambda g: g.contiguous())
            back(y).backward()
            (want if contiguous else got).extend(p.grad.clone() for p in (emb.weight, norm.weight))
            emb.weight.grad = norm.weight.grad = None
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(a.abs().sum() > 0 for a in got)


def test_two_graphs_and_eager_work_between(dyt):
    """Two captured training steps of the operators replayed in turn, with eager
    calls of other sizes between: no workspace is shared."""
    def make(seed, V, D, T):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)
        return dict(w=r(V, D), g=1 + 0.1 * r(D), t=torch.randint(-1, V, (T,), device="cuda", generator=g), up=r(T))

    def step(s):
        x = dyt.dyt_embed_forward(s["w"], s["t"])
        y, rstd = dyt.dyt_rms_forward(x, s["g"])
        logits = y @ s["w"].t()
        logp, entropy, lse = dyt.dyt_logprob_forward(logits, s["t"])
        dl = dyt.dyt_logprob_backward(logits, s["t"], entropy, lse, s["up"], s["up"])
        dx, dg = dyt.dyt_rms_backward(x, dl @ s["w"], rstd, s["g"])
        return logp, entropy, dx, dg, dyt.dyt_embed_backward(dx, s["t"], s["w"].shape[0])

    sets = [make(1, 300, 64, 4000), make(2, 50, 96, 900)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            step(s)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in sets], []
    for graph, s in zip(graphs, sets):
        with torch.cuda.graph(graph):
            outs.append(step(s))
    for i in range(4):
        for s in sets:
            s["t"].copy_(torch.randint(-1, s["w"].shape[0], s["t"].shape, generator=torch.Generator().manual_seed(i)).cuda())
        want = [step(s) for s in sets]
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        step(make(i, 100, 32, 5000))
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), i


def test_single_rows_and_single_tokens(dyt):
    """A vector in place of a batch: one dimension, and tokens of none."""
    emb, norm, res = dyt.Embedding(7, 40, device="cuda"), dyt.RMSNorm(40, device="cuda"), dyt.RMSNormResidual(40, device="cuda")
    token = torch.tensor(3, device="cuda")
    h, y = res(emb(token), norm(emb(token)))
    assert h.shape == y.shape == (40,)
    logits = emb.weight @ y
    logp, entropy, best, places = dyt.token_log_probs(logits, token, top=2)
    assert logp.shape == entropy.shape == () and best.shape == places.shape == (2,)
    (logp + entropy).backward()
    # logp is next to 0 here (the token's own row): its error is that of a sum of seven
    # exponentials and its logarithm (10 roundings of numbers of order one) and of the
    # difference of two logits (two roundings of them)
    off = (d(logp) - torch.log_softmax(d(logits), 0)[3]).abs()
    assert off <= (10 + 2 * d(logits).abs().max()) * 2.0 ** -24
    assert emb.weight.grad.shape == (7, 40) and torch.isfinite(emb.weight.grad).all() and norm.weight.grad.abs().sum() > 0
    q, s = norm.quantized(y.detach(), group=32)
    assert q.shape == (40,) and s.shape == (2,)


def test_two_streams_at_once(dyt):
    """The same calls on two streams at the same time: no memory between them."""
    g = torch.Generator(device="cuda").manual_seed(8)
    sets = [dict(t=torch.randint(-1, 900, (T,), device="cuda", generator=g), dy=torch.randn(T, 200, device="cuda", generator=g),
                 x=torch.randn(T, 900, device="cuda", generator=g), gamma=torch.ones(200, device="cuda")) for T in (6000, 7000)]

    def work(s):
        dw = dyt.dyt_embed_backward(s["dy"], s["t"], 900)
        logp, entropy, lse, best, at = dyt.dyt_logprob_forward(s["x"][:300], s["t"][:300], top=5)
        y, rstd = dyt.dyt_rms_forward(s["dy"], s["gamma"])
        return (dw, logp, entropy, lse, best, at, y, *dyt.dyt_rms_backward(s["dy"], y, rstd, s["gamma"]))

    want = [work(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for stream, s in zip(streams, sets):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                got.append(work(s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("capturable", [False, True])
def test_a_capture_without_states_or_counter_is_refused(dyt, capturable):
    p = nn.Parameter(torch.randn(64, device="cuda"))
    p.grad = torch.ones_like(p)
    opt = dyt.AdamW([p], capturable=capturable)
    if not capturable:
        opt.step()
    before = p.detach().clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(RuntimeError, match="capture"):
            opt.step()
        p.grad.add_(0)   # a graph of something
    torch.cuda.synchronize()
    assert torch.equal(p, before)
    opt.step()
    assert not torch.equal(p, before)
