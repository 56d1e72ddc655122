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
