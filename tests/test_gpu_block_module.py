"""Autograd functions and modules of the block operators, and the small
decoder that runs them together."""
import importlib.util
import os

import pytest
import torch

from block_ref import HALF, Attention, check_ln_backward, check_ln_forward, d

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("small_decoder", os.path.join(ROOT, "examples", "small_decoder.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dt", DTYPES)
def test_layer_norm_modules(dyt, dt):
    T = DTYPES[dt]
    g = torch.Generator().manual_seed(1)
    layer = dyt.LayerNorm(200, device="cuda")
    res = dyt.LayerNormResidual(200, device="cuda")
    with torch.no_grad():
        for m in (layer, res):
            m.weight.copy_(1 + 0.1 * torch.randn(200, generator=g))
            m.bias.copy_(0.1 * torch.randn(200, generator=g))
    x = torch.randn(3, 7, 200, generator=g).to(T).cuda().requires_grad_()
    r = torch.randn(3, 7, 200, generator=g).to(T).cuda().requires_grad_()
    dy = torch.randn(3, 7, 200, generator=g).to(T).cuda()
    dh = torch.randn(3, 7, 200, generator=g).to(T).cuda()
    y = layer(x)
    y.backward(dy)
    flat = lambda t: t.detach().reshape(21, 200)
    _, mean, rstd = dyt.dyt_ln_forward(flat(x), layer.weight.detach(), layer.bias.detach())
    check_ln_forward(flat(x), layer.weight, layer.bias, 1e-5, flat(y), mean, rstd)
    check_ln_backward(flat(x), flat(dy), mean, rstd, layer.weight, flat(x.grad), layer.weight.grad, layer.bias.grad)
    for use_h in (True, False):
        x.grad = r.grad = res.weight.grad = res.bias.grad = None
        h, y = res(x, r)
        torch.autograd.backward([h, y] if use_h else [y], [dh, dy] if use_h else [dy])
        assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
        _, mean, rstd = dyt.dyt_ln_forward(flat(h), res.weight.detach(), res.bias.detach())
        check_ln_backward(flat(h), flat(dy), mean, rstd, res.weight, flat(x.grad), res.weight.grad, res.bias.grad,
                          dres=flat(dh) if use_h else None)
    x.grad = None
    h, _ = res(x, r)
    h.backward(dh)
    assert torch.equal(x.grad, dh)
    with pytest.raises(ValueError):
        layer(x[..., :100])


@pytest.mark.parametrize("dt", DTYPES)
def test_attention_function(dyt, dt):
    """Slices of one projection as inputs, an upstream gradient that is no
    contiguous tensor, gradients of all four inputs."""
    T = DTYPES[dt]
    g = torch.Generator().manual_seed(2)
    B, S, H, Hkv, D = 2, 90, 4, 2, 32
    qkv = torch.randn(B, S, H + 2 * Hkv, D, generator=g).to(T).cuda().requires_grad_()
    table = torch.randn(16, H, generator=g).cuda().requires_grad_()
    q, k, v = qkv.split([H, Hkv, Hkv], dim=2)
    lens = torch.tensor([90, 41], dtype=torch.int32).cuda()
    kw = dict(causal=True, seqlens_k=lens, max_distance=50, bidirectional=False)
    o = dyt.attention(q, k, v, table=table, **kw)
    do = torch.randn(B, H, S, D, generator=g).to(T).cuda().transpose(1, 2)
    o.backward(do)
    ref = Attention(q, k, v, table=table, **kw)
    _, stats = dyt.dyt_attn_forward(q.detach(), k.detach(), v.detach(), table=table.detach(), **kw)
    ref.check_forward(o, stats)
    ref.check_backward(do, *qkv.grad.split([H, Hkv, Hkv], dim=2), table.grad)
    # a sum's gradient is one value expanded over the tensor
    q2 = q.detach().requires_grad_()
    dyt.attention(q2, k.detach(), v.detach()).sum().backward()
    ones = torch.ones(B, S, H, D, dtype=T, device="cuda")
    o, stats = dyt.dyt_attn_forward(q2.detach(), k.detach(), v.detach())
    want = dyt.dyt_attn_backward(q2.detach(), k.detach(), v.detach(), o, ones, stats)[0]
    assert torch.equal(q2.grad, want)


@pytest.mark.parametrize("buckets", [0, 32])
def test_a_cache_gives_what_the_whole_sequence_gives(dyt, buckets):
    """float32: prompt and single tokens over the cache against one call."""
    torch.manual_seed(3)
    m = dyt.Attention(96, 6, 2, num_buckets=buckets, max_distance=40, device="cuda")
    if buckets:
        torch.nn.init.normal_(m.table)
    x = torch.randn(3, 30, 96, device="cuda")
    with torch.no_grad():
        want = m(x)
        cache = dyt.KVCache(3, 30, 2, 16, torch.float32)
        got = [m(x[:, :20], cache=cache)] + [m(x[:, i:i + 1], cache=cache) for i in range(20, 30)]
        assert cache.length.tolist() == [30, 30, 30]
    # both sides sum the same 96 and 30 terms of order one in other orders
    assert (torch.cat(got, 1) - want).abs().max() <= 200 * 2.0 ** -24 * 4
    with pytest.raises(ValueError):
        m(x, seqlens=cache.length, cache=cache)
    with pytest.raises(ValueError, match="no room"):
        m(x[:, :1], cache=cache)
    assert cache.length.tolist() == [30, 30, 30]


@pytest.mark.parametrize("norm", ["dyt", "layernorm"])
def test_small_decoder_learns_and_generates(dyt, example, norm):
    torch.manual_seed(4)
    model = example.Decoder(16, dim=64, heads=4, kv_heads=2, norm=norm)
    losses = example.train(model, 151, length=12, vocab=16)
    assert losses[0] > 2.5 and losses[-1] < 0.8 * losses[0]
    for name, p in model.named_parameters():
        if not name.startswith(("embed", "head")):
            assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().sum() > 0, name
    # token by token over the cache: the logits of the whole sequence, each
    # rounding of bfloat16 counted once per operator on the way (about 30)
    tokens = torch.randint(16, (5, 20), device="cuda")
    with torch.no_grad():
        want = model(tokens).float()
        caches = model.caches(5, 20)
        got = [model(tokens[:, :7], caches)] + [model(tokens[:, i:i + 1], caches) for i in range(7, 20)]
    err = (torch.cat(got, 1).float() - want).norm() / want.norm()
    assert err <= 30 * HALF[torch.bfloat16], err
    assert example.generate(model, tokens, 5).shape == (5, 5)


def test_training_matches_plain_operations(dyt):
    """One block's step in float32 against the same formulas in float64 torch
    operations on the CPU: every parameter's gradient."""
    torch.manual_seed(5)
    attn = dyt.Attention(64, 4, 2, num_buckets=16, max_distance=30, device="cuda")
    torch.nn.init.normal_(attn.table)
    norm = dyt.LayerNormResidual(64, device="cuda")
    x = torch.randn(2, 50, 64, device="cuda")
    w = torch.randn(2, 50, 64, device="cuda")
    h, y = norm(x, attn(x))
    ((h * 0.5 + y) * w).sum().backward()

    from block_ref import bucket
    p = {n: d(t).requires_grad_() for n, t in (("qkv", attn.qkv.weight), ("out", attn.out.weight), ("table", attn.table),
                                                ("g", norm.weight), ("b", norm.bias))}
    x64, w64 = d(x), d(w)
    q, k, v = (x64 @ p["qkv"].t()).view(2, 50, 8, 16).transpose(1, 2).split([4, 2, 2], 1)
    k, v = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    pos = torch.arange(50)
    rel = pos.view(1, -1) - pos.view(-1, 1)
    s = q @ k.transpose(2, 3) / 4 + p["table"].t()[:, bucket(rel, 16, 30, False)]
    o = torch.softmax(s.masked_fill(rel > 0, float("-inf")), -1) @ v
    h = x64 + o.transpose(1, 2).reshape(2, 50, 64) @ p["out"].t()
    y = torch.nn.functional.layer_norm(h, (64,), p["g"], p["b"])
    ((h * 0.5 + y) * w64).sum().backward()
    for n, got in (("qkv", attn.qkv.weight), ("out", attn.out.weight), ("table", attn.table), ("g", norm.weight),
                   ("b", norm.bias)):
        err = (d(got.grad) - p[n].grad).norm() / p[n].grad.norm()
        # sums of 100 rows' and 64 columns' float32 terms, a few operators deep
        assert err <= 500 * 2.0 ** -24, (n, err)
