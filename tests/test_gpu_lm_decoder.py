"""The small decoder example on the decoder operators: it runs, and its
gradients are those of the same formulas in float64 torch operations."""
import importlib.util
import os

import pytest
import torch

from block_ref import HALF, d

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("small_decoder", os.path.join(ROOT, "examples", "small_decoder.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_it_runs(example, bits):
    torch.manual_seed(4)
    model = example.Decoder(16, dim=64, heads=4, kv_heads=2, norm="rmsnorm")
    before = [p.detach().clone() for p in model.parameters()]
    losses = example.train(model, 3, length=12, vocab=16, log=lambda line: None, state_bits=bits)
    assert all(0 < x < 10 for x in losses)
    for (name, p), b in zip(model.named_parameters(), before):
        assert torch.isfinite(p).all() and torch.isfinite(p.grad).all() and p.grad.abs().sum() > 0, name
        assert not torch.equal(p, b), name
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


def test_its_gradients(example):
    import bwd_dyt_forward_amd as dyt
    torch.manual_seed(5)
    V, D, H, Hkv, B, S = 24, 64, 4, 2, 3, 17
    model = example.Decoder(V, dim=D, heads=H, kv_heads=Hkv, norm="rmsnorm", dtype=torch.float32)
    for name, p in model.named_parameters():
        if name.endswith("table"):
            torch.nn.init.normal_(p)
    tokens = torch.randint(V, (B, S + 1), device="cuda")
    targets = tokens[:, 1:].clone()
    targets[1, 4:] = -1
    logp, entropy = dyt.token_log_probs(model(tokens[:, :-1]), targets)
    (-logp.sum() - 0.1 * entropy.sum()).backward()

    P = {n: d(p).requires_grad_() for n, p in model.named_parameters()}

    def rms(x, name):
        return x * (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * P[name + ".weight"]

    rel = torch.arange(S).view(1, -1) - torch.arange(S).view(-1, 1)
    bucket = torch.searchsorted(torch.tensor(dyt.dyt_attn_bucket_borders(32, 128, False)), (-rel).clamp(min=0),
                                right=True) - 1

    def attend(y, name):
        h = D // H
        q, k, v = (y @ P[name + ".qkv.weight"].t()).view(B, S, H + 2 * Hkv, h).transpose(1, 2).split([H, Hkv, Hkv], 1)
        s = q @ k.repeat_interleave(H // Hkv, 1).transpose(2, 3) / h ** 0.5 + P[name + ".table"].t()[:, bucket]
        o = torch.softmax(s.masked_fill(rel > 0, float("-inf")), -1) @ v.repeat_interleave(H // Hkv, 1)
        return o.transpose(1, 2).reshape(B, S, D) @ P[name + ".out.weight"].t()

    x = P["embed.weight"][tokens[:, :-1].cpu()]
    y = rms(x, "first")
    for i in range(2):
        b = f"blocks.{i}."
        x = x + attend(y, b + "attn")
        y = torch.nn.functional.gelu(rms(x, b + "norm") @ P[b + "mlp.0.weight"].t() + P[b + "mlp.0.bias"])
        x = x + y @ P[b + "mlp.2.weight"].t() + P[b + "mlp.2.bias"]
        y = rms(x, f"norms.{i}")
    lp = torch.log_softmax(y @ P["head.weight"].t(), -1)
    at = targets.cpu()
    logp64 = lp.gather(-1, at.clamp(min=0).unsqueeze(-1)).squeeze(-1) * (at >= 0)
    (-logp64.sum() + 0.1 * (lp.exp() * lp).sum()).backward()
    assert (d(logp) - logp64.detach()).abs().max() <= 2000 * 2.0 ** -24
    for name, p in model.named_parameters():
        err = ((d(p.grad) - P[name].grad).norm() / P[name].grad.norm()).item()
        # sums of some hundred float32 terms in each of about 20 operators
        assert err <= 2000 * 2.0 ** -24, (name, err)
