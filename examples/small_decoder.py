"""A small pre-norm decoder on the package's operators: trained to repeat a
random sequence, then asked for it token by token over a key cache.

    python examples/small_decoder.py [--norm dyt|layernorm|rmsnorm] [--steps N] [--state-bits 32|8]

Each block is h = x + attention, y = norm(h) with the residual add fused into
the norm's kernel, for the norm DyT, layer norm or root-mean-square norm; the
attention shares key heads between query heads and learns a relative position
bias. The embedding, the loss and the optimizer are the package's too; of the
loss only the second halves' places count, the others' targets are -1.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_dyt_forward_amd as dyt  # noqa: E402

NORMS = {"dyt": (dyt.DyT, dyt.DyTResidual), "layernorm": (dyt.LayerNorm, dyt.LayerNormResidual),
         "rmsnorm": (dyt.RMSNorm, dyt.RMSNormResidual)}


class Block(nn.Module):
    def __init__(self, dim: int, heads: int, kv_heads: int, norm: str, **kw):
        super().__init__()
        self.attn = dyt.Attention(dim, heads, kv_heads, num_buckets=32, max_distance=128, **kw)
        self.norm = NORMS[norm][1](dim, device=kw["device"])
        self.mlp = nn.Sequential(nn.Linear(dim, 4 * dim, **kw), nn.GELU(), nn.Linear(4 * dim, dim, **kw))

    def forward(self, x, y, cache=None):
        """x: the residual stream; y: its normalised form. Returns the stream
        and what the next norm has to add to it."""
        h, y = self.norm(x, self.attn(y, cache=cache))
        return h, self.mlp(y)


class Decoder(nn.Module):
    def __init__(self, vocab: int, dim: int = 128, depth: int = 2, heads: int = 4, kv_heads: int = 2, norm: str = "dyt",
                 dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        kw = {"dtype": dtype, "device": device}
        self.embed = dyt.Embedding(vocab, dim, **kw)
        self.blocks = nn.ModuleList(Block(dim, heads, kv_heads, norm, **kw) for _ in range(depth))
        plain, residual = NORMS[norm]
        self.first = plain(dim, device=device)
        self.norms = nn.ModuleList(residual(dim, device=device) for _ in range(depth))
        self.head = nn.Linear(dim, vocab, bias=False, **kw)

    def caches(self, batch: int, max_len: int):
        a = self.blocks[0].attn
        return [dyt.KVCache(batch, max_len, a.num_kv_heads, a.head_dim, self.head.weight.dtype, self.head.weight.device)
                for _ in self.blocks]

    def forward(self, tokens, caches=None):
        x = self.embed(tokens)
        y = self.first(x)
        for i, (block, norm) in enumerate(zip(self.blocks, self.norms)):
            x, add = block(x, y, cache=caches[i] if caches else None)
            x, y = norm(x, add)
        return self.head(y)


@torch.no_grad()
def generate(model, tokens, count: int):
    """The `count` most likely next tokens of each row, one by one."""
    caches = model.caches(tokens.shape[0], tokens.shape[1] + count)
    logits = model(tokens, caches)[:, -1]
    out = []
    for i in range(count):
        out.append(logits.argmax(-1, keepdim=True))
        if i + 1 < count:
            logits = model(out[-1], caches)[:, -1]
    return torch.cat(out, 1)


def train(model, steps: int, batch: int = 32, length: int = 24, vocab: int = 32, lr: float = 2e-3, log=print,
          state_bits: int = 32):
    """Sequences of `length` tokens followed by themselves; returns the losses
    on the second halves."""
    g = torch.Generator(device="cuda").manual_seed(0)
    opt = dyt.AdamW(model.parameters(), lr=lr, weight_decay=0.0, state_bits=state_bits)
    losses = []
    for step in range(steps):
        half = torch.randint(vocab, (batch, length), device="cuda", generator=g)
        tokens = torch.cat([half, half], 1)
        targets = tokens[:, 1:].clone()
        targets[:, :length - 1] = -1
        logp, _ = dyt.token_log_probs(model(tokens[:, :-1]), targets)
        loss = -logp.sum() / half.numel()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        if step % 50 == 0 or step == steps - 1:
            losses.append(loss.item())
            log(f"step {step}: loss {losses[-1]:.3f}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--norm", choices=sorted(NORMS), default="dyt")
    ap.add_argument("--steps", type=int, default=600)
    ap.add_argument("--state-bits", type=int, choices=[8, 32], default=32)
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Decoder(32, norm=args.norm)
    train(model, args.steps, state_bits=args.state_bits)
    half = torch.randint(32, (8, 24), device="cuda")
    got = generate(model, torch.cat([half, half[:, :1]], 1), 23)
    print(f"repeated {(got == half[:, 1:]).float().mean().item():.1%} of the tokens")


if __name__ == "__main__":
    main()
