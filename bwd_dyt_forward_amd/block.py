"""PyTorch autograd functions and modules for the block operators: layer norm
(plain and with the residual add in front) and attention with grouped key
heads, masks and a learned relative position bias.

``LayerNorm`` and ``LayerNormResidual`` take the places of ``DyT`` and
``DyTResidual``: same arguments, same shapes, so a block can be built with
either. ``Attention`` wraps the kernels with its two projections and a cache
for generation. All computation of the operators runs in the HIP library;
this module only reshapes and wires autograd.
"""
from __future__ import annotations

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import _block
from .module import _dense_rows, _rows


# --------------------------------------------------------------- layer norm
class LayerNormFunction(torch.autograd.Function):
    """Saves x and the rows' mean and reciprocal deviation."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float) -> torch.Tensor:
        x2 = _rows(x)
        y, mean, rstd = _block.dyt_ln_forward(x2, gamma, beta, eps)
        ctx.save_for_backward(x2, mean, rstd, gamma)
        ctx.x_shape = x.shape
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor):
        x2, mean, rstd, gamma = ctx.saved_tensors
        dx, dgamma, dbeta = _block.dyt_ln_backward(x2, _rows(dy.to(x2.dtype)), mean, rstd, gamma)
        return dx.view(ctx.x_shape), dgamma, dbeta, None


class LayerNormResidualFunction(torch.autograd.Function):
    """(x, r) -> (h = x + r, y = layer norm of h); the gradient of h, where
    there is one, joins in the same kernel."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float):
        h, y, mean, rstd = _block.dyt_ln_forward_residual(_dense_rows(x), _dense_rows(r.to(x.dtype)), gamma, beta, eps)
        ctx.save_for_backward(h, mean, rstd, gamma)
        ctx.set_materialize_grads(False)   # an unused output's gradient arrives as None
        ctx.x_shape = x.shape
        return h.view(x.shape), y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h: torch.Tensor | None, grad_y: torch.Tensor | None):
        h, mean, rstd, gamma = ctx.saved_tensors
        if grad_y is None:
            if grad_h is None:
                return None, None, None, None, None
            dh = _dense_rows(grad_h.to(h.dtype)).view(ctx.x_shape)
            return dh, dh, None, None, None
        dy = _dense_rows(grad_y.to(h.dtype))
        if grad_h is None:
            dh, dgamma, dbeta = _block.dyt_ln_backward(h, dy, mean, rstd, gamma)
        else:
            dh, dgamma, dbeta = _block.dyt_ln_backward_residual(h, dy, _dense_rows(grad_h.to(h.dtype)), mean, rstd,
                                                                gamma)
        # one tensor object for both inputs, as in DyTResidualFunction
        dh = dh.view(ctx.x_shape)
        return dh, dh, dgamma, dbeta, None


def layer_norm(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float = 1e-5) -> torch.Tensor:
    """Layer norm over the last dimension of x, with autograd support."""
    return LayerNormFunction.apply(x, gamma, beta, eps)


def layer_norm_residual(x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float = 1e-5):
    """(h, y) = (x + r, layer norm of x + r), with autograd support."""
    return LayerNormResidualFunction.apply(x, r, gamma, beta, eps)


class LayerNorm(nn.Module):
    """Layer norm over the last dimension; parameters in ``dtype`` (float32,
    bfloat16 or float16), inputs in any of the three independently of it."""

    def __init__(self, num_features: int, eps: float = 1e-5, dtype=torch.float32, device=None):
        super().__init__()
        self.num_features, self.eps = num_features, eps
        self.weight = nn.Parameter(torch.ones(num_features, dtype=dtype, device=device))
        self.bias = nn.Parameter(torch.zeros(num_features, dtype=dtype, device=device))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.num_features:
            raise ValueError(f"expected last dimension {self.num_features}, got {x.shape[-1]}")
        return LayerNormFunction.apply(x, self.weight, self.bias, self.eps)

    def extra_repr(self) -> str:
        return f"{self.num_features}, eps={self.eps:g}"


class LayerNormResidual(LayerNorm):
    """``forward(x, r)`` returns ``(h, y)``: h = x + r and its layer norm."""

    def forward(self, x: torch.Tensor, r: torch.Tensor):  # type: ignore[override]
        if x.shape[-1] != self.num_features or r.shape != x.shape:
            raise ValueError(f"expected x and r of equal shape with last dimension {self.num_features}")
        return LayerNormResidualFunction.apply(x, r, self.weight, self.bias, self.eps)


# ---------------------------------------------------------------- attention
def _unit_last(t: torch.Tensor) -> torch.Tensor:
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


_LISTS = ("seqlens_k", "q_start")


class AttentionFunction(torch.autograd.Function):
    """Saves q, k, v, the output and the rows' log sums; the probabilities are
    recomputed in the backward."""

    @staticmethod
    def forward(ctx, q, k, v, table, options: dict):
        q, k, v = _unit_last(q), _unit_last(k), _unit_last(v)
        o, stats = _block.dyt_attn_forward(q, k, v, table=table, **options)
        # the lists are saved like the others: a change before the backward is an error
        ctx.save_for_backward(q, k, v, o, stats, table, *(options.get(n) for n in _LISTS))
        ctx.options = {n: x for n, x in options.items() if n not in _LISTS}
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do: torch.Tensor):
        q, k, v, o, stats, table, *lists = ctx.saved_tensors
        grads = _block.dyt_attn_backward(q, k, v, o, _unit_last(do.to(q.dtype)), stats, table=table,
                                         **dict(zip(_LISTS, lists)), **ctx.options)
        return (*grads, None) if table is not None else (*grads, None, None)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False, scale: float | None = None,
              seqlens_k: torch.Tensor | None = None, q_start: torch.Tensor | None = None,
              table: torch.Tensor | None = None, max_distance: int = 128, bidirectional: bool = True) -> torch.Tensor:
    """dyt_attn_forward with autograd support (q, k, v and table); returns o."""
    options = dict(causal=causal, scale=scale, seqlens_k=seqlens_k, q_start=q_start, max_distance=max_distance,
                   bidirectional=bidirectional)
    return AttentionFunction.apply(q, k, v, table, options)


class KVCache:
    """Keys and values of a batch of growing sequences: k, v [B, max_len,
    heads, head_dim] and the sequences' lengths (int32, on the device).

    A cache holds values: gradients reach the keys and values of the call that
    adds them, not those of the calls before.

    An append may be captured into a graph. Its replays move the device's
    lengths only, which stop at max_len: what finds no room is dropped there (a
    position behind the last takes it) and refused by the next eager append."""

    def __init__(self, batch: int, max_len: int, num_kv_heads: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        self._k = torch.zeros(batch, max_len + 1, num_kv_heads, head_dim, dtype=dtype, device=device)
        self._v = torch.zeros_like(self._k)
        self.k, self.v = self._k[:, :max_len], self._v[:, :max_len]
        self.length = torch.zeros(batch, dtype=torch.int32, device=device)
        self._rows = torch.arange(batch, device=device).view(-1, 1)
        self._steps = torch.arange(max_len, device=device)
        self._used = 0            # the longest length, known on the host
        self._captured = False    # replays may have moved the lengths since

    def append(self, k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
        """Adds [B, S, heads, head_dim] behind each sequence; returns the
        lengths before."""
        S, max_len = k.shape[1], self.k.shape[1]
        if self.k.is_cuda and torch.cuda.is_current_stream_capturing():
            self._captured = True
        elif self._captured and self.length.numel():
            self._used = int(self.length.max())
        if S > max_len - self._used:
            raise ValueError(f"the cache holds {max_len} positions, {self._used} are taken: no room for {S} more")
        start = self.length.clone()
        at = self._places(start, S)
        with torch.no_grad():
            self._k[self._rows, at] = k
            self._v[self._rows, at] = v
        self.length.add_(S).clamp_(max=max_len)
        self._used += S   # last: what fails above takes no room
        return start

    def _places(self, start: torch.Tensor, count: int) -> torch.Tensor:
        return (start.view(-1, 1) + self._steps[:count]).clamp_(max=self.k.shape[1])

    def with_gradient(self, k: torch.Tensor, v: torch.Tensor, start: torch.Tensor):
        """The cache's keys and values, those of an append of k and v at
        `start` as part of their graph (a copy where one is needed)."""
        if not torch.is_grad_enabled() or not (k.requires_grad or v.requires_grad):
            return self.k, self.v
        at = (self._rows, self._places(start, k.shape[1]))
        return tuple(all_.index_put(at, new)[:, :-1] for all_, new in ((self._k, k), (self._v, v)))


class Attention(nn.Module):
    """Multi-head attention with its projections: one for queries, keys and
    values (whose slices the kernels read in place), one for the output.

    ``num_kv_heads`` < ``num_heads`` shares key heads between query heads;
    ``num_buckets`` > 0 adds a learned relative position bias."""

    def __init__(self, dim: int, num_heads: int, num_kv_heads: int | None = None, head_dim: int | None = None,
                 causal: bool = True, num_buckets: int = 0, max_distance: int = 128, dtype=torch.float32, device=None):
        super().__init__()
        kw = {"dtype": dtype, "device": device}
        self.num_heads, self.num_kv_heads = num_heads, num_kv_heads or num_heads
        self.head_dim = head_dim or dim // num_heads
        self.causal, self.max_distance = causal, max_distance
        self.qkv = nn.Linear(dim, (num_heads + 2 * self.num_kv_heads) * self.head_dim, bias=False, **kw)
        self.out = nn.Linear(num_heads * self.head_dim, dim, bias=False, **kw)
        self.table = nn.Parameter(torch.zeros(num_buckets, num_heads, **kw)) if num_buckets else None

    def forward(self, x: torch.Tensor, seqlens: torch.Tensor | None = None, cache: KVCache | None = None) -> torch.Tensor:
        """x [B, S, dim]. ``seqlens`` [B] int32: valid positions of each
        sequence; ``cache``: x are the next positions of its sequences."""
        B, S, _ = x.shape
        H, Hkv = self.num_heads, self.num_kv_heads
        q, k, v = self.qkv(x).view(B, S, H + 2 * Hkv, self.head_dim).split([H, Hkv, Hkv], dim=2)
        start = None
        if cache is not None:
            if seqlens is not None:
                raise ValueError("a cache keeps its own lengths: seqlens must be None")
            if B != cache.k.shape[0]:
                raise ValueError(f"the cache holds {cache.k.shape[0]} sequences, x has {B}")
            start = cache.append(k, v)
            k, v = cache.with_gradient(k, v, start)
            seqlens = cache.length.clone()
        o = attention(q, k, v, causal=self.causal, seqlens_k=seqlens, q_start=start, table=self.table,
                      max_distance=self.max_distance, bidirectional=not self.causal)
        return self.out(o.reshape(B, S, H * self.head_dim))
