"""PyTorch autograd functions, modules and the optimizer for the operators
around a decoder's blocks: root-mean-square norm, embedding, log probabilities
of tokens, AdamW.

``RMSNorm`` and ``RMSNormResidual`` take the places of ``DyT`` and
``DyTResidual``: same arguments, same shapes, so a block can be built with
either. All computation of the operators runs in the HIP library; this module
only reshapes and wires autograd and the optimizer's states.
"""
from __future__ import annotations

from itertools import chain

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import _lm
from .module import _dense_rows, _rows


# ---------------------------------------------------- root-mean-square norm
class RMSNormFunction(torch.autograd.Function):
    """Saves x and the rows' reciprocal root mean square."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, gamma: torch.Tensor, eps: float) -> torch.Tensor:
        x2 = _rows(x)
        y, rstd = _lm.dyt_rms_forward(x2, gamma, eps)
        ctx.save_for_backward(x2, rstd, gamma)
        ctx.x_shape = x.shape
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor):
        x2, rstd, gamma = ctx.saved_tensors
        dx, dgamma = _lm.dyt_rms_backward(x2, _rows(dy.to(x2.dtype)), rstd, gamma)
        return dx.view(ctx.x_shape), dgamma, None


class RMSNormResidualFunction(torch.autograd.Function):
    """(x, r) -> (h = x + r, y = norm of h); the gradient of h, where there is
    one, joins in the same kernel."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, eps: float):
        h, y, rstd = _lm.dyt_rms_forward_residual(_dense_rows(x), _dense_rows(r.to(x.dtype)), gamma, eps)
        ctx.save_for_backward(h, rstd, gamma)
        ctx.set_materialize_grads(False)   # an unused output's gradient arrives as None
        ctx.x_shape = x.shape
        return h.view(x.shape), y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h: torch.Tensor | None, grad_y: torch.Tensor | None):
        h, rstd, gamma = ctx.saved_tensors
        if grad_y is None:
            if grad_h is None:
                return None, None, None, None
            dh = _dense_rows(grad_h.to(h.dtype)).view(ctx.x_shape)
            return dh, dh, None, None
        dy = _dense_rows(grad_y.to(h.dtype))
        if grad_h is None:
            dh, dgamma = _lm.dyt_rms_backward(h, dy, rstd, gamma)
        else:
            dh, dgamma = _lm.dyt_rms_backward_residual(h, dy, _dense_rows(grad_h.to(h.dtype)), rstd, gamma)
        # one tensor object for both inputs, as in DyTResidualFunction
        dh = dh.view(ctx.x_shape)
        return dh, dh, dgamma, None


def rms_norm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5) -> torch.Tensor:
    """Root-mean-square norm over the last dimension of x, with autograd support."""
    return RMSNormFunction.apply(x, gamma, eps)


def rms_norm_residual(x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5):
    """(h, y) = (x + r, norm of x + r), with autograd support."""
    return RMSNormResidualFunction.apply(x, r, gamma, eps)


class RMSNorm(nn.Module):
    """Root-mean-square norm over the last dimension; ``weight`` in ``dtype``
    (float32, bfloat16 or float16), inputs in any of the three independently of
    it. ``quantized(x, group)`` gives the norm in 8 bits with its scales."""

    def __init__(self, num_features: int, eps: float = 1e-5, dtype=torch.float32, device=None):
        super().__init__()
        self.num_features, self.eps = num_features, eps
        self.weight = nn.Parameter(torch.ones(num_features, dtype=dtype, device=device))

    def _check(self, x: torch.Tensor) -> None:
        if x.shape[-1] != self.num_features:
            raise ValueError(f"expected last dimension {self.num_features}, got {x.shape[-1]}")

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        self._check(x)
        return RMSNormFunction.apply(x, self.weight, self.eps)

    @torch.no_grad()
    def quantized(self, x: torch.Tensor, group: int = 0):
        """(q, scales) of the norm of x, for inference: q float8_e4m3fn like x,
        scales [..., 1] or [..., ceil(num_features / group)] float32."""
        self._check(x)
        q, scales = _lm.dyt_rms_forward_q8(_rows(x), self.weight, self.eps, group)
        return q.view(x.shape), scales.view(*x.shape[:-1], scales.shape[1])

    def extra_repr(self) -> str:
        return f"{self.num_features}, eps={self.eps:g}"


class RMSNormResidual(RMSNorm):
    """``forward(x, r)`` returns ``(h, y)``: h = x + r and its norm."""

    def _check2(self, x: torch.Tensor, r: torch.Tensor) -> None:
        if x.shape[-1] != self.num_features or r.shape != x.shape:
            raise ValueError(f"expected x and r of equal shape with last dimension {self.num_features}")

    def forward(self, x: torch.Tensor, r: torch.Tensor):  # type: ignore[override]
        self._check2(x, r)
        return RMSNormResidualFunction.apply(x, r, self.weight, self.eps)

    @torch.no_grad()
    def quantized(self, x: torch.Tensor, r: torch.Tensor, group: int = 0):  # type: ignore[override]
        """(h, q, scales): h = x + r and its norm in 8 bits, for inference."""
        self._check2(x, r)
        h, q, scales = _lm.dyt_rms_forward_residual_q8(_dense_rows(x), _dense_rows(r.to(x.dtype)), self.weight, self.eps,
                                                       group)
        return h.view(x.shape), q.view(x.shape), scales.view(*x.shape[:-1], scales.shape[1])


# --------------------------------------------------------------- embedding
class EmbeddingFunction(torch.autograd.Function):
    """Saves the tokens only."""

    @staticmethod
    def forward(ctx, weight: torch.Tensor, tokens: torch.Tensor, scale: float, dtype):
        at = tokens.reshape(-1).contiguous()
        w2 = _rows(weight)
        y = _lm.dyt_embed_forward(w2, at, scale, dtype)
        ctx.save_for_backward(at)
        ctx.scale, ctx.rows, ctx.w_dtype = scale, weight.shape[0], weight.dtype
        return y.view(*tokens.shape, weight.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor):
        (at,) = ctx.saved_tensors
        dw = _lm.dyt_embed_backward(_rows(dy), at, ctx.rows, ctx.scale, dtype=ctx.w_dtype)
        return dw, None, None, None


def embedding(weight: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, dtype=None) -> torch.Tensor:
    """scale * weight[tokens] in ``dtype`` (weight's), with autograd support;
    tokens outside [0, weight.shape[0]) give zeros and no gradient."""
    return EmbeddingFunction.apply(weight, tokens, scale, dtype)


class Embedding(nn.Module):
    """``scale * weight[tokens]``: a table of ``num_embeddings`` rows in
    ``dtype``. Its gradient is summed in the order of the places, so a step is
    reproducible bit by bit."""

    def __init__(self, num_embeddings: int, embedding_dim: int, scale: float = 1.0, dtype=torch.float32, device=None):
        super().__init__()
        self.num_embeddings, self.embedding_dim, self.scale = num_embeddings, embedding_dim, scale
        self.weight = nn.Parameter(torch.randn(num_embeddings, embedding_dim, dtype=dtype, device=device))

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        return EmbeddingFunction.apply(self.weight, tokens, self.scale, None)

    def extra_repr(self) -> str:
        return f"{self.num_embeddings}, {self.embedding_dim}, scale={self.scale:g}"


# ------------------------------------------------- token log probabilities
class LogProbFunction(torch.autograd.Function):
    """Saves the logits and, of each row, its log sum in two numbers (so that the
    gradient's digits do not depend on where the logits lie) and its entropy, which
    the caller may change in its own copy; the probabilities are computed again in the
    backward."""

    @staticmethod
    def forward(ctx, logits: torch.Tensor, tokens: torch.Tensor, scale: float, top: int):
        x2, at = _rows(logits), tokens.reshape(-1).contiguous()
        ctx.set_materialize_grads(False)   # an unused output's gradient arrives as None
        ctx.scale, ctx.shape = scale, logits.shape
        if x2.is_cuda and ctx.needs_input_grad[0]:
            norm = torch.empty((x2.shape[0], 3), dtype=torch.float32, device=x2.device)
            logp, entropy, _, *best = _lm.dyt_logprob_forward(x2, at, scale=scale, top=top, norm=norm)
            ctx.save_for_backward(x2, at, norm)
        else:   # (the call refuses tensors on the host)
            logp, entropy, lse, *best = _lm.dyt_logprob_forward(x2, at, scale=scale, top=top)
            ctx.save_for_backward(x2, at, entropy, lse)
            if ctx.needs_input_grad[0]:
                entropy = entropy.clone()   # the caller may change its results, the backward needs the entropy
        best = tuple(t.view(*tokens.shape, top) for t in best)
        ctx.mark_non_differentiable(*best)
        return (logp.view(tokens.shape), entropy.view(tokens.shape), *best)

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy, *_):
        x2, at, *sums = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None, None
        up = [g if g is None else g.reshape(-1).contiguous() for g in (dlogp, dentropy)]
        if len(sums) == 1:
            dx = _lm.dyt_logprob_backward(x2, at, None, None, *up, scale=ctx.scale, norm=sums[0])
        else:
            dx = _lm.dyt_logprob_backward(x2, at, *sums, *up, scale=ctx.scale)
        return dx.view(ctx.shape), None, None, None


def token_log_probs(logits: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, top: int = 0):
    """(logp, entropy), float32 like tokens: the log probabilities of tokens
    under softmax(scale * logits) over the last dimension and its entropy, both
    with autograd support. A token outside [0, V) (an ignored place) has logp 0
    and no gradient. With ``top`` also (top_logp, top_tokens) [..., top], the
    likeliest tokens in falling order, without gradient."""
    if tokens.shape != logits.shape[:-1]:
        raise ValueError(f"tokens must have shape {tuple(logits.shape[:-1])}")
    return LogProbFunction.apply(logits, tokens, scale, top)


# ------------------------------------------------------------------- AdamW
class AdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay) as one kernel over all tensors of a group.

    ``state_bits`` 8 holds both moments in 8 bits (parameters of fewer than
    ``min_8bit`` elements in 32), rounded at random by ``seed``; ``master``
    keeps a float32 copy of 16-bit parameters that the steps are taken on.
    ``capturable``: the step counter is on the device, and ``lr`` may be a
    float32 tensor there, so that a step captured into a graph moves on with
    each replay; every parameter of a group then needs a gradient, and the
    states have to be there (one step) before the capture."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01, *,
                 state_bits: int = 32, min_8bit: int = 4096, master: bool = False, seed: int = 0,
                 capturable: bool = False):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        if isinstance(lr, torch.Tensor) and not capturable:
            raise ValueError("lr as a tensor needs capturable=True")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      min_8bit=min_8bit, master=master, seed=seed, capturable=capturable))

    def _init_state(self, p: torch.Tensor, group: dict) -> dict:
        state = self.state[p]
        n, dev = p.numel(), p.device
        state["step"] = 0
        if group["state_bits"] == 8 and n >= group["min_8bit"]:
            state["exp_avg"] = torch.zeros_like(p, dtype=torch.int8)
            state["exp_avg_sq"] = torch.zeros_like(p, dtype=torch.uint8)
            for name in ("avg_scale", "sq_scale"):
                state[name] = torch.zeros(-(-n // _lm.DYT_ADAMW_BLOCK), dtype=torch.float32, device=dev)
        else:
            state["exp_avg"] = torch.zeros_like(p, dtype=torch.float32)
            state["exp_avg_sq"] = torch.zeros_like(p, dtype=torch.float32)
        if group["master"] and p.dtype != torch.float32:
            state["master"] = p.detach().float()
        return state

    @torch.no_grad()
    def step(self, closure=None, grad_scale: torch.Tensor | None = None):
        """``grad_scale``: a float32 device tensor of one element that the
        gradients are multiplied with (a clipping or unscaling factor)."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # all calls of the step, checked before the first one: a step that is refused
        # moves and counts nothing
        calls, counters = [], []
        for index, group in enumerate(self.param_groups):
            self._group_calls(index, group, grad_scale, calls, counters)
        tables = None   # (one call is checked by itself; of tensors on the host the first is refused)
        if len(calls) > 1 and any(args[0][0].is_cuda for args, _, _ in calls):
            tables = [_lm._adamw_table(*args, **kw) for args, kw, _ in calls]
            for table in tables:
                _lm._adamw_check(table)
        for counter in counters:
            counter.add_(1)
        begun = False
        try:
            for i, (args, kw, states) in enumerate(calls):
                if tables:
                    _lm._adamw_run(args[0], tables[i])
                else:
                    _lm.dyt_adamw_step(*args, **kw)
                begun = True
                if not isinstance(kw["step"], torch.Tensor):
                    for s in states:
                        s["step"] = kw["step"]
        except Exception:
            for counter in () if begun else counters:
                counter.sub_(1)
            raise
        return loss

    def _group_calls(self, index: int, group: dict, grad_scale, calls: list, counters: list) -> None:
        """Appends a group's calls, (arguments, keywords, states) each, and its
        counter on the device."""
        with_grad = [p for p in group["params"] if p.grad is not None]
        if not with_grad:
            return
        if with_grad[0].is_cuda and torch.cuda.is_current_stream_capturing():
            # a replay would take the same step again, or begin with new states
            counts = [self.state[p].get("step") for p in with_grad]
            if not group["capturable"] or not all(isinstance(c, torch.Tensor) and c is counts[0] for c in counts):
                raise RuntimeError("a captured step needs capturable=True and a step before the capture")
        for p in with_grad:
            if p.grad.is_sparse:
                raise ValueError("sparse gradients are not supported")
            if not self.state[p]:
                self._init_state(p, group)
        states = [self.state[p] for p in with_grad]
        if group["capturable"]:
            if len(with_grad) != len(group["params"]):
                raise ValueError("capturable: every parameter of a group needs a gradient")
            if not self._join_counters(states, with_grad[0].device):
                raise ValueError("capturable: a group's parameters have taken different numbers of steps")
            counters.append(states[0]["step"])
        # a call for each step count and width of the states
        members: dict = {}
        for p, s in zip(with_grad, states):
            at = None if group["capturable"] else int(s["step"]) + 1
            members.setdefault((at, "avg_scale" in s), []).append((p, s))
        for (at, bits8), pairs in members.items():
            ps = [p for p, _ in pairs]
            ss = [s for _, s in pairs]
            kw = {}
            if bits8:
                kw.update(avg_scales=[s["avg_scale"] for s in ss], sq_scales=[s["sq_scale"] for s in ss],
                          seed=group["seed"] + 0x632BE5AB * index)
            if group["master"]:
                kw.update(masters=[s.get("master") for s in ss])
            args = (ps, [p.grad.contiguous() for p in ps], [s["exp_avg"] for s in ss], [s["exp_avg_sq"] for s in ss])
            kw.update(lr=group["lr"], betas=group["betas"], eps=group["eps"], weight_decay=group["weight_decay"],
                      step=ss[0]["step"] if at is None else at, grad_scale=grad_scale)
            calls.append((args, kw, ss))

    @staticmethod
    def _join_counters(states: list, device) -> bool:
        """One counter on the device for all the states, whose counts have to be equal
        (else False, and they stay as they are)."""
        counter = states[0]["step"]
        if isinstance(counter, torch.Tensor) and all(s["step"] is counter for s in states):
            return True
        counts = {int(s["step"]) for s in states}
        if len(counts) > 1:
            return False
        if not (isinstance(counter, torch.Tensor) and counter.dtype == torch.int64 and counter.device == device):
            counter = torch.tensor(counts.pop(), dtype=torch.int64, device=device)
        for s in states:
            s["step"] = counter
        return True

    def load_state_dict(self, state_dict) -> None:
        """As the base class's, but the states keep their own types (it casts
        them to their parameters')."""
        super().load_state_dict(state_dict)
        keys = chain.from_iterable(g["params"] for g in state_dict["param_groups"])
        mine = chain.from_iterable(g["params"] for g in self.param_groups)
        for k, p in zip(keys, mine):
            for name, value in state_dict["state"].get(k, {}).items():
                if isinstance(value, torch.Tensor):
                    value = value.detach().to(p.device, copy=True)
                self.state[p][name] = value
        for group in self.param_groups:
            if isinstance(group["lr"], torch.Tensor):   # saved on whatever device
                group["lr"] = group["lr"].to(group["params"][0].device)
            # (counts that differ are refused by the next step)
            states = [self.state[p] for p in group["params"] if "step" in self.state.get(p, ())]
            if group["capturable"] and states:
                self._join_counters(states, group["params"][0].device)
