"""The block operators from their formulas in float64 on the CPU, and how far
a float32 (or 16-bit, float32-accumulating) computation may be from them.

Every bound is a sum of first-order terms, each a rounding times what it
multiplies: `half` is half a step of the storage type (eps / 2), u = 2^-24
that of float32. No constant is fitted to a result."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# smallest step of a type (its subnormals): what a rounding near zero may cost
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def d(t):
    return t.detach().double().cpu()


def check(name, got, want, bound, rms=None):
    """got within bound of want everywhere, and, for 16-bit results, the root
    mean square of the errors within twice what independent roundings give."""
    got = d(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    err = (got - want).abs()
    bad = err > bound
    if bad.any():
        i = int((err / bound.clamp(min=1e-300)).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{got.flatten()[i]:.9g}, want {want.flatten()[i]:.9g}, bound {bound.flatten()[i]:.3g}")
    if rms is not None and got.numel() >= 1000:
        e, r = err.square().mean().sqrt().item(), rms.square().mean().sqrt().item()
        assert e <= 2 * r, f"{name}: rms error {e:.4g}, of independent roundings {r:.4g}"


# --------------------------------------------------------------- layer norm
def layer_norm(x, gamma, beta, eps):
    x, gamma, beta = d(x), d(gamma), d(beta)
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    n = (x - mean) * rstd
    return n * gamma + beta, mean, rstd, n


def _sum_steps(N):
    """Roundings on the way of one element through a row's sum: in a thread
    (at most 64 of its columns, or N / 1,024 of a long row) and the lanes'
    and waves' trees."""
    return 80 + N / 1024


def check_ln_forward(x, gamma, beta, eps, y, mean, rstd):
    yr, mr, rr, n = layer_norm(x, gamma, beta, eps)
    k = _sum_steps(x.shape[1]) * U
    size = d(x).abs().mean(1, keepdim=True)
    dmean = k * size + 2 * U * mr.abs()
    check("mean", mean.view(-1, 1), mr, dmean)
    # the variance is a sum of squares around the computed mean: relative
    # error k, and the mean's own error squared (below it) counted in full
    drel = k + 4 * U + (rr * dmean).square()
    check("rstd", rstd.view(-1, 1), rr, rr * drel)
    dn = n.abs() * (drel + 4 * U) + rr * dmean + rr * U * (d(x) - mr).abs()
    h = HALF[y.dtype]
    check("y", y, yr, h * yr.abs() + TINY[y.dtype] + 1.01 * (dn * d(gamma).abs() + 2 * U * (yr.abs() + d(beta).abs())))


def check_ln_backward(x, dy, mean, rstd, gamma, dx, dgamma, dbeta, dres=None):
    """mean and rstd are the forward's float32 values, taken as given."""
    M, N = x.shape
    x64, dy64, g, m, r = d(x), d(dy), d(gamma), d(mean).view(-1, 1), d(rstd).view(-1, 1)
    n = (x64 - m) * r
    dn = 3 * U * n.abs()
    g1 = dy64 * g
    c1, c2 = g1.mean(1, keepdim=True), (g1 * n).mean(1, keepdim=True)
    want = r * (g1 - c1 - n * c2)
    k = _sum_steps(N) * U
    d1 = k * g1.abs().mean(1, keepdim=True)
    d2 = (k + 4 * U) * (g1 * n).abs().mean(1, keepdim=True)
    bound = r * (6 * U * (g1.abs() + c1.abs() + (n * c2).abs()) + d1 + n.abs() * d2 + dn * c2.abs())
    if dres is not None:
        want = want + d(dres)
        bound = bound + 2 * U * (want.abs() + d(dres).abs())
    h = HALF[dx.dtype]
    check("dx", dx, want, 1.01 * bound + h * want.abs() + TINY[dx.dtype])
    # a column's sum: rows of a thread, row groups, 16 slices
    steps = (M / 256 + 256 + 100) * U
    hp = HALF[dgamma.dtype]
    for name, got, terms in (("dgamma", dgamma, dy64 * n), ("dbeta", dbeta, dy64)):
        w = terms.sum(0)
        check(name, got, w, hp * w.abs() + TINY[dgamma.dtype] + 1.01 * steps * terms.abs().sum(0))


# ---------------------------------------------------------------- attention
def borders(buckets, distance, bidirectional):
    """Smallest distance of each bucket of one direction, in whole numbers."""
    n = buckets // 2 if bidirectional else buckets
    e = n // 2
    out = list(range(e))
    for t in range(n - e):
        x = max(out[-1], e)
        while x ** (n - e) * e ** t < distance ** t * e ** (n - e):
            x += 1
        out.append(x)
    return out


def bucket(rel, buckets, distance, bidirectional):
    b = torch.tensor(borders(buckets, distance, bidirectional))
    far = rel.abs() if bidirectional else (-rel).clamp(min=0)
    t = torch.searchsorted(b, far, right=True) - 1
    return t + (rel > 0) * (buckets // 2) if bidirectional else t


class Attention:
    """Reference and bounds of one problem. The arguments are those of
    dyt_attn_forward; results are float64, heads first."""

    def __init__(self, q, k, v, *, causal=False, scale=None, seqlens_k=None, q_start=None, table=None,
                 max_distance=128, bidirectional=True):
        B, Sq, Hq, D = q.shape
        Sk, Hkv = k.shape[1:3]
        self.dt, self.shape, self.G = q.dtype, (B, Sq, Sk, Hq, Hkv, D), Hq // Hkv
        self.scale = scale = D ** -0.5 if scale is None else scale
        lens = torch.full((B,), Sk) if seqlens_k is None else seqlens_k.cpu().long().clamp(0, Sk)
        start = torch.full((B,), Sk - Sq) if q_start is None else q_start.cpu().long()
        j = torch.arange(Sk)
        pos = start.view(-1, 1) + torch.arange(Sq)
        seen = (j < lens.view(B, 1, 1)).expand(B, Sq, Sk)
        if causal:
            seen = seen & (j <= pos.unsqueeze(-1))
        self.seen = seen.unsqueeze(1)
        used = seen.any(1).view(B, Sk, 1, 1)   # memory of keys nobody sees may hold anything
        self.q, self.k, self.v = self.heads(q), self.keys(k, used), self.keys(v, used)
        s = self.q @ self.k.transpose(2, 3) * scale
        # a float32 product of D terms and its scaling; the exponent's and the
        # logarithm's own errors (2^-22 each, and 2^-24 of their arguments)
        err = (D + 4) * U * scale * (self.q.abs() @ self.k.abs().transpose(2, 3))
        self.buckets = None
        if table is not None:
            self.table_dt = table.dtype
            self.buckets = bucket(j - pos.unsqueeze(-1), table.shape[0], max_distance, bidirectional)
            self.n_buckets = table.shape[0]
            s = s + d(table).t()[:, self.buckets].transpose(0, 1)
        s = s.masked_fill(~self.seen, -math.inf)
        top = s.amax(-1, keepdim=True) if Sk else torch.full((B, Hq, Sq, 1), -math.inf, dtype=torch.float64)
        top0 = top.masked_fill(top == -math.inf, 0)
        e = (s - top0).exp()
        total = e.sum(-1, keepdim=True)
        self.p = e / total.masked_fill(total == 0, 1)
        self.lse = (top0 + total.log()).squeeze(-1)
        size = s.masked_fill(~self.seen, 0).abs()
        # relative error of a probability
        worst = (err + 6 * U * size).amax(-1, keepdim=True) if Sk else top0 * 0
        self.rho = 2 * worst + 2.0 ** -20 + (80 + Sk / 32) * U + 4 * U * top0.abs()
        self.o = self.p @ self.v
        # 16-bit probabilities: half a step each (relative; below the type's
        # normal range, of values up to 1, absolute)
        self.hp = HALF[self.dt] if self.dt != torch.float32 else 0.0
        self.tp = 2.0 ** -25 if self.dt == torch.float16 else 0.0

    def heads(self, t):
        return d(t).transpose(1, 2)

    def keys(self, t, used=None):
        t = d(t)
        if used is not None:
            t = torch.where(used, t, torch.zeros((), dtype=torch.float64))
        return t.transpose(1, 2).repeat_interleave(self.G, 1)

    def _rounded(self, name, got, want, bound, var):
        h = HALF[got.dtype]
        bound = 1.05 * bound + h * want.abs() + TINY[got.dtype]
        rms = None
        if self.dt != torch.float32:
            rms = (var * self.hp ** 2 / 3 + (h * want) ** 2 / 3).sqrt() + TINY[got.dtype]
        check(name, got, want, bound, rms)

    def check_forward(self, o, stats):
        av = self.v.abs()
        bound = (self.hp + self.rho) * (self.p @ av) + self.tp * (self.seen.double().expand_as(self.p) @ av)
        # float32 error terms count in full next to the roundings' variance
        var = self.p.square() @ self.v.square() + self._extra((self.rho * (self.p @ av)), self.tp)
        self._rounded("o", o.transpose(1, 2), self.o, bound, var)
        s = d(stats)
        none = self.lse == -math.inf
        assert ((s == -math.inf) == none).all(), "stats: rows that see no key"
        s, w = s.masked_fill(none, 0), self.lse.masked_fill(none, 0)
        check("stats", s, w, self.rho.squeeze(-1) + 4 * U * w.abs())
        assert (d(o.transpose(1, 2))[none] == 0).all(), "o: rows that see no key"

    def _extra(self, f32, tiny):
        if not self.hp:
            return f32 * 0
        return (f32 / self.hp).square() * 3 + (tiny / self.hp) ** 2 * 3

    def check_backward(self, do, dq, dk, dv, dtable=None, o=None):
        """o: the forward's result as stored (its rounding enters delta)."""
        B, Sq, Sk, Hq, Hkv, D = self.shape
        do64 = self.heads(do)
        p, rho = self.p, self.rho
        adp = do64.abs() @ self.v.abs().transpose(2, 3)
        dp = do64 @ self.v.transpose(2, 3)
        delta = (do64 * self.o).sum(-1, keepdim=True)
        adelta = (do64.abs() * self.o.abs()).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        # what the stored o's delta is off by, as a bound and as a variance
        half = HALF[self.dt]
        doff = half * adelta + (self.hp + rho) * (do64.abs() * (p @ self.v.abs())).sum(-1, keepdim=True)
        voff = (do64 * self.o).square().sum(-1, keepdim=True) * (half ** 2 / 3)
        voff = voff + ((p.square() @ self.v.square()) * do64.square()).sum(-1, keepdim=True) * (self.hp ** 2 / 3)
        if Sk <= 256:   # dq takes it out with a second walk over the keys
            doff, voff = doff * 0, voff * 0
        dds = p * (2 * rho * (dp.abs() + delta.abs()) + (D + 8) * U * (adp + adelta))
        tiny_ds = self.tp

        def group(t):   # query heads of a key head, added up
            return t.view(B, Hkv, self.G, Sk, -1).sum(2)

        k, q = self.k, self.q
        want = ds @ k * self.scale
        steps = (80 + Sk / 32) * U
        f32 = ((dds + steps * ds.abs() + tiny_ds) @ k.abs()) * self.scale
        bound = f32 + (self.hp * ds.abs() + p * doff) @ k.abs() * self.scale
        var = ds.square() @ k.square() * self.scale ** 2
        if self.hp:
            var = var + voff * (3 / self.hp ** 2) * (p @ k * self.scale).square()
        self._rounded("dq", dq.transpose(1, 2), want, bound, var + self._extra(f32, 0.0))

        # the dk/dv kernel's delta has the rounding of o taken out up to the
        # same error made over again on dS: first order, float32 terms only,
        # and (bound) the rounding of p * dp's sum in the keys' own order
        pt, dst = p.transpose(2, 3), ds.transpose(2, 3)
        steps = (80 + Sq * self.G / 32) * U
        want = group(pt @ do64)
        f32 = group(((rho + steps) * p).transpose(2, 3) @ do64.abs()) + self.tp * group(
            self.seen.double().expand_as(p).transpose(2, 3) @ do64.abs())
        bound = f32 + self.hp * group(pt @ do64.abs())
        self._rounded("dv", dv.transpose(1, 2), want, bound, group(pt.square() @ do64.square()) + self._extra(f32, 0.0))
        want = group(dst @ q) * self.scale
        f32 = group((dds + steps * ds.abs() + tiny_ds + p * dds.sum(-1, keepdim=True)).transpose(2, 3) @ q.abs()) * self.scale
        bound = f32 + group((self.hp * ds.abs()).transpose(2, 3) @ q.abs()) * self.scale
        self._rounded("dk", dk.transpose(1, 2), want, bound,
                      group(dst.square() @ q.square()) * self.scale ** 2 + self._extra(f32, 0.0))
        if dtable is not None:
            want = torch.zeros(self.n_buckets, Hq, dtype=torch.float64)
            bound = torch.zeros_like(want)
            each = dds + p * dds.sum(-1, keepdim=True) + ds.abs() * (200 + B * Sq * Sk / 1024) * U
            for h in range(Hq):
                at = self.buckets.expand(B, Sq, Sk).reshape(-1)
                want[:, h].index_add_(0, at, ds[:, h].reshape(-1))
                bound[:, h].index_add_(0, at, each[:, h].reshape(-1))
            hb = HALF[self.table_dt]
            check("dtable", dtable, want, 1.05 * bound + hb * want.abs() + TINY[self.table_dt])
