"""The operators around a decoder's blocks from their formulas in float64 on
the CPU, and how far a float32 (or 16-bit, float32-accumulating) computation
may be from them. As in block_ref.py every bound is a sum of first-order terms,
each a rounding times what it multiplies, and no constant is fitted to a
result; EXP2 is the error of a hardware exponential or logarithm (two units in
the last place at most)."""
from __future__ import annotations

import math

import torch

from block_ref import HALF, TINY, U, _sum_steps, check, d

EXP2 = 2.0 ** -22


# ---------------------------------------------------- root-mean-square norm
def rms_norm(x, gamma, eps):
    x = d(x)
    rstd = (x.square().mean(1, keepdim=True) + eps).rsqrt()
    n = x * rstd
    return n * d(gamma), rstd, n


def _rstd_rel(N):
    """Relative error of rstd: a sum of positive squares, its mean and root."""
    return (_sum_steps(N) + 6) * U


def check_rms_forward(x, gamma, eps, y, rstd):
    want, r, _ = rms_norm(x, gamma, eps)
    rel = _rstd_rel(x.shape[1])
    check("rstd", rstd.view(-1, 1), r, rel * r)
    check("y", y, want, HALF[y.dtype] * want.abs() + TINY[y.dtype] + 1.01 * (rel + 3 * U) * want.abs())


def check_rms_q8(x, gamma, eps, group, q, scales):
    y, _, _ = rms_norm(x, gamma, eps)
    M, N = y.shape
    G = group or max(N, 1)
    rel = _rstd_rel(N) + 3 * U
    parts = y.split(G, dim=1)
    top = torch.stack([p.abs().amax(1) for p in parts], 1)
    want = (top / 448).clamp(min=2.0 ** -126)
    check("scales", scales, want, (rel + 2 * U) * want)
    s = d(scales).repeat_interleave(G, 1)[:, :N]
    value = d(q.float()) * s
    # half a step of four significant bits, or of the multiples of 2^-9 below
    # 2^-6; the quotient that is rounded is off by rel and two roundings more
    bound = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * 1.001 + 1.01 * (rel + 4 * U) * y.abs()
    check("q", value, y, bound)
    assert (d(q.float()).abs() <= 448).all()


def check_rms_backward(x, dy, rstd, gamma, dx, dgamma, dres=None):
    """rstd is the forward's float32 value, taken as given."""
    M, N = x.shape
    x64, dy64, g, r = d(x), d(dy), d(gamma), d(rstd).view(-1, 1)
    n = x64 * r
    g1 = dy64 * g
    c2 = (g1 * n).mean(1, keepdim=True)
    want = r * (g1 - n * c2)
    d2 = (_sum_steps(N) + 4) * U * (g1 * n).abs().mean(1, keepdim=True)
    bound = r * (6 * U * (g1.abs() + (n * c2).abs()) + n.abs() * d2)
    if dres is not None:
        want = want + d(dres)
        bound = bound + 2 * U * (want.abs() + d(dres).abs())
    check("dx", dx, want, 1.01 * bound + HALF[dx.dtype] * want.abs() + TINY[dx.dtype])
    # a column's sum: rows of a thread, row groups, 16 slices
    steps = (M / 256 + 256 + 100) * U
    terms = dy64 * n
    w = terms.sum(0)
    check("dgamma", dgamma, w, HALF[dgamma.dtype] * w.abs() + TINY[dgamma.dtype] + 1.01 * steps * terms.abs().sum(0))


# --------------------------------------------------------------- embedding
def _real(tokens, V):
    t = tokens.cpu().long()
    return t, (t >= 0) & (t < V)


def check_embed_forward(weight, tokens, scale, y):
    t, real = _real(tokens, weight.shape[0])
    want = torch.zeros(y.shape, dtype=torch.float64)
    if weight.shape[0]:
        want[real] = d(weight)[t[real]] * scale
    # the scale and the product in float32, then the result's type
    check("y", y, want, HALF[y.dtype] * want.abs() + 2.01 * U * want.abs() + TINY[y.dtype])
    assert (d(y)[~real] == 0).all()


def check_embed_backward(dy, tokens, V, scale, dweight, before=None):
    """before: what dweight held, where the gradient is added to it."""
    t, real = _real(tokens, V)
    dy64 = d(dy)[real]
    want = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, t[real], dy64) * scale
    size = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, t[real], dy64.abs()) * abs(scale)
    count = torch.zeros(V, 1, dtype=torch.float64).index_add_(0, t[real], torch.ones(int(real.sum()), 1, dtype=torch.float64))
    # a sum of n terms rounds n - 1 times, in whatever order; the scale and its product
    bound = 1.01 * (count + 2) * U * size
    if before is not None:
        want = want + d(before)
        bound = bound + U * want.abs()
    h = HALF[dweight.dtype]
    touched = (count > 0).expand_as(want)
    check("dweight", dweight, want, torch.where(touched, bound + h * want.abs() + TINY[dweight.dtype], 0.0))


# ------------------------------------------------- token log probabilities
class LogProb:
    """Reference and bounds of one problem."""

    def __init__(self, logits, tokens, scale=1.0):
        x = d(logits)
        self.raw, self.scale = x, scale
        # beyond float32 as a power of two: masked, as -inf
        x = x.masked_fill(x * scale < -3.402823466e38 * math.log(2), -math.inf)
        self.x = x
        T, V = x.shape
        self.t, self.real = _real(tokens, V)
        m = x.amax(1, keepdim=True)
        self.none = (m == -math.inf).squeeze(1)
        m = m.masked_fill(m == -math.inf, 0)
        self.top = m
        z = (x - m) * scale
        e = z.exp()
        s = e.sum(1, keepdim=True)
        s1 = s.masked_fill(s == 0, 1)
        self.p = e / s1
        z0 = z.masked_fill(z == -math.inf, 0)
        self.away = (self.p * z0.abs()).sum(1)       # mean distance from the maximum
        self.log_s, self.m = s.log().squeeze(1), (m * scale).squeeze(1)
        self.lse = self.m + self.log_s
        self.entropy = torch.where(self.none, 0.0, self.log_s + self.away)
        at = self.t.where(self.real, torch.zeros_like(self.t)).view(-1, 1)
        self.z_token = z.gather(1, at).squeeze(1)
        self.logp = torch.where(self.real, self.z_token - self.log_s, 0.0)
        self.logp[self.real & self.none] = -math.inf
        # relative error of s: of its exponentials (argument off by 3 U, then the
        # hardware's error), its sum in a thread and ten joins of two factors each
        self.rel = 3 * U * self.away + EXP2 + (V / 256 + 64) * U + 10 * (2 * EXP2 + 4 * U)

    def _finite(self, name, got, want, bound):
        got = d(got)
        same = torch.isfinite(want)
        assert torch.equal(got[~same], want[~same]), name
        check(name, got[same], want[same], bound.expand_as(want)[same])

    def check_forward(self, logp, entropy, lse):
        ls = self.log_s.masked_fill(self.none, 0).abs()
        zt = self.z_token.masked_fill(~torch.isfinite(self.z_token), 0).abs()
        self._finite("lse", lse, self.lse, self.rel + 4 * U * (ls + self.m.abs()))
        self._finite("logp", logp, self.logp, self.rel + 4 * U * (ls + zt))
        self._finite("entropy", entropy, self.entropy, self.rel * (1 + 2 * self.away) + 6 * U * (ls + self.away))

    def check_top(self, k, top_logp, top_tokens):
        place = torch.sort(self.raw, dim=1, descending=True, stable=True).indices
        value = self.x.gather(1, place)
        assert torch.equal(top_tokens.cpu(), place[:, :k]), "top_tokens"
        # from the maximum: next to a logit of -3.4e38 float64 keeps no digit of log s
        want = (value[:, :k] - self.top) * self.scale - self.log_s.masked_fill(self.none, 0).view(-1, 1)
        ls = self.log_s.masked_fill(self.none, 0).abs().view(-1, 1)
        z = want.masked_fill(~torch.isfinite(want), 0).abs() + ls
        self._finite("top_logp", top_logp, want, self.rel.view(-1, 1) + 4 * U * (ls + z))

    def check_backward(self, dlogp, dentropy, entropy, lse, dlogits):
        """entropy and lse are the forward's float32 values, taken as given."""
        T, V = self.x.shape
        zero = torch.zeros(T, dtype=torch.float64)
        up = (d(dlogp) if dlogp is not None else zero).masked_fill(~self.real, 0).view(-1, 1)
        ue = (d(dentropy) if dentropy is not None else zero).view(-1, 1)
        h, l = d(entropy).view(-1, 1), d(lse).view(-1, 1)
        dead = self.none.view(-1, 1)
        z = (self.x * self.scale - l.masked_fill(dead, 0)).masked_fill(dead, -math.inf)
        p = z.exp()
        z = z.masked_fill(z == -math.inf, 0)
        hit = torch.zeros_like(p)
        hit[self.real, self.t[self.real]] = 1
        want = self.scale * (up * hit - p * (up + ue * (z + h)))
        want = want.masked_fill(dead, 0)
        size = up.abs() + (ue * h).abs() + (ue * z).abs()
        # the exponent's argument: x scale - lse rounds once at the size of the
        # larger of the two; then the constant and the product
        rel = U * (z.abs() * 3) + EXP2
        # an exponential below float32's normal range counts as 0: p is off by
        # up to 2^-126 (and a product with it by a subnormal step)
        p_off = p * (rel + 8 * U) + torch.where(p < 2.0 ** -125, 2.0 ** -126, 0.0)
        bound = self.scale * (p_off * size + 2 * U * (up * hit).abs()) + U * want.abs() + 2.0 ** -149
        check("dlogits", dlogits, want, 1.02 * bound + HALF[dlogits.dtype] * want.abs() + TINY[dlogits.dtype])


# ------------------------------------------------------------------- AdamW
def mix(x):
    x &= 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def dice(n, number, seed, step):
    """The random numbers of a tensor's elements, as the header's kernels take them."""
    key = mix(seed + 0x9E3779B9 * step) ^ mix(0x85EBCA77 * (number + 1))
    one, two = [], []
    for i in range(n):
        if i % 8 == 0:
            x = mix((i // 8 & 0xFFFFFFFF) ^ key ^ mix((i // 8) >> 32)) | 1
        else:
            x ^= (x << 13) & 0xFFFFFFFF
            x ^= x >> 17
            x = (x ^ (x << 5)) & 0xFFFFFFFF
        one.append(((x >> 16) + 0.5) / 65536)
        two.append(((x & 0xFFFF) + 0.5) / 65536)
    return torch.tensor(one, dtype=torch.float64), torch.tensor(two, dtype=torch.float64)


def _each(scale, n):
    return d(scale).repeat_interleave(128)[:n]


def avg_values(codes, scale):
    c = d(codes.reshape(-1))
    return c.sign() * (c / 127).square() * _each(scale, c.numel())


def sq_values(codes, scale):
    c = d(codes.reshape(-1))
    return (c / 255).pow(4) * _each(scale, c.numel())


def adamw(p, g, m, v, *, lr, betas, eps, weight_decay, step, grad_scale=1.0):
    """float64 (p, m, v) and the bounds of float32 ones."""
    b1, b2 = betas
    g = g * grad_scale
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g.square()
    em = 3 * U * ((b1 * m).abs() + ((1 - b1) * g).abs())
    ev = 5 * U * v1
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    root = (v1 / c2).sqrt() + eps
    update = lr / c1 * m1 / root
    p1 = p - lr * weight_decay * p - update
    # the root: half of v's error, the square root, its factor and the sum; its
    # reciprocal; two products
    ep = 3 * U * p.abs() + 1.01 * (update.abs() * (2.5 * U + EXP2 + 2 * U + 2 * U + EXP2 + 4 * U) + lr / c1 * em / root)
    return (p1, m1, v1), (ep + U * p1.abs(), em, ev)


def check_codes(name, codes, scale, want, off, power, most, random):
    """Codes of the values `want`, known up to `off`, rounded by `random`."""
    n = want.numel()
    c = d(codes.reshape(-1)).abs()
    blocks = torch.nn.functional.pad(want.abs(), (0, -n % 128)).view(-1, 128).amax(1).clamp(min=2.0 ** -126)
    offs = torch.nn.functional.pad(off, (0, -n % 128)).view(-1, 128).amax(1)
    check(f"{name} scale", scale, blocks, offs + U * blocks)
    at = want.abs() / _each(scale, n)
    # the place of the value, as the codes count: for the first moment the
    # scale's reciprocal (2 U) and two products; for the second the moment's root
    # (2 U) times the scale's reciprocal root (2 U and its factor, U), squared
    # (6 U twice and one more). Then the distance from the lower code and the
    # random number's product with the gap
    slack = (off / _each(scale, n) + 16 * U * at) * most ** power + 1e-30
    y = at * most ** power
    low = torch.floor(y.clamp(min=0).pow(1 / power) + 1e-9).clamp(0, most - 1)
    low = torch.where(low.pow(power) > y, low - 1, low).clamp(min=0)
    gap = (low + 1).pow(power) - low.pow(power)
    up = random * gap < y - low.pow(power)
    want_c = low + up
    if power == 4:
        # a float32 square vanishes below 2^-150: no moment of that size is held
        want_c = torch.where(want.abs() >= 2.0 ** -150, want_c.clamp(min=1), want_c)
    near = ((random * gap - (y - low.pow(power))).abs() <= slack + 4 * U * gap) | \
        ((y - low.pow(power)).abs() <= slack) | ((y - (low + 1).pow(power)).abs() <= slack)
    wrong = (c != want_c) & ~(near & ((c - want_c).abs() <= 1))
    assert not wrong.any(), f"{name}: {int(wrong.sum())} codes, first at {int(wrong.nonzero()[0])}: " \
                            f"{c[wrong][0]} for {want_c[wrong][0]}"
    # next to a code or to its random number either neighbour is right; such places are few
    assert (c != want_c).double().mean() < 0.01 or n < 1000, name
