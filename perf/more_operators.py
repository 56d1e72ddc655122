"""Measured cases of the operators around a decoder's blocks: root-mean-square
norm (plain, with the residual add in front, with an 8-bit output), embedding
lookup with its gradient, log probabilities of given tokens with entropy, top
alternatives and gradient, and an AdamW step over many tensors.

With ``own`` false, ``run`` computes them in their plain form: elementary
torch operations in float32, rounded once at the end. With ``own`` true it
makes the package's calls. ``exact`` computes the same outputs in float64.

A token outside [0, V) stands for a place that is padded or ignored: its
embedding is zero, its log probability is 0, and it takes part in no gradient.

8-bit optimizer states are held in blocks of 128 elements with a float32 scale
each, a, the block's largest absolute value (2^-126 at least). First moment: int8 codes c that
stand for a sign(c) (c / 127)^2. Second moment: uint8 codes c that stand for
a (c / 255)^4. A value between two codes goes to the upper one with the
probability of its place between them, for a random number that the seed, the
step, the tensor's number and the element's index give; the second moment's
code is at least 1 where the moment is not zero.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
STEP = 100
BLOCK = 128
E4M3_MOST = 448.0
SCALE_LEAST = 2.0 ** -126


# ------------------------------------------------------------------- cases
def _rms(name, M, N, dt, pdt="f32", res=False, train=True, q8=False, group=0):
    return dict(name=name, op="rms", M=M, N=N, dtype=dt, pdtype=pdt, residual=res, train=train, q8=q8, group=group)


def _embed(name, T, V, D, dt, wdt, gdt):
    return dict(name=name, op="embed", T=T, V=V, D=D, dtype=dt, wdtype=wdt, gdtype=gdt)


def _lp(name, T, V, dt, top=0, train=True, masked=False):
    return dict(name=name, op="logprob", T=T, V=V, dtype=dt, top=top, train=train, masked=masked)


def _adamw(name, dim, depth, vocab, dt, gdt, bits, master):
    return dict(name=name, op="adamw", dim=dim, depth=depth, vocab=vocab, dtype=dt, gdtype=gdt, bits=bits, master=master)


def listed():
    return [
        # one layer of a small float32 network: every launch counts
        _rms("rms_train_1024x64_f32", 1024, 64, "f32"),
        # the pre-norm step of a transformer block of 8 x 4096 tokens
        _rms("rms_res_train_32768x4096_bf16", 32768, 4096, "bf16", res=True),
        # the norm before an 8-bit projection, a batch of single tokens
        _rms("rms_res_q8_64x8192_bf16", 64, 8192, "bf16", "bf16", res=True, train=False, q8=True),
        # a small decoder's training batch: few, often repeated tokens
        _embed("embed_train_1504x32x128_bf16", 1504, 32, 128, "bf16", "bf16", "bf16"),
        # a large vocabulary, 8 x 4096 tokens, float32 gradient
        _embed("embed_train_32768x128000x2048_bf16", 32768, 128000, 2048, "bf16", "bf16", "f32"),
        # the same small decoder's loss
        _lp("logprob_train_1504x32_f32", 1504, 32, "f32"),
        # one new token each for four requests, part of the vocabulary masked, with alternatives
        _lp("logprob_token_4x128000_bf16", 4, 128000, "bf16", top=20, train=False, masked=True),
        # scores of a prompt's tokens
        _lp("logprob_prompt_2048x100003_f16", 2048, 100003, "f16", top=5, train=False),
        # the loss of 2 x 4096 tokens over a vocabulary of odd size
        _lp("logprob_train_8192x50257_bf16", 8192, 50257, "bf16"),
        # a small decoder's parameters: some twenty tensors, a few hundred thousand elements
        _adamw("adamw32_128x2_f32", 128, 2, 32, "f32", "f32", 32, False),
        # bfloat16 parameters with float32 masters and states
        _adamw("adamw32_2048x4_bf16", 2048, 4, 32000, "bf16", "bf16", 32, True),
        # the same parameters, states in 8 bits
        _adamw("adamw8_2048x4_bf16", 2048, 4, 32000, "bf16", "bf16", 8, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dt = rng.choice(["f32", "bf16", "bf16", "f16"])
    op = rng.choice(["rms", "rms", "embed", "logprob", "logprob", "adamw"])
    if op == "rms":
        N = _log_int(rng, 8, 40000)
        M = max(1, _log_int(rng, 1 << 12, 1 << 26) // N)
        q8 = rng.random() < 0.4
        c = _rms("", M, N, dt, rng.choice(["f32", dt]), rng.random() < 0.5, not q8 and rng.random() < 0.8, q8,
                 rng.choice([0, 32, 64, 128]) if q8 else 0)
    elif op == "embed":
        D = _log_int(rng, 8, 8192)
        V = min(_log_int(rng, 16, 200000), (1 << 28) // D)
        T = min(_log_int(rng, 1, 200000), (1 << 26) // D)
        c = _embed("", T, V, D, dt, rng.choice([dt, "f32"]), rng.choice([dt, "f32"]))
    elif op == "logprob":
        V = _log_int(rng, 16, 200000)
        T = max(1, min(_log_int(rng, 1, 20000), (1 << 27) // V))
        train = rng.random() < 0.5
        c = _lp("", T, V, dt, 0 if train else rng.choice([0, 1, 5, 16]), train, rng.random() < 0.3)
    else:
        dim = _log_int(rng, 30, 2000)
        depth = rng.randint(1, 8)
        while depth * 12 * dim * dim > 3 << 26:
            depth -= 1
        bits = rng.choice([8, 32])
        c = _adamw("", dim, depth, min(_log_int(rng, 30, 50000), (1 << 25) // dim), dt, rng.choice([dt, "f32"]), bits,
                   dt != "f32" and rng.random() < 0.5)
    del c["name"]
    return c


def _shapes(c):
    """The parameters of a decoder: embedding, blocks, last norm and head."""
    n = c["dim"]
    block = [n, (3 * n, n), (n, n), n, (4 * n, n), 4 * n, (n, 4 * n), n]
    sizes = [(c["vocab"], n)] + block * c["depth"] + [n, (c["vocab"], n)]
    return [s if isinstance(s, int) else s[0] * s[1] for s in sizes]


def _places(c):
    """Offsets of the parameters in one flat buffer, and its length."""
    at, places = 0, []
    for n in _shapes(c):
        places.append(at)
        at += -(-n // BLOCK) * BLOCK
    return places, at


def work(case):
    c = case
    s = SIZE[c["dtype"]]
    if c["op"] == "rms":
        MN, p = c["M"] * c["N"], SIZE[c["pdtype"]]
        fwd = (3 if c["residual"] else 1) * MN * s + MN * (1 if c["q8"] else s) + c["N"] * p
        if c["q8"]:
            fwd += 4 * c["M"] * (-(-c["N"] // c["group"]) if c["group"] else 1)
        else:
            fwd += 4 * c["M"]
        bwd = (3 if c["residual"] else 2) * MN * s + c["N"] * p if c["train"] else 0
        return {"bytes": fwd + bwd, "flops": MN * (6 + (10 if c["train"] else 0))}
    if c["op"] == "embed":
        T, V, D = c["T"], c["V"], c["D"]
        rows = min(T, V)
        return {"bytes": 8 * T + rows * D * SIZE[c["wdtype"]] + 2 * T * D * s + V * D * SIZE[c["gdtype"]],
                "flops": 2 * T * D}
    if c["op"] == "logprob":
        TV = c["T"] * c["V"]
        n = TV * s * (2 if c["train"] else 1) + c["T"] * (20 + 12 * c["top"])
        return {"bytes": n, "flops": TV * (6 + (6 if c["train"] else 0))}
    n = sum(_shapes(c))
    each = 2 * s + SIZE[c["gdtype"]] + (8 if c["master"] else 0)
    if c["master"]:
        each -= s   # the parameter is written only
    # states: read and written; 8 bits also as the values they stand for
    each += 16 if c["bits"] == 32 else 4 + 16 / BLOCK + 4
    return {"bytes": n * each, "flops": 16 * n}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0, dtype=None):
        t = torch.randn(*shape, device="cuda", generator=g)
        return t.mul_(scale).add_(shift).to(dtype or DTYPES[c["dtype"]])

    def tokens(T, V, ignored):
        """Frequent tokens have low numbers; some places are ignored."""
        u = torch.rand(T, device="cuda", generator=g, dtype=torch.float64)
        t = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
        return torch.where(torch.rand(T, device="cuda", generator=g) < ignored, -1, t)

    st = {"case": c}
    if c["op"] == "rms":
        M, N = c["M"], c["N"]
        st["x"], st["gamma"] = normal(M, N, scale=1.5, shift=0.3), normal(N, scale=0.1, shift=1.0, dtype=DTYPES[c["pdtype"]])
        st["x"][:, ::61] *= 8  # a residual stream's few large columns
        if c["residual"]:
            st["r"] = normal(M, N)
        if c["train"]:
            st["dy"] = normal(M, N)
            if c["residual"]:
                st["dres"] = normal(M, N)
    elif c["op"] == "embed":
        st["weight"] = normal(c["V"], c["D"], scale=0.02, dtype=DTYPES[c["wdtype"]])
        st["tokens"] = tokens(c["T"], c["V"], 0.03)
        st["dy"] = normal(c["T"], c["D"])
    elif c["op"] == "logprob":
        T, V = c["T"], c["V"]
        st["logits"] = normal(T, V, scale=2.5)
        st["tokens"] = tokens(T, V, 0.05 if c["train"] else 0.0)
        likely = st["tokens"].clamp(min=0).view(-1, 1)
        up = torch.rand(T, 1, device="cuda", generator=g) * 15
        st["logits"].scatter_(1, likely, up.to(DTYPES[c["dtype"]]))   # what a model expects is often right
        if c["masked"]:
            hidden = torch.rand(V, device="cuda", generator=g) < 0.3
            st["logits"].masked_fill_(hidden, -math.inf)
            st["logits"].scatter_(1, likely, up.to(DTYPES[c["dtype"]]))
        st["scale"] = 1.0 if c["train"] else 1.25   # a temperature of 0.8
        if c["train"]:
            st["dlogp"] = normal(T, dtype=torch.float32, shift=-1.0)
            st["dentropy"] = normal(T, scale=0.05, dtype=torch.float32)
    else:
        places, n = _places(c)
        size = torch.exp(torch.randn(n, device="cuda", generator=g))
        grad = torch.randn(n, device="cuda", generator=g).mul_(size).mul_(1e-3)
        avg = torch.randn(n, device="cuda", generator=g).mul_(size).mul_(3e-4)
        sq = size.mul_(1e-3).square_().mul_(torch.rand(n, device="cuda", generator=g) + 0.5)
        master = torch.randn(n, device="cuda", generator=g).mul_(0.02)
        gaps = torch.ones(n, dtype=torch.bool, device="cuda")
        for at, k in zip(places, _shapes(c)):
            gaps[at:at + k] = False
        for t in (grad, avg, sq, master):
            t.masked_fill_(gaps, 0.0)
        st["param"], st["grad"] = master.to(DTYPES[c["dtype"]]), grad.to(DTYPES[c["gdtype"]])
        if c["master"]:
            st["master"] = master
        if c["bits"] == 32:
            st["avg"], st["sq"] = avg, sq
        else:
            half = torch.full((), 0.5, device="cuda")
            st["avg"], st["avg_scale"] = _encode_avg(avg, half)
            st["sq"], st["sq_scale"] = _encode_sq(sq, half)
        st["seed"] = seed & 0xFFFF
        # the parameters as their program has them: slices of the flat buffers
        for name in ("param", "grad", "master", "avg", "sq"):
            if name in st:
                st[name + "s"] = [st[name][a:a + k] for a, k in zip(places, _shapes(c))]
        if c["bits"] == 8:
            for name in ("avg_scale", "sq_scale"):
                st[name + "s"] = [st[name][a // BLOCK:a // BLOCK - (-k // BLOCK)] for a, k in zip(places, _shapes(c))]
    return st


# --------------------------------------------------------------------- run
def run(state):
    c = state["case"]
    if own:
        return {"rms": _own_rms, "embed": _own_embed, "logprob": _own_logprob, "adamw": _own_adamw}[c["op"]](c, state)
    return {"rms": _plain_rms, "embed": _plain_embed, "logprob": _plain_logprob, "adamw": _plain_adamw}[c["op"]](c, state)


def _own_rms(c, s):
    import bwd_dyt_forward_amd as dyt
    out = {}
    if c["q8"]:
        if c["residual"]:
            out["h"], out["q"], out["scales"] = dyt.dyt_rms_forward_residual_q8(s["x"], s["r"], s["gamma"], EPS, group=c["group"])
        else:
            out["q"], out["scales"] = dyt.dyt_rms_forward_q8(s["x"], s["gamma"], EPS, group=c["group"])
        return out
    if c["residual"]:
        out["h"], out["y"], rstd = dyt.dyt_rms_forward_residual(s["x"], s["r"], s["gamma"], EPS)
    else:
        out["y"], rstd = dyt.dyt_rms_forward(s["x"], s["gamma"], EPS)
    if not c["train"]:
        out["rstd"] = rstd
    elif c["residual"]:
        out["dx"], out["dgamma"] = dyt.dyt_rms_backward_residual(out["h"], s["dy"], s["dres"], rstd, s["gamma"])
    else:
        out["dx"], out["dgamma"] = dyt.dyt_rms_backward(s["x"], s["dy"], rstd, s["gamma"])
    return out


def _own_embed(c, s):
    import bwd_dyt_forward_amd as dyt
    scale = math.sqrt(c["D"])
    return {"y": dyt.dyt_embed_forward(s["weight"], s["tokens"], scale, dtype=DTYPES[c["dtype"]]),
            "dweight": dyt.dyt_embed_backward(s["dy"], s["tokens"], c["V"], scale, dtype=DTYPES[c["gdtype"]])}


def _own_logprob(c, s):
    import bwd_dyt_forward_amd as dyt
    got = dyt.dyt_logprob_forward(s["logits"], s["tokens"], scale=s["scale"], top=c["top"])
    out = dict(zip(("logp", "entropy", "lse", "top_logp", "top_tokens"), got))
    if c["train"]:
        out["dlogits"] = dyt.dyt_logprob_backward(s["logits"], s["tokens"], out["entropy"], out["lse"], s["dlogp"],
                                                  s["dentropy"], scale=s["scale"])
    return out


def _own_adamw(c, s):
    import bwd_dyt_forward_amd as dyt
    kw = dict(lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY, step=STEP, masters=s.get("masters"))
    out = {"param": s["param"]}
    if c["master"]:
        out["master"] = s["master"]
    if c["bits"] == 32:
        dyt.dyt_adamw_step(s["params"], s["grads"], s["avgs"], s["sqs"], **kw)
        out.update(avg=s["avg"], sq=s["sq"])
    else:
        dyt.dyt_adamw_step(s["params"], s["grads"], s["avgs"], s["sqs"], avg_scales=s["avg_scales"],
                           sq_scales=s["sq_scales"], seed=s["seed"], **kw)
        out["avg"], out["sq"] = dyt.dyt_adamw_values([s["avg"], s["sq"]], [s["avg_scale"], s["sq_scale"]],
                                                     dtype=torch.bfloat16)
    return out


def _plain_rms(c, s):
    dt, p = DTYPES[c["dtype"]], DTYPES[c["pdtype"]]
    out = {}
    if c["residual"]:
        out["h"] = (s["x"].float() + s["r"].float()).to(dt)
        x = out["h"].float()
    else:
        x = s["x"].float()
    rstd = (x * x).mean(1, keepdim=True).add(EPS).rsqrt()
    n = x * rstd
    gamma = s["gamma"].float()
    y = n * gamma
    if c["q8"]:
        G = c["group"] or c["N"]
        pad = -c["N"] % G
        y = torch.nn.functional.pad(y, (0, pad)).view(c["M"], -1, G)
        scales = (y.abs().amax(2) / E4M3_MOST).clamp(min=SCALE_LEAST)
        q = (y / scales.unsqueeze(2)).to(torch.float8_e4m3fn)
        out["q"], out["scales"] = q.view(c["M"], -1)[:, :c["N"]].contiguous(), scales
        return out
    out["y"] = y.to(dt)
    if not c["train"]:
        out["rstd"] = rstd.squeeze(1)
        return out
    dy = s["dy"].float()
    d = dy * gamma
    dx = rstd * (d - n * (d * n).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + s["dres"].float()
    out["dx"] = dx.to(dt)
    out["dgamma"] = (dy * n).sum(0).to(p)
    return out


def _plain_embed(c, s):
    scale = math.sqrt(c["D"])
    real = (s["tokens"] >= 0) & (s["tokens"] < c["V"])
    at = torch.where(real, s["tokens"], 0)
    keep = real.view(-1, 1)
    y = torch.where(keep, s["weight"][at].float() * scale, 0.0).to(DTYPES[c["dtype"]])
    d = torch.zeros(c["V"], c["D"], device="cuda")
    d.index_add_(0, at, torch.where(keep, s["dy"].float(), 0.0))
    return {"y": y, "dweight": d.mul_(scale).to(DTYPES[c["gdtype"]])}


def _plain_logprob(c, s):
    T, V = c["T"], c["V"]
    x = s["logits"].float()
    real = (s["tokens"] >= 0) & (s["tokens"] < V)
    at = torch.where(real, s["tokens"], 0).view(-1, 1)
    z = x * s["scale"]
    m = z.amax(1, keepdim=True)
    z = z - m
    e = z.exp()
    total = e.sum(1, keepdim=True)
    z = z.masked_fill(z == -math.inf, 0.0)
    log_total = total.log()
    entropy = log_total - (e * z).sum(1, keepdim=True) / total
    logp = (x.gather(1, at) * s["scale"] - m - log_total).squeeze(1)
    out = {"logp": torch.where(real, logp, 0.0), "entropy": entropy.squeeze(1), "lse": (m + log_total).squeeze(1)}
    if c["top"]:
        # the order of the values, then of the places from the first on, as one whole number
        bits = (x + 0.0).view(torch.int32).long()   # no negative zeros
        order = torch.where(bits < 0, ~bits & 0x7FFFFFFF, bits | 0x80000000)
        key = order * (1 << 31) + (V - 1 - torch.arange(V, device="cuda"))
        best = key.topk(c["top"], dim=1).values
        out["top_tokens"] = V - 1 - best % (1 << 31)
        out["top_logp"] = x.gather(1, out["top_tokens"]) * s["scale"] - m - log_total
    if c["train"]:
        p = e / total
        d = -p * (s["dlogp"].masked_fill(~real, 0.0).view(-1, 1) + s["dentropy"].view(-1, 1) * (z - log_total + entropy))
        d.scatter_add_(1, at, torch.where(real, s["dlogp"], 0.0).view(-1, 1))
        out["dlogits"] = (d * s["scale"]).to(DTYPES[c["dtype"]])
    return out


# -------------------------------------------------------- 8-bit states' plain form
def _mix(x):
    """A 32-bit hash (the finalizer of a published one: Appleby, 2011)."""
    x = x & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _dice(n, tensor, seed, step):
    """Two random numbers in (0, 1) for each of a tensor's n elements: the
    first element of each 8 has a hash of its index, the next ones go on from
    there (xorshift: Marsaglia, 2003); 16 bits for each number."""
    key = _mix(torch.tensor(seed + 0x9E3779B9 * step)) ^ _mix(torch.tensor(0x85EBCA77 * (tensor + 1)))
    first = torch.arange(-(-n // 8), device="cuda")
    x = _mix((first & 0xFFFFFFFF) ^ key.item() ^ _mix(first >> 32)) | 1
    every = [x]
    for _ in range(7):
        x = (x ^ (x << 13)) & 0xFFFFFFFF
        x = x ^ (x >> 17)
        x = (x ^ (x << 5)) & 0xFFFFFFFF
        every.append(x)
    x = torch.stack(every, 1).view(-1)[:n]
    return ((x >> 16).float() + 0.5) * 2.0 ** -16, ((x & 0xFFFF).float() + 0.5) * 2.0 ** -16


def _blocks(t):
    return torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)).view(-1, BLOCK)


def _encode_avg(avg, dice):
    a = _blocks(avg).abs().amax(1).clamp(min=SCALE_LEAST)
    y = (_blocks(avg).abs() / a.unsqueeze(1) * 127.0 ** 2).view(-1)[:avg.numel()]
    low = y.sqrt().floor().clamp(max=126)
    code = low + (dice * (2 * low + 1) < y - low * low)
    return (code * avg.sign()).to(torch.int8), a


def _encode_sq(sq, dice):
    a = _blocks(sq).amax(1).clamp(min=SCALE_LEAST)
    y = (_blocks(sq) / a.unsqueeze(1) * 255.0 ** 4).view(-1)[:sq.numel()]
    low = y.sqrt().sqrt().floor().clamp(max=254)
    code = low + (dice * (((4 * low + 6) * low + 4) * low + 1) < y - (low * low).square())
    return torch.where(sq > 0, code.clamp(min=1), code).to(torch.uint8), a


def _decode_avg(code, a):
    c = code.float()
    return (_blocks(c * c.abs() / 127.0 ** 2) * a.unsqueeze(1)).view(-1)[:code.numel()]


def _decode_sq(code, a):
    c = code.float().square().square()
    return (_blocks(c / 255.0 ** 4) * a.unsqueeze(1)).view(-1)[:code.numel()]


def _plain_adamw(c, s):
    c1, c2 = 1 - BETA1 ** STEP, 1 - BETA2 ** STEP
    for i, (param, grad) in enumerate(zip(s["params"], s["grads"])):
        g = grad.float()
        avg, sq = s["avgs"][i], s["sqs"][i]
        if c["bits"] == 8:
            m, v = _decode_avg(avg, s["avg_scales"][i]), _decode_sq(sq, s["sq_scales"][i])
        else:
            m, v = avg, sq
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + g * g * (1 - BETA2)
        p = s["masters"][i] if c["master"] else param.float()
        p = p * (1 - LR * DECAY) - (LR / c1) * m / ((v / c2).sqrt() + ADAM_EPS)
        if c["master"]:
            s["masters"][i].copy_(p)
        param.copy_(p)
        if c["bits"] == 8:
            one, two = _dice(g.numel(), i, s["seed"], STEP)
            for t, new in zip((avg, s["avg_scales"][i]), _encode_avg(m, one)):
                t.copy_(new)
            for t, new in zip((sq, s["sq_scales"][i]), _encode_sq(v, two)):
                t.copy_(new)
        else:
            avg.copy_(m)
            sq.copy_(v)
    out = {"param": s["param"], "avg": s["avg"], "sq": s["sq"]}
    if c["master"]:
        out["master"] = s["master"]
    if c["bits"] == 8:
        out["avg"] = _decode_avg(s["avg"], s["avg_scale"]).bfloat16()
        out["sq"] = _decode_sq(s["sq"], s["sq_scale"]).bfloat16()
    return out


# ------------------------------------------------------------------- exact
def _nearest_e4m3(y):
    """y, of at most 448, to the nearest of the values with four significant
    bits from 2^-6 on and of the multiples of 2^-9 below; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_codes(values, dice, power, most, least):
    """Codes of one block a row, by the place between the two codes around."""
    a = values.amax(1, keepdim=True).clamp(min=SCALE_LEAST)
    at = values / a
    low = torch.floor(at.pow(1.0 / power) * most).clamp(0, most - 1)
    lower, upper = (low / most).pow(power), ((low + 1) / most).pow(power)
    code = torch.where(dice < (at - lower) / (upper - lower), low + 1, low)
    code = torch.where(values > 0, code.clamp(min=least), 0.0)
    return (code / most).pow(power) * a


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rms":
        x = s["x"].double()
        out = {}
        if c["residual"]:
            x = x + s["r"].double()
            out["h"] = x
            x = x.to(DTYPES[c["dtype"]]).double()  # the norm's input is h as stored
        inv = 1.0 / torch.sqrt((x * x).sum(1, keepdim=True) / c["N"] + EPS)
        gamma = s["gamma"].double()
        n = x * inv
        if c["q8"]:
            parts = (n * gamma).split(c["group"] or c["N"], dim=1)
            scales = [(t.abs().max(1, keepdim=True).values / E4M3_MOST).clamp(min=SCALE_LEAST) for t in parts]
            out["q"] = torch.cat([_nearest_e4m3(t / a) for t, a in zip(parts, scales)], 1)
            out["scales"] = torch.cat(scales, 1)
            return out
        out["y"] = n * gamma
        if not c["train"]:
            out["rstd"] = inv[:, 0]
            return out
        dy = s["dy"].double()
        out["dgamma"] = (dy * n).sum(0)
        dn = dy * gamma
        dx = (dn - n * ((dn * n).sum(1, keepdim=True) / c["N"])) * inv
        out["dx"] = dx + (s["dres"].double() if c["residual"] else 0.0)
        return out
    if c["op"] == "embed":
        keep = (s["tokens"] >= 0).nonzero().squeeze(1)
        at = s["tokens"][keep]
        y = torch.zeros(c["T"], c["D"], device="cuda", dtype=torch.float64)
        y[keep] = s["weight"][at].double() * math.sqrt(c["D"])
        d = torch.zeros(c["V"], c["D"], device="cuda", dtype=torch.float64)
        d.index_put_((at,), s["dy"][keep].double(), accumulate=True)
        return {"y": y, "dweight": d * math.sqrt(c["D"])}
    if c["op"] == "logprob":
        parts = []
        for rows in torch.arange(c["T"], device="cuda").split(max(1, (1 << 26) // c["V"])):
            x, t = s["logits"][rows].double(), s["tokens"][rows]
            keep = (t >= 0).double()
            lse = torch.logsumexp(x * s["scale"], 1, keepdim=True)
            lp = x * s["scale"] - lse
            p = torch.exp(lp)
            lp0 = torch.where(p > 0, lp, 0.0)
            h = -(p * lp0).sum(1)
            got = {"logp": lp.gather(1, t.clamp(min=0).view(-1, 1)).squeeze(1) * keep, "entropy": h, "lse": lse.squeeze(1)}
            if c["top"]:
                value, place = torch.sort(x, dim=1, descending=True, stable=True)
                got["top_tokens"] = place[:, :c["top"]].contiguous()
                got["top_logp"] = value[:, :c["top"]] * s["scale"] - lse
            if c["train"]:
                up = (s["dlogp"][rows].double() * keep).view(-1, 1)
                hit = torch.zeros_like(p).scatter_(1, t.clamp(min=0).view(-1, 1), 1.0)
                got["dlogits"] = s["scale"] * (up * (hit - p) - s["dentropy"][rows].double().view(-1, 1) * p * (lp0 + h.view(-1, 1)))
                got["dlogits"] = torch.where(p > 0, got["dlogits"], 0.0)
            parts.append(got)
        return {k: torch.cat([g[k] for g in parts]) for k in parts[0]}
    n = s["param"].numel()
    out = {"param": s["param"].double()}
    if c["master"]:
        out["master"] = s["master"].double()
    out["avg"], out["sq"] = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    for i, (at, k) in enumerate(zip(_places(c)[0], _shapes(c))):
        g = s["grads"][i].double()
        if c["bits"] == 32:
            m, v = s["avgs"][i].double(), s["sqs"][i].double()
        else:
            cm, cv = s["avgs"][i].double(), s["sqs"][i].double()
            m = torch.sign(cm) * (cm / 127).square() * s["avg_scales"][i].double().repeat_interleave(BLOCK)[:k]
            v = (cv / 255).pow(4) * s["sq_scales"][i].double().repeat_interleave(BLOCK)[:k]
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g.square()
        p = s["masters"][i].double() if c["master"] else s["params"][i].double()
        mh, vh = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        p = p - LR * DECAY * p - LR * mh / (vh.sqrt() + ADAM_EPS)
        out["param"][at:at + k] = p
        if c["master"]:
            out["master"][at:at + k] = p
        if c["bits"] == 8:
            dice = [_blocks(t.double()) for t in _dice(k, i, s["seed"], STEP)]
            m = m.sign() * _exact_codes(_blocks(m).abs(), dice[0], 2, 127, 0).view(-1)[:k]
            v = _exact_codes(_blocks(v), dice[1], 4, 255, 1).view(-1)[:k]
        out["avg"][at:at + k], out["sq"][at:at + k] = m, v
    return out
