"""The AdamW step on the GPU against float64 (tests/lm_ref.py)."""
import math

import pytest
import torch

from block_ref import HALF, TINY, check, d
from lm_ref import U, adamw, avg_values, check_codes, dice, sq_values

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KW = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


class Tensors:
    """A list of parameters with gradients and states of a few steps."""

    def __init__(self, seed, sizes, dt, gdt, bits8=False, master=False, zero=False):
        g = torch.Generator().manual_seed(seed)
        r = lambda n: torch.randn(n, generator=g)
        self.bits8, self.sizes = bits8, sizes
        self.p = [r(n).to(dt).cuda() for n in sizes]
        self.g = [(r(n) * torch.exp(2 * r(n)) * 0.01).to(gdt).cuda() for n in sizes]
        self.master = [p.float() + (r(p.numel()) * 1e-3).cuda() for p in self.p] if master else None
        if bits8:
            blocks = [-(-n // 128) for n in sizes]
            self.m = [torch.randint(-127, 128, (n,), generator=g).to(torch.int8).cuda() for n in sizes]
            self.v = [torch.randint(0, 256, (n,), generator=g).to(torch.uint8).cuda() for n in sizes]
            self.sm = [(torch.rand(b, generator=g) * 0.03).cuda() for b in blocks]
            self.sv = [(torch.rand(b, generator=g) * 1e-3).cuda() for b in blocks]
        else:
            self.m = [(r(n) * 0.01).cuda() for n in sizes]
            self.v = [(r(n).square() * 1e-4).cuda() for n in sizes]
        if zero:
            for x in self.m + self.v + (self.sm + self.sv if bits8 else []):
                x.zero_()

    def all(self):
        return [t for x in (self.p, self.g, self.m, self.v, self.master, *((self.sm, self.sv) if self.bits8 else ()))
                if x is not None for t in x]

    def step(self, dyt, step=3, **kw):
        if self.bits8:
            kw.update(avg_scales=self.sm, sq_scales=self.sv)
        dyt.dyt_adamw_step(self.p, self.g, self.m, self.v, step=step, masters=self.master, **{**KW, **kw})

    def values(self):
        """float64 (p, m, v) of every tensor."""
        out = []
        for i, p in enumerate(self.master or self.p):
            m = avg_values(self.m[i], self.sm[i]) if self.bits8 else d(self.m[i])
            v = sq_values(self.v[i], self.sv[i]) if self.bits8 else d(self.v[i])
            out.append((d(p), m, v))
        return out

    def run(self, dyt, step=3, grad_scale=1.0, seed=None, **kw):
        """A step and its check."""
        before = self.values()
        more = {} if grad_scale == 1.0 else {"grad_scale": torch.tensor([grad_scale], device="cuda")}
        self.step(dyt, step, seed=seed, **more, **kw)
        for i, (p, m, v) in enumerate(before):
            want, off = adamw(p, d(self.g[i]), m, v, step=step, grad_scale=grad_scale, **{**KW, **kw})
            if self.master:
                check("master", self.master[i], want[0], off[0])
                assert torch.equal(self.p[i], self.master[i].to(self.p[i].dtype))
            else:
                h = HALF[self.p[i].dtype]
                check("param", self.p[i], want[0], off[0] + h * want[0].abs() + TINY[self.p[i].dtype])
            if self.bits8:
                n = p.numel()
                one, two = dice(n, i, seed, step) if seed is not None else (torch.full((n,), 0.5).double(),) * 2
                # the codes' values before the step, of which the betas keep a share: the
                # scale's factor and two products (4 U), or the root of the scale (2 U), its
                # factor (2 U) and a product, squared (5 U twice and one more)
                b1, b2 = {**KW, **kw}["betas"]
                check_codes("avg", self.m[i], self.sm[i], want[1], off[1] + 4 * U * b1 * m.abs(), 2, 127, one)
                assert ((d(self.m[i]) * want[1]) >= 0).all()
                check_codes("sq", self.v[i], self.sv[i], want[2], off[2] + 11 * U * b2 * v, 4, 255, two)
            else:
                check("avg", self.m[i], want[1], off[1] + U * want[1].abs())
                check("sq", self.v[i], want[2], off[2] + U * want[2].abs())


SIZES = [1, 2, 3, 4, 5, 7, 8, 9, 15, 127, 128, 129, 0, 1000, 1023, 2048, 4100, 8191, 8192, 8193, 20011]
TYPES = [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", False), ("bf16", "f32", True),
         ("f16", "f16", False), ("f16", "f16", True), ("f16", "f32", False), ("f16", "f32", True)]


@pytest.mark.parametrize("dt,gdt,master", TYPES)
@pytest.mark.parametrize("bits8", [False, True])
def test_sizes_and_types(dyt, dt, gdt, master, bits8):
    t = Tensors(1, SIZES, DTYPES[dt], DTYPES[gdt], bits8, master)
    t.run(dyt)
    t.run(dyt, step=4, grad_scale=0.25)
    t.run(dyt, step=1000, seed=7 if bits8 else None)


@pytest.mark.parametrize("bits8", [False, True])
def test_first_steps_from_zero_states(dyt, bits8):
    t = Tensors(2, [300, 5000], torch.float32, torch.float32, bits8, zero=True)
    t.g[0][100:] = 0
    for step in (1, 2, 3):
        t.run(dyt, step=step, seed=11 if bits8 else None)
    assert torch.isfinite(t.p[0]).all()


@pytest.mark.parametrize("kw", [dict(lr=0.0), dict(weight_decay=0.0), dict(betas=(0.0, 0.0)), dict(betas=(0.9, 0.9999)),
                                dict(eps=1e-3)])
def test_options(dyt, kw):
    Tensors(3, [257, 4000], torch.float32, torch.float32).run(dyt, **kw)
    Tensors(3, [257, 4000], torch.bfloat16, torch.bfloat16, True).run(dyt, seed=1, **kw)


@pytest.mark.parametrize("bits8", [False, True])
def test_many_tensors_of_all_kinds(dyt, bits8):
    """More than a launch's table, kinds mixed: as one call and one by one."""
    a, b = [], []
    for out in (a, b):
        for i in range(60):
            dt, gdt, master = TYPES[i % len(TYPES)]
            out.append(Tensors(i, [37 * i + 1, 9000], DTYPES[dt], DTYPES[gdt], bits8, master))
    cat = lambda ts, name: [x for t in ts for x in (getattr(t, name) or [None, None])]
    kw = dict(avg_scales=cat(a, "sm"), sq_scales=cat(a, "sv"), seed=None) if bits8 else {}
    dyt.dyt_adamw_step(cat(a, "p"), cat(a, "g"), cat(a, "m"), cat(a, "v"), step=5, masters=cat(a, "master"), **KW, **kw)
    for t in b:
        t.step(dyt, 5)
    for x, y in zip(a, b):
        assert all(torch.equal(p, q) for p, q in zip(x.all(), y.all()))


def test_unaligned_slices(dyt):
    """Tensors at every element offset of one buffer; their neighbours stay."""
    for dt, bits8 in (("f32", False), ("bf16", False), ("bf16", True), ("f32", True)):
        X = DTYPES[dt]
        ref = Tensors(8, [1000] * 7, X, X, bits8)
        t = Tensors(8, [1000] * 7, X, X, bits8)
        hold = []
        for name in ("p", "g", "m", "v"):
            x = getattr(t, name)
            buf = torch.full((7 * 1010,), 77, dtype=x[0].dtype, device="cuda")
            new = [buf[1001 * i + i + 1:1001 * i + i + 1001] for i in range(7)]
            for a, b in zip(new, x):
                a.copy_(b)
            setattr(t, name, new)
            hold.append(buf)
        t.step(dyt, seed=3)
        ref.step(dyt, seed=3)
        assert all(torch.equal(a, b) for a, b in zip(t.all(), ref.all()))
        assert all(int((b == 77).sum()) >= 70 for b in hold)


def test_random_rounding_keeps_the_mean(dyt):
    """Over 400 seeds the codes' mean value is the value: within five standard
    deviations of a step's two outcomes (half a step each at most)."""
    n, seeds = 2048, 400
    sums = [torch.zeros(n, dtype=torch.float64) for _ in range(2)]
    for seed in range(seeds):
        t = Tensors(9, [n], torch.float32, torch.float32, True)
        before = t.values()[0]
        t.step(dyt, seed=seed)
        sums[0] += avg_values(t.m[0], t.sm[0])
        sums[1] += sq_values(t.v[0], t.sv[0])
    want, off = adamw(*before[:1], d(t.g[0]), *before[1:], step=3, **KW)
    for k, (power, most, scale) in enumerate(((2, 127, t.sm[0]), (4, 255, t.sv[0]))):
        s = d(scale).repeat_interleave(128)
        low = ((want[k + 1].abs() / s).pow(1 / power) * most).floor()
        gap = ((low + 1) ** power - low ** power) / most ** power * s
        err = (sums[k] / seeds - want[k + 1]).abs()
        # (a second moment below the first code is rounded up to it)
        fine = (err <= 5 * 0.5 * gap / math.sqrt(seeds) + gap * 1e-3 + off[k + 1]) | ((power == 4) & (low == 0))
        assert fine.all(), (k, err[~fine] / gap[~fine])
        assert (low > 0).double().mean() > 0.5


def test_small_values_beside_large_ones(dyt):
    """A second moment never becomes zero where there was a gradient, and a
    moment's block keeps its scale down to 2^-126."""
    t = Tensors(10, [256], torch.float32, torch.float32, True, zero=True)
    t.g[0].fill_(1e-12)
    t.g[0][0] = 1.0
    t.g[0][128:] = 1e-25
    t.g[0][130] = 0.0
    t.run(dyt, step=1)
    assert (t.v[0][:128] > 0).all() and (t.sv[0] >= 2.0 ** -126).all() and t.v[0][130] == 0 and torch.isfinite(t.p[0]).all()


def test_nan_and_infinity_spoil_their_block_only(dyt):
    clean, t = (Tensors(12, [1024], torch.float32, torch.float32, True) for _ in range(2))
    t.g[0][130], t.g[0][700] = math.nan, math.inf
    t.step(dyt)
    clean.step(dyt)
    (v,), (c,) = t.values(), clean.values()
    assert math.isnan(v[0][130]) and math.isnan(v[0][700])
    bad = torch.zeros(1024, dtype=torch.bool)
    bad[[130, 700]] = True
    assert torch.equal(v[0][~bad], c[0][~bad])
    blocks = bad.view(-1, 128).any(1).repeat_interleave(128)
    for k in (1, 2):
        assert torch.equal(v[k][~blocks], c[k][~blocks]) and not torch.isfinite(v[k][bad]).any()
    t, clean = (Tensors(12, [1024], torch.float32, torch.float32) for _ in range(2))
    t.g[0][130] = math.nan
    t.step(dyt)
    clean.step(dyt)
    assert int(torch.isnan(t.p[0]).sum()) == int(torch.isnan(t.m[0]).sum()) == int(torch.isnan(t.v[0]).sum()) == 1


@pytest.mark.parametrize("bits8", [False, True])
def test_counter_and_rate_on_the_device_and_in_a_graph(dyt, bits8):
    a, b = (Tensors(14, [3000, 77], torch.bfloat16, torch.bfloat16, bits8, True) for _ in range(2))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.tensor([1e-2], device="cuda")
    gs = torch.tensor([1.0], device="cuda")

    def move():
        step.add_(1)
        a.step(dyt, step, lr=lr, grad_scale=gs, seed=5 if bits8 else None)

    move()
    b.step(dyt, 1, grad_scale=gs, seed=5 if bits8 else None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        move()
    for i in range(4):
        for t in (a, b):
            for k, g in enumerate(t.g):
                g.copy_(torch.randn(g.shape, generator=torch.Generator().manual_seed(i + k)).cuda() * 0.01)
        rate = 1e-2 / (i + 1)
        lr.fill_(rate)
        gs.fill_(1.0 / (i + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.step(dyt, i + 2, lr=lr.item(), grad_scale=gs, seed=5 if bits8 else None)
        for x, y in zip(a.master, b.master):
            # the corrections on the device and on the host may differ in their last bits
            assert ((x - y).abs() <= 2.0 ** -21 * (x.abs() + 20 * rate) * (i + 2)).all(), i
    assert step.item() == 5
    if not bits8:
        assert all(((x - y).abs() <= 1e-6 * y.abs()).all() for x, y in zip(a.m, b.m))


def test_values_of_codes(dyt):
    t = Tensors(15, [1, 100, 128, 129, 9000], torch.float32, torch.float32, True)
    for dt in DTYPES.values():
        got = dyt.dyt_adamw_values(t.m + t.v, t.sm + t.sv, dtype=dt)
        for x, (_, m, v) in zip(zip(got[:5], got[5:]), t.values()):
            for a, b in zip(x, (m, v)):
                check("values", a, b, HALF[dt] * b.abs() + 6 * U * b.abs() + TINY[dt])


def test_same_bits_every_time_and_on_another_stream(dyt):
    for bits8 in (False, True):
        a, b = (Tensors(16, [5000, 129], torch.float16, torch.float16, bits8) for _ in range(2))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        a.step(dyt, seed=2)
        b.step(dyt, seed=2, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(x, y) for x, y in zip(a.all(), b.all()))


def test_offsets_past_32_bits(dyt):
    """One tensor of over 2^32 elements: both ends."""
    n = (1 << 32) + 5000
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sm, sv = (torch.zeros(-(-n // 128), device="cuda") for _ in range(2))
    dyt.dyt_adamw_step([p], [g], [m], [v], step=1, lr=0.5, weight_decay=0.0, avg_scales=[sm], sq_scales=[sv], seed=1)
    # p = 1 - 0.5 m / sqrt(v) of the corrected moments, both 1
    assert p.min().item() == p.max().item() == 0.5
    assert m.min().item() == m.max().item() == 127 and v.min().item() == v.max().item() == 255
    assert sm.min().item() == sm.max().item()
