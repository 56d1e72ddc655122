"""Host side of the block operators, without a GPU: the ABI, the buckets'
borders, what each entry refuses before anything is enqueued, the binding's
checks, and the build's list of sources. The pointers here are made up: every
call must come back before it would use them."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from block_ref import borders

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dyt_block.h")
CSRC = os.path.join(ROOT, "bwd_dyt_forward_amd", "csrc")
OK, INVALID, DTYPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def dyt():
    import __graft_entry__ as ge
    ge._ensure_built()
    import bwd_dyt_forward_amd as m
    return m


@pytest.fixture(scope="module")
def codes(dyt):
    """The status codes as the header of the library names them."""
    src = open(os.path.join(ROOT, "include", "dyt.h")).read()
    return {n: int(v) for n, v in re.findall(r"(DYT_(?:OK|ERR_[A-Z_]+))\s*=\s*(\d+)", src)}


def test_the_binding_declares_what_the_header_does(dyt):
    from bwd_dyt_forward_amd import _block
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(dyt_[a-z_]+)\s*\(", src))
    assert names == set(_block.SIGNATURES)
    for n in names:
        assert hasattr(dyt.block_lib, n)
    for n, (_, args) in _block.SIGNATURES.items():
        params = re.search(rf"\b{n}\s*\((.*?)\)", src, flags=re.S).group(1).strip()
        assert len(args) == (0 if params == "void" else params.count(",") + 1), n
    out = subprocess.run(["nm", "-D", "--defined-only", dyt.BLOCK_LIB_FILE], capture_output=True, text=True).stdout
    for n in names:
        assert re.search(rf"\bT {n}\b", out), n


def test_the_header_is_plain_c(tmp_path):
    c = tmp_path / "t.c"
    c.write_text('#include "dyt_block.h"\nint main(void) { return sizeof(dyt_attn_desc) != 296; }\n')
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(c),
                    "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0
    from bwd_dyt_forward_amd import _block
    assert _block._DESC.size == 296


def test_every_included_source_enters_the_build_id():
    from bwd_dyt_forward_amd import build
    known = {os.path.basename(p) for p in build.BLOCK_DEPENDS}
    todo = [os.path.basename(p) for p in build.BLOCK_SOURCES]
    seen = set()
    while todo:
        name = todo.pop()
        if name in seen:
            continue
        seen.add(name)
        path = os.path.join(CSRC, name)
        if not os.path.exists(path):
            path = os.path.join(ROOT, "include", name)
        todo += re.findall(r'#include "([^"]+)"', open(path).read())
    assert seen == known


@pytest.mark.parametrize("n,dist,bidi", [(32, 128, True), (32, 128, False), (4, 2, True), (2, 2, False), (128, 1024, True),
                                         (64, 256, False), (33, 100, False), (10, 1000, True), (127, 70, False)])
def test_borders(dyt, n, dist, bidi):
    assert dyt.dyt_attn_bucket_borders(n, dist, bidi) == borders(n, dist, bidi)


def test_borders_of_every_shape(dyt):
    for n in range(2, 129, 3):
        for bidi in (False, True):
            if bidi and (n % 2 or n < 4):
                continue
            half = (n // 2 if bidi else n) // 2
            for dist in {half + 1, half + 2, 2 * half + 1, 128, 999, 1024}:
                if half < dist <= 1024:
                    got = dyt.dyt_attn_bucket_borders(n, dist, bidi)
                    assert got == borders(n, dist, bidi), (n, dist, bidi)
                    # the last bucket starts no later than max_distance: what the
                    # kernels' tables by position are sized for
                    assert got[-1] <= dist


def test_borders_refused(dyt):
    out = (ctypes.c_int32 * 256)()
    f = dyt.block_lib.dyt_attn_bucket_borders
    for n, dist, bidi in ((1, 128, 0), (2, 128, 1), (129, 500, 0), (33, 128, 1), (32, 8, 1), (32, 16, 0), (32, 1025, 0),
                          (32, 0, 0), (32, -1, 0), (32, 128, 2)):
        assert f(n, dist, bidi, out) == 0, (n, dist, bidi)
    assert f(32, 128, 1, None) == 0
    with pytest.raises(ValueError):
        dyt.dyt_attn_bucket_borders(33, 128, True)


# --------------------------------------------------------------- layer norm
P = 1 << 20   # made-up addresses, far apart


def ln_fwd(dyt, **kw):
    a = dict(x=P << 8, ldx=0, gamma=P, beta=P + 4096, y=P << 9, ldy=0, mean=P << 10, rstd=(P << 10) + (1 << 20), M=16, N=64,
             eps=1e-5, xdt=BF16, pdt=F32)
    a.update(kw)
    return dyt.block_lib.dyt_ln_forward(*a.values(), None)


def ln_bwd(dyt, **kw):
    a = dict(x=P << 8, ldx=0, dy=P << 9, lddy=0, mean=P << 10, rstd=P << 11, gamma=P << 12, dx=P << 13, lddx=0,
             dgamma=P << 14, dbeta=P << 15, ws=P << 16, ws_bytes=1 << 24, M=16, N=64, xdt=BF16, pdt=F32)
    a.update(kw)
    return dyt.block_lib.dyt_ln_backward(*a.values(), None)


def test_layer_norm_refusals(dyt, codes):
    bad, mis = codes["DYT_ERR_INVALID_ARG"], codes["DYT_ERR_MISALIGNED"]
    for kw in (dict(x=None), dict(gamma=None), dict(beta=None), dict(y=None), dict(mean=None), dict(rstd=None),
               dict(M=-1), dict(N=-1), dict(N=1 << 31), dict(M=1 << 62), dict(ldx=63), dict(ldy=63), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=1 << 62), dict(y=P << 8), dict(y=(P << 8) + 128),
               dict(mean=(P << 8) + 64), dict(rstd=(P << 10) + 32)):
        assert ln_fwd(dyt, **kw) == bad, kw
    for kw in (dict(x=(P << 8) + 1), dict(gamma=P + 2), dict(mean=(P << 10) + 2)):
        assert ln_fwd(dyt, **kw) == mis, kw
    for kw in (dict(xdt=3), dict(pdt=-1)):
        assert ln_fwd(dyt, **kw) == codes["DYT_ERR_UNSUPPORTED_DTYPE"], kw
    assert ln_fwd(dyt, M=0, x=None, y=None) == OK and ln_fwd(dyt, N=0, gamma=None) == OK
    for kw in (dict(x=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(gamma=None), dict(dx=None),
               dict(dgamma=None), dict(dbeta=None), dict(lddy=5), dict(lddx=5), dict(dx=P << 8), dict(dx=P << 9),
               dict(dgamma=P << 15), dict(dx=P << 16)):
        assert ln_bwd(dyt, **kw) == bad, kw
    for kw in (dict(ws=None), dict(ws_bytes=100)):
        assert ln_bwd(dyt, **kw) == codes["DYT_ERR_WORKSPACE_TOO_SMALL"], kw
    for kw in (dict(ws=(P << 16) + 8), dict(dx=(P << 13) + 1), dict(dgamma=(P << 14) + 2)):
        assert ln_bwd(dyt, **kw) == mis, kw
    assert ln_bwd(dyt, N=0, dgamma=None) == OK


def test_layer_norm_workspace(dyt):
    for M, N in ((1, 1), (7, 64), (100000, 64), (1 << 26, 8), (32768, 4096), (10, 100000)):
        for xdt in (torch.float32, torch.bfloat16):
            n = dyt.dyt_ln_backward_workspace_size(M, N, xdt, torch.float32)
            assert 8 * N <= n <= 8 * (N + 32) * 1024 and n % 128 == 0
    assert dyt.dyt_ln_backward_workspace_size(0, 5, torch.float32, torch.float32) == 0
    assert dyt.dyt_ln_backward_workspace_size(-1, 5, torch.float32, torch.float32) == 0


# ---------------------------------------------------------------- attention
TENSORS = ("q", "k", "v", "o", "dout", "dq", "dk", "dv")


def desc(**kw):
    from bwd_dyt_forward_amd import _block
    a = dict(B=2, Sq=33, Sk=65, Hq=4, Hkv=2, D=64, lens=0, starts=0, table=0, dtype=BF16, table_dtype=F32, causal=0,
             bidirectional=0, buckets=0, distance=0, scale=0.125, reserved=0)
    strides = {t: kw.pop(t) for t in TENSORS if t in kw}
    a.update(kw)
    st = []
    for t in TENSORS:
        S, H = (a["Sk"], a["Hkv"]) if t in ("k", "v", "dk", "dv") else (a["Sq"], a["Hq"])
        st += strides.get(t, (S * H * a["D"], H * a["D"], a["D"]))
    return _block._DESC.pack(a["B"], a["Sq"], a["Sk"], a["Hq"], a["Hkv"], a["D"], *st, a["lens"], a["starts"], a["table"],
                             a["dtype"], a["table_dtype"], a["causal"], a["bidirectional"], a["buckets"], a["distance"],
                             a["scale"], a["reserved"])


AT = {t: (i + 1) << 32 for i, t in enumerate(TENSORS + ("stats", "dtable", "ws"))}


def fwd(dyt, d, n=1 << 31, **kw):
    p = dict(AT, **kw)
    return dyt.block_lib.dyt_attn_forward(d, p["q"], p["k"], p["v"], p["o"], p["stats"], p["ws"], n, None)


def bwd(dyt, d, n=1 << 31, **kw):
    p = dict(AT, **kw)
    return dyt.block_lib.dyt_attn_backward(d, p["q"], p["k"], p["v"], p["o"], p["dout"], p["stats"], p["dq"], p["dk"],
                                           p["dv"], p["dtable"], p["ws"], n, None)


def test_attention_descriptor_refusals(dyt, codes):
    bad = codes["DYT_ERR_INVALID_ARG"]
    table = dict(table=1 << 44, buckets=32, distance=128)
    for kw in (dict(B=-1), dict(Sq=-1), dict(Sk=-1), dict(Hq=-4), dict(Hkv=0), dict(Hkv=3), dict(D=0), dict(D=129),
               dict(causal=2), dict(bidirectional=2), dict(reserved=1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(Sk=(1 << 28) + 1), dict(Sq=1 << 28),
               dict(B=1 << 25), dict(Hq=1 << 21), dict(table, buckets=1), dict(table, buckets=130),
               dict(table, buckets=33, bidirectional=1), dict(table, distance=16), dict(table, distance=1025),
               dict(q=(-64, 64, 64)), dict(k=(1 << 60, 64, 64)), dict(v=(0, 1 << 60, 64))):
        assert fwd(dyt, desc(**kw)) == bad, kw
        assert bwd(dyt, desc(**kw)) == bad, kw
        assert dyt.block_lib.dyt_attn_forward_workspace_size(desc(**kw)) == 0 or "q" in kw or "k" in kw or "v" in kw
    for kw in (dict(dtype=3), dict(dtype=-1), dict(table, table_dtype=5)):
        assert fwd(dyt, desc(**kw)) == codes["DYT_ERR_UNSUPPORTED_DTYPE"], kw
        assert bwd(dyt, desc(**kw)) == codes["DYT_ERR_UNSUPPORTED_DTYPE"], kw
    assert fwd(dyt, None) == bad and bwd(dyt, None) == bad


def test_outputs_whose_elements_share_memory_are_refused(dyt, codes):
    bad = codes["DYT_ERR_INVALID_ARG"]
    assert fwd(dyt, desc(o=(0, 256, 64))) == bad            # one batch entry over the other
    assert fwd(dyt, desc(o=(33 * 256, 128, 64))) == bad     # positions overlap
    assert fwd(dyt, desc(o=(33 * 256, 256, 32))) == bad     # heads overlap
    for t in ("dq", "dk", "dv"):
        assert bwd(dyt, desc(**{t: (0, 256, 64)})) == bad, t
        assert bwd(dyt, desc(**{t: (1 << 20, 256, 0)})) == bad, t


def test_attention_pointer_refusals(dyt, codes):
    bad, mis, ws = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED", "WORKSPACE_TOO_SMALL"))
    table = dict(table=1 << 44, buckets=32, distance=128)
    for t in ("q", "k", "v", "o", "stats"):
        assert fwd(dyt, desc(), **{t: None}) == bad, t
    for t in TENSORS + ("stats",):
        assert bwd(dyt, desc(), **{t: None}) == bad, t
    assert bwd(dyt, desc(**table), dtable=None) == bad
    for t in ("q", "k", "v", "o"):
        assert fwd(dyt, desc(), **{t: AT[t] + 1}) == mis, t
    for t in TENSORS:
        assert bwd(dyt, desc(), **{t: AT[t] + 1}) == mis, t
    assert fwd(dyt, desc(), stats=AT["stats"] + 2) == mis
    assert fwd(dyt, desc(lens=2)) == mis and fwd(dyt, desc(starts=6)) == mis
    assert fwd(dyt, desc(**dict(table, table=(1 << 44) + 2))) == mis
    assert bwd(dyt, desc(**table), dtable=AT["dtable"] + 2) == mis
    # overlaps of what is written with anything else
    assert fwd(dyt, desc(), o=AT["q"]) == bad and fwd(dyt, desc(), o=AT["v"] + 128) == bad
    assert fwd(dyt, desc(), stats=AT["o"] + 256) == bad
    for t in ("dq", "dk", "dv"):
        for other in ("q", "k", "v", "o", "dout", "stats", "ws"):
            assert bwd(dyt, desc(), **{t: AT[other]}) == bad, (t, other)
    assert bwd(dyt, desc(), dk=AT["dv"]) == bad
    assert bwd(dyt, desc(**table), dtable=AT["dq"]) == bad
    # workspace
    need = dyt.block_lib.dyt_attn_backward_workspace_size(desc())
    assert need > 0
    assert bwd(dyt, desc(), n=255) == ws and bwd(dyt, desc(), ws=None) == ws
    assert bwd(dyt, desc(), ws=AT["ws"] + 8) == mis


def test_split_forward_needs_its_workspace(dyt, codes):
    one = desc(B=1, Sq=1, Sk=100000, Hq=8, Hkv=1, D=128)
    need = dyt.block_lib.dyt_attn_forward_workspace_size(one)
    assert need >= 2 * 8 * (128 + 2) * 4
    assert fwd(dyt, one, n=4096) == codes["DYT_ERR_WORKSPACE_TOO_SMALL"]
    assert fwd(dyt, one, ws=None, n=0) == codes["DYT_ERR_WORKSPACE_TOO_SMALL"]


def test_nothing_to_do_is_no_error(dyt):
    assert fwd(dyt, desc(B=0), q=None, k=None, v=None, o=None, stats=None) == OK
    assert fwd(dyt, desc(Sq=0), q=None, o=None, stats=None) == OK
    assert fwd(dyt, desc(Hq=0), q=None, o=None, stats=None) == OK
    assert bwd(dyt, desc(B=0), **{t: None for t in TENSORS}) == OK


def test_workspace_grows_with_the_problem_and_fits_any_alignment(dyt):
    sizes = dyt.block_lib.dyt_attn_backward_workspace_size
    for kw in (dict(), dict(Sk=4096, Sq=4096), dict(D=128, Hq=32, Hkv=1), dict(dtype=F32, Sk=2000)):
        n = sizes(desc(**kw))
        d0 = dict(B=2, Sq=33, Sk=65, Hq=4, Hkv=2, D=64)
        d0.update({k: v for k, v in kw.items() if k in d0})
        assert n >= 8 * d0["B"] * d0["Hq"] * d0["Sq"]


# ------------------------------------------------------------------ binding
def test_the_binding_refuses_host_tensors_and_wrong_shapes(dyt):
    x, g = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="device"):
        dyt.dyt_ln_forward(x, g, g)
    with pytest.raises(ValueError, match="device"):
        dyt.dyt_ln_forward_residual(x, x, g, g)
    with pytest.raises(ValueError, match="device"):
        dyt.dyt_ln_backward(x, x, torch.zeros(4), torch.zeros(4), g)
    with pytest.raises(ValueError):
        dyt.dyt_ln_backward_residual(x, x, None, torch.zeros(4), torch.zeros(4), g)
    q = torch.zeros(1, 2, 2, 16)
    with pytest.raises(ValueError, match="device"):
        dyt.dyt_attn_forward(q, q, q)
    with pytest.raises(ValueError, match="device"):
        dyt.dyt_attn_backward(q, q, q, q, q, torch.zeros(1, 2, 2))


# ---------------------------------------------------------- autograd wiring
def test_residual_wiring_and_attention_gradients_on_stand_ins(dyt, monkeypatch):
    """The kernels replaced by plain operations on CPU tensors: which gradient
    goes to which input, and that x and r do not share their gradient's memory."""
    from bwd_dyt_forward_amd import _block, block

    def fwd(x, r, g, b, eps):
        h = x + r
        return h, h * g + b, h.mean(1), h.mean(1)

    def bwd(h, dy, dres, mean, rstd, g):
        return dres + dy * g, (dy * h).sum(0), dy.sum(0)

    monkeypatch.setattr(_block, "dyt_ln_forward_residual", fwd)
    monkeypatch.setattr(_block, "dyt_ln_backward_residual", bwd)
    x, r = (torch.randn(4, 6, requires_grad=True) for _ in range(2))
    g, b = torch.randn(6, requires_grad=True), torch.zeros(6, requires_grad=True)
    for n in (1, 2):
        h, y = block.layer_norm_residual(x, r, g, b)
        (2 * h + 3 * y).sum().backward()
        assert torch.allclose(x.grad, n * (2 + 3 * g.detach()).expand(4, 6)) and torch.equal(x.grad, r.grad)
        assert x.grad.data_ptr() != r.grad.data_ptr()
    seen = {}

    def attn_fwd(q, k, v, *, table, **kw):
        seen.update(kw, strides=q.stride())
        return q * 2, q[..., 0]

    def attn_bwd(q, k, v, o, do, stats, *, table, **kw):
        assert do.stride(-1) == 1 and {**kw} == {n: seen[n] for n in kw}
        out = (do * 2, k * 0 + 3, v * 0 + 5)
        return out if table is None else (*out, table * 0 + 7)

    monkeypatch.setattr(_block, "dyt_attn_forward", attn_fwd)
    monkeypatch.setattr(_block, "dyt_attn_backward", attn_bwd)
    q, k, v = (torch.randn(1, 3, 2, 4, requires_grad=True) for _ in range(3))
    t = torch.randn(8, 2, requires_grad=True)
    for table in (None, t):
        q.grad = k.grad = v.grad = None
        block.attention(q, k, v, causal=True, table=table).sum().backward()
        assert (q.grad == 2).all() and (k.grad == 3).all() and (v.grad == 5).all()
    assert (t.grad == 7).all() and seen["causal"] is True
    block.attention(q.transpose(2, 3).contiguous().transpose(2, 3), k, v)
    assert seen["strides"][-1] == 1


def test_a_full_cache_refuses_more(dyt):
    c = dyt.KVCache(2, 5, 1, 4, torch.float32, "cpu")
    x = torch.ones(2, 3, 1, 4)
    assert c.append(x, x).tolist() == [0, 0] and c.length.tolist() == [3, 3]
    with pytest.raises(ValueError, match="no room"):
        c.append(x, x)
    assert c.append(x[:, :2], 2 * x[:, :2]).tolist() == [3, 3] and c.length.tolist() == [5, 5]
    assert (c.k == 1).all() and (c.v[:, 3:] == 2).all()
