"""Host side of the decoder operators, without a GPU: the ABI, what each entry
refuses before anything is enqueued, the binding's checks, and the build's list
of sources. The pointers here are made up: every call must come back before it
would use them."""
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

from test_block_cpu import codes, dyt  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dyt_lm.h")
CSRC = os.path.join(ROOT, "bwd_dyt_forward_amd", "csrc")
OK, F32, BF16, F16 = 0, 0, 1, 2
P = 1 << 32   # made-up addresses, far apart
INF, NAN = float("inf"), float("nan")


def test_the_binding_declares_what_the_header_does(dyt):  # noqa: F811
    from bwd_dyt_forward_amd import _lm
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(dyt_[a-z0-9_]+)\s*\(", src))
    assert names == set(_lm.SIGNATURES)
    for n, (_, args) in _lm.SIGNATURES.items():
        params = re.search(rf"\b{n}\s*\((.*?)\)", src, flags=re.S).group(1).strip()
        assert len(args) == (0 if params == "void" else params.count(",") + 1), n
    out = subprocess.run(["nm", "-D", "--defined-only", dyt.LM_LIB_FILE], capture_output=True, text=True).stdout
    for n in names:
        assert re.search(rf"\bT {n}\b", out), n


def test_the_header_is_plain_c(tmp_path):
    from bwd_dyt_forward_amd import _lm
    c = tmp_path / "t.c"
    c.write_text('#include "dyt_lm.h"\nint main(void) { return sizeof(dyt_adamw_tensor) != %d || '
                 "sizeof(dyt_adamw_options) != %d || sizeof(dyt_adamw_codes) != %d; }\n"
                 % (_lm._ADAMW_TENSOR.size, _lm._ADAMW_OPTIONS.size, _lm._ADAMW_CODES.size))
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(c),
                    "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_every_included_source_enters_the_build_id():
    from bwd_dyt_forward_amd import build
    known = {os.path.basename(p) for p in build.LM_DEPENDS}
    todo = [os.path.basename(p) for p in build.LM_SOURCES]
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


def test_a_build_at_the_default_path_brings_the_library(monkeypatch):
    from bwd_dyt_forward_amd import build
    made = []
    monkeypatch.setattr(build, "_compile", lambda out, *a, **kw: made.append(out))
    build.build()
    assert build.LM_LIB_PATH in made


@pytest.mark.parametrize("state", ["missing", "other sources"])
def test_the_package_without_the_library(dyt, tmp_path, state):  # noqa: F811
    package = "bwd_dyt_forward_amd"
    os.mkdir(tmp_path / package)
    for name in os.listdir(os.path.join(ROOT, package)):
        if name.endswith((".py", ".so", ".json")) and name != "libdyt_lm.so" or name == "csrc":
            os.symlink(os.path.join(ROOT, package, name), tmp_path / package / name)
    os.remove(tmp_path / package / "build.py")
    shutil.copy(os.path.join(ROOT, package, "build.py"), tmp_path / package / "build.py")
    os.symlink(os.path.join(ROOT, "include"), tmp_path / "include")
    if state == "other sources":
        lib = open(dyt.LM_LIB_FILE, "rb").read()
        mark = lib.index(b"DYT_BUILD_ID=") + 13
        open(tmp_path / package / "libdyt_lm.so", "wb").write(lib[:mark] + b"0" * 16 + lib[mark + 16:])
    word = "not found" if state == "missing" else "other sources"
    code = f"""
import sys
sys.path.insert(0, {str(tmp_path)!r})
import {package} as m
from {package} import *
assert m.__file__.startswith({str(tmp_path)!r}) and DyT(8).num_features == 8 and LayerNorm(8).num_features == 8
for name in ("RMSNorm", "dyt_adamw_step", "lm_lib"):
    assert name not in globals()
    try:
        getattr(m, name)
    except ImportError as e:
        assert {word!r} in str(e), e
    else:
        raise SystemExit(name)
assert not hasattr(m, "no_such_name")
"""
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path)
    assert run.returncode == 0, run.stderr


# ---------------------------------------------------- root-mean-square norm
def rms_fwd(lib, **kw):
    a = dict(x=P, ldx=0, gamma=2 * P, y=3 * P, ldy=0, rstd=4 * P, M=16, N=64, eps=1e-5, xdt=BF16, pdt=F32)
    a.update(kw)
    return lib.dyt_rms_forward(*a.values(), None)


def rms_q8(lib, **kw):
    a = dict(x=P, ldx=0, r=5 * P, gamma=2 * P, h=6 * P, q=3 * P, scales=4 * P, M=16, N=64, group=32, eps=1e-5, xdt=BF16, pdt=F32)
    a.update(kw)
    return lib.dyt_rms_forward_q8(*a.values(), None)


def rms_bwd(lib, **kw):
    a = dict(x=P, ldx=0, dy=2 * P, lddy=0, rstd=3 * P, gamma=4 * P, dx=5 * P, lddx=0, dgamma=6 * P, ws=7 * P, ws_bytes=1 << 24,
             M=16, N=64, xdt=BF16, pdt=F32)
    a.update(kw)
    return lib.dyt_rms_backward(*a.values(), None)


def test_rms_refusals(dyt, codes):  # noqa: F811
    lib = dyt.lm_lib
    bad, mis, ws, dt = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED", "WORKSPACE_TOO_SMALL", "UNSUPPORTED_DTYPE"))
    for kw in (dict(x=None), dict(gamma=None), dict(y=None), dict(rstd=None), dict(M=-1), dict(N=-1), dict(N=1 << 31),
               dict(M=1 << 62), dict(ldx=63), dict(ldy=63), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(ldx=1 << 62),
               dict(y=P), dict(y=P + 128), dict(rstd=P + 64), dict(y=2 * P)):
        assert rms_fwd(lib, **kw) == bad, kw
    for kw in (dict(x=P + 1), dict(gamma=2 * P + 2), dict(rstd=4 * P + 2)):
        assert rms_fwd(lib, **kw) == mis, kw
    for kw in (dict(xdt=3), dict(pdt=-1)):
        assert rms_fwd(lib, **kw) == dt and rms_q8(lib, **kw) == dt and rms_bwd(lib, **kw) == dt, kw
    assert rms_fwd(lib, M=0, x=None, y=None) == OK and rms_fwd(lib, N=0, gamma=None) == OK
    for kw in (dict(group=16), dict(group=-1), dict(group=256), dict(r=None), dict(h=None), dict(q=None), dict(scales=None),
               dict(ldx=65), dict(q=P), dict(q=5 * P + 8), dict(h=P), dict(h=3 * P), dict(scales=3 * P + 1020), dict(eps=NAN)):
        assert rms_q8(lib, **kw) == bad, kw
    assert rms_q8(lib, scales=4 * P + 1) == mis and rms_q8(lib, h=6 * P + 1) == mis
    for kw in (dict(x=None), dict(dy=None), dict(rstd=None), dict(gamma=None), dict(dx=None), dict(dgamma=None),
               dict(lddy=5), dict(lddx=5), dict(dx=P), dict(dx=2 * P), dict(dx=7 * P), dict(dgamma=4 * P)):
        assert rms_bwd(lib, **kw) == bad, kw
    for kw in (dict(ws=None), dict(ws_bytes=100)):
        assert rms_bwd(lib, **kw) == ws, kw
    for kw in (dict(ws=7 * P + 8), dict(dx=5 * P + 1), dict(dgamma=6 * P + 2)):
        assert rms_bwd(lib, **kw) == mis, kw
    assert rms_bwd(lib, N=0, dgamma=None) == OK
    for M, N in ((1, 1), (7, 64), (100000, 64), (1 << 26, 8), (32768, 4096), (10, 100000)):
        for xdt in (torch.float32, torch.bfloat16):
            n = dyt.dyt_rms_backward_workspace_size(M, N, xdt, torch.float32)
            assert 4 * N <= n <= 4 * (N + 32) * 1024 and n % 128 == 0
    assert dyt.dyt_rms_backward_workspace_size(0, 5, torch.float32, torch.float32) == 0
    assert dyt.dyt_rms_backward_workspace_size(-1, 5, torch.float32, torch.float32) == 0


# --------------------------------------------------------------- embedding
def emb_fwd(lib, **kw):
    a = dict(w=P, ldw=0, t=2 * P, y=3 * P, ldy=0, T=50, V=100, D=64, scale=1.0, wdt=BF16, ydt=BF16, bits=64)
    a.update(kw)
    return lib.dyt_embed_forward(*a.values(), None)


def emb_bwd(lib, **kw):
    a = dict(dy=P, lddy=0, t=2 * P, dw=3 * P, lddw=0, ws=4 * P, n=1 << 24, T=50, V=100, D=64, scale=1.0, ydt=BF16, wdt=F32,
             bits=64, accumulate=0)
    a.update(kw)
    return lib.dyt_embed_backward(*a.values(), None)


def test_embedding_refusals(dyt, codes):  # noqa: F811
    lib = dyt.lm_lib
    bad, mis, ws, dt = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED", "WORKSPACE_TOO_SMALL", "UNSUPPORTED_DTYPE"))
    big = (dict(T=-1), dict(V=-1), dict(D=-1), dict(T=1 << 31), dict(V=1 << 31), dict(D=1 << 31), dict(bits=16),
           dict(scale=NAN), dict(scale=INF))
    for kw in (*big, dict(w=None), dict(t=None), dict(y=None), dict(ldw=63), dict(ldy=63), dict(y=P), dict(y=P + 12800 - 2),
               dict(y=2 * P + 8)):
        assert emb_fwd(lib, **kw) == bad, kw
    for kw in (*big, dict(dy=None), dict(t=None), dict(dw=None), dict(lddy=63), dict(lddw=63), dict(accumulate=2), dict(dw=P),
               dict(dw=2 * P), dict(ws=3 * P), dict(ws=P)):
        assert emb_bwd(lib, **kw) == bad, kw
    for kw in (dict(wdt=3), dict(ydt=-1)):
        assert emb_fwd(lib, **kw) == dt and emb_bwd(lib, **kw) == dt
    assert emb_fwd(lib, w=P + 1) == mis and emb_fwd(lib, t=2 * P + 4) == mis
    assert emb_bwd(lib, dw=3 * P + 2) == mis and emb_bwd(lib, ws=4 * P + 8) == mis
    for kw in (dict(ws=None), dict(n=400), dict(V=0x7ffffffe, T=0x7ffffffe), dict(T=0x7ffffffe, D=1 << 28)):
        assert emb_bwd(lib, **kw) == ws, kw
    assert emb_fwd(lib, T=0, t=None, y=None) == OK and emb_fwd(lib, D=0) == OK
    assert emb_bwd(lib, V=0, dw=None) == OK and emb_bwd(lib, T=0, accumulate=1) == OK
    for T, V, D in ((1, 1, 1), (1000, 50, 64), (100000, 300000, 8), (1 << 20, 10, 4096)):
        n = dyt.dyt_embed_backward_workspace_size(T, V, D)
        assert 16 * T <= n <= 16 * (T + 4) + 4 * 512 * (T // 16384 + 1) + 2 * 4 * D * (T // 16 + 1)
    assert dyt.dyt_embed_backward_workspace_size(-1, 5, 5) == 0


# ------------------------------------------------- token log probabilities
def lp_fwd(lib, **kw):
    a = dict(x=P, ld=0, t=2 * P, logp=3 * P, ent=4 * P, lse=5 * P, top_logp=6 * P, top_tokens=7 * P, ws=8 * P, n=1 << 24,
             T=50, V=100, scale=1.0, top=3, dt=BF16, bits=64)
    a.update(kw)
    return lib.dyt_logprob_forward(*a.values(), None)


def lp_bwd(lib, **kw):
    a = dict(x=P, ld=0, t=2 * P, ent=3 * P, lse=4 * P, dlogp=5 * P, dent=6 * P, dx=7 * P, ldd=0, T=50, V=100, scale=1.0, dt=BF16,
             bits=64)
    a.update(kw)
    return lib.dyt_logprob_backward(*a.values(), None)


def test_logprob_refusals(dyt, codes):  # noqa: F811
    lib = dyt.lm_lib
    bad, mis, ws, dt = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED", "WORKSPACE_TOO_SMALL", "UNSUPPORTED_DTYPE"))
    both = (dict(T=-1), dict(V=-1), dict(T=1 << 31), dict(V=(1 << 26) + 1), dict(V=0), dict(bits=16), dict(scale=0.0),
            dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(x=None), dict(t=None), dict(lse=None), dict(ent=None),
            dict(ld=99))
    for kw in (*both, dict(logp=None), dict(top=-1), dict(top=65), dict(V=2), dict(top=0), dict(top_logp=None),
               dict(top_tokens=None), dict(logp=P), dict(lse=4 * P + 4), dict(top_tokens=P + 16), dict(top_logp=7 * P + 8),
               dict(logp=2 * P)):
        assert lp_fwd(lib, **kw) == bad, kw
    for kw in (*both, dict(dx=None), dict(ldd=99), dict(dx=P + 2), dict(dx=P, ldd=101), dict(dx=4 * P), dict(dx=5 * P)):
        assert lp_bwd(lib, **kw) == bad, kw
    assert lp_fwd(lib, dt=3) == dt and lp_bwd(lib, dt=-1) == dt
    for kw in (dict(x=P + 1), dict(t=2 * P + 4), dict(logp=3 * P + 2), dict(top_tokens=7 * P + 4)):
        assert lp_fwd(lib, **kw) == mis, kw
    for kw in (dict(dx=7 * P + 1), dict(dlogp=5 * P + 2), dict(dent=6 * P + 1)):
        assert lp_bwd(lib, **kw) == mis, kw
    # few rows of many logits are cut into parts, which meet in the workspace
    few = dict(T=2, V=100000)
    need = dyt.dyt_logprob_forward_workspace_size(2, 100000, 3, torch.bfloat16)
    assert need > 0
    assert lp_fwd(lib, n=need - 1, **few) == ws and lp_fwd(lib, ws=None, **few) == ws
    assert lp_fwd(lib, ws=8 * P + 8, **few) == mis and lp_fwd(lib, ws=P, **few) == bad
    assert dyt.dyt_logprob_forward_workspace_size(5000, 100000, 0, torch.bfloat16) == 0
    assert dyt.dyt_logprob_forward_workspace_size(2, 100, 101, torch.bfloat16) == 0
    assert lp_fwd(lib, T=0, x=None) == OK and lp_bwd(lib, T=0, x=None) == OK


# ------------------------------------------------------------------- AdamW
def tensor(i=1, **kw):
    from bwd_dyt_forward_amd import _lm
    at = 16 * i * P
    a = dict(p=at, g=at + P, m=at + 2 * P, v=at + 3 * P, ma=0, va=0, master=0, n=1000, pdt=BF16, gdt=BF16)
    a.update(kw)
    return _lm._ADAMW_TENSOR.pack(*a.values())


def options(**kw):
    from bwd_dyt_forward_amd import _lm
    a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, decay=0.01, step=1, lr_dev=0, step_dev=0, gs=0, seed=0, seeded=0,
             bits=32, reserved=0)
    a.update(kw)
    return _lm._ADAMW_OPTIONS.pack(*a.values())


def test_adamw_refusals(dyt, codes):  # noqa: F811
    step = dyt.lm_lib.dyt_adamw_step
    bad, mis, dt = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED", "UNSUPPORTED_DTYPE"))
    o = options()
    assert step(None, 0, o, None) == OK and step(tensor(n=0, p=0), 1, o, None) == OK
    assert step(None, 1, o, None) == bad and step(tensor(), 1, None, None) == bad and step(tensor(), -1, o, None) == bad
    for kw in (dict(lr=-1.0), dict(lr=INF), dict(lr=NAN), dict(beta1=1.0), dict(beta2=1.0), dict(beta1=-0.1), dict(eps=-1.0),
               dict(eps=NAN), dict(decay=-1.0), dict(step=0), dict(step=-3), dict(seeded=2), dict(bits=16), dict(reserved=1)):
        assert step(tensor(n=0), 1, options(**kw), None) == bad, kw
    at = 16 * P
    for kw in (dict(p=0), dict(g=0), dict(m=0), dict(v=0), dict(n=-1), dict(n=(1 << 34) + 1), dict(ma=8 * P, va=9 * P),
               dict(pdt=F32, gdt=F32, master=8 * P), dict(m=at + 3 * P), dict(v=at + 1000), dict(g=at + 1998),
               dict(master=at + 2 * P + 3996)):
        assert step(tensor(**kw), 1, o, None) == bad, kw
    for kw in (dict(ma=8 * P, va=0), dict(), dict(ma=8 * P, va=8 * P + 28)):
        assert step(tensor(**kw), 1, options(bits=8), None) == bad, kw
    for kw in (dict(p=at + 1), dict(m=at + 2 * P + 2), dict(master=8 * P + 2)):
        assert step(tensor(**kw), 1, o, None) == mis, kw
    assert step(tensor(ma=8 * P + 2, va=9 * P), 1, options(bits=8), None) == mis
    assert step(tensor(n=0), 1, options(lr_dev=2), None) == mis and step(tensor(n=0), 1, options(step_dev=4), None) == mis
    for kw in (dict(pdt=3), dict(gdt=F16), dict(pdt=F32, gdt=BF16)):
        assert step(tensor(**kw), 1, o, None) == dt, kw
    # tensors that share what is written, or the device's numbers
    assert step(tensor(1) + tensor(1), 2, o, None) == bad
    assert step(tensor(1) + tensor(2, v=at + 1996), 2, o, None) == bad
    assert step(tensor(1) + tensor(2, g=at + 2 * P + 100), 2, o, None) == bad
    assert step(tensor(1), 1, options(lr_dev=at + 4), None) == bad


def test_adamw_values_refusals(dyt, codes):  # noqa: F811
    from bwd_dyt_forward_amd import _lm
    bad, mis, dt = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED", "UNSUPPORTED_DTYPE"))

    def call(vdt=BF16, count=1, **kw):
        a = dict(c=P, s=2 * P, v=3 * P, n=1000, second=0, reserved=0)
        a.update(kw)
        return dyt.lm_lib.dyt_adamw_values(_lm._ADAMW_CODES.pack(*a.values()), count, vdt, None)

    for kw in (dict(c=0), dict(s=0), dict(v=0), dict(n=-1), dict(second=2), dict(reserved=1), dict(v=P), dict(v=2 * P),
               dict(count=-1)):
        assert call(**kw) == bad, kw
    assert call(s=2 * P + 2) == mis and call(v=3 * P + 1) == mis and call(vdt=5) == dt and call(n=0, c=0) == OK


# ------------------------------------------------------------------ binding
def test_the_binding_refuses_host_tensors_and_wrong_arguments(dyt):  # noqa: F811
    x, g = torch.zeros(4, 8), torch.zeros(8)
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dyt.dyt_rms_forward(x, g), lambda: dyt.dyt_rms_forward_residual(x, x, g),
                 lambda: dyt.dyt_rms_forward_q8(x, g), lambda: dyt.dyt_rms_forward_residual_q8(x, x, g),
                 lambda: dyt.dyt_rms_backward(x, x, torch.zeros(4), g), lambda: dyt.dyt_embed_forward(x, t),
                 lambda: dyt.dyt_embed_backward(x, t, 9), lambda: dyt.dyt_logprob_forward(x, t),
                 lambda: dyt.dyt_logprob_backward(x, t, torch.zeros(4), torch.zeros(4)),
                 lambda: dyt.dyt_adamw_step([x], [x], [x], [x], lr=1e-3, step=1)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError):
        dyt.dyt_rms_backward_residual(x, x, None, torch.zeros(4), g)
    with pytest.raises(ValueError):
        dyt.dyt_rms_forward_residual_q8(x, None, g)
    with pytest.raises(ValueError, match="equal lengths"):
        dyt.dyt_adamw_step([x], [], [x], [x], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="scales"):
        dyt.dyt_adamw_step([x], [x], [x], [x], lr=1e-3, step=1, avg_scales=[x])
    dyt.dyt_adamw_step([], [], [], [], lr=1e-3, step=1)
    assert dyt.dyt_adamw_values([], []) == []
    with pytest.raises(ValueError):
        dyt.token_log_probs(torch.zeros(2, 3, 4), t)


# ---------------------------------------------------------- autograd wiring
def test_wiring_on_stand_ins(dyt, monkeypatch):  # noqa: F811
    """The kernels replaced by plain operations on CPU tensors: which gradient
    goes to which input, and that x and r do not share their gradient's memory."""
    from bwd_dyt_forward_amd import _lm, lm
    monkeypatch.setattr(_lm, "dyt_rms_forward_residual", lambda x, r, g, eps: (x + r, (x + r) * g, (x + r).mean(1)))
    monkeypatch.setattr(_lm, "dyt_rms_backward_residual", lambda h, dy, dres, rstd, g: (dres + dy * g, (dy * h).sum(0)))
    x, r = (torch.randn(4, 6, requires_grad=True) for _ in range(2))
    g = torch.randn(6, requires_grad=True)
    for n in (1, 2):
        h, y = lm.rms_norm_residual(x, r, g)
        (2 * h + 3 * y).sum().backward()
        assert torch.allclose(x.grad, n * (2 + 3 * g.detach()).expand(4, 6)) and torch.equal(x.grad, r.grad)
        assert x.grad.data_ptr() != r.grad.data_ptr()
    seen = []
    monkeypatch.setattr(_lm, "dyt_embed_forward", lambda w, t, s, dt: w[t] * s)
    monkeypatch.setattr(_lm, "dyt_embed_backward",
                        lambda dy, t, V, s, dtype: torch.zeros(V, dy.shape[1], dtype=dtype).index_add_(0, t, dy * s))
    w = torch.randn(5, 3, requires_grad=True)
    t = torch.tensor([[1, 1, 4], [0, 1, 2]])
    y = lm.embedding(w, t, 2.0)
    assert y.shape == (2, 3, 3)
    y.sum().backward()
    assert torch.equal(w.grad[:, 0], torch.tensor([2.0, 6.0, 2.0, 0.0, 2.0]))

    def forward(x, t, scale, top):
        return (x[:, 0] * 1, x[:, 1] * 1, x[:, 2] * 1, *((x[:, :top] * 1, t.view(-1, 1).expand(-1, top) * 1) if top else ()))

    def backward(x, t, entropy, lse, dlogp, dentropy, *, scale):
        seen.append((dlogp, dentropy))
        return x * 0 + 7

    monkeypatch.setattr(_lm, "dyt_logprob_forward", forward)
    monkeypatch.setattr(_lm, "dyt_logprob_backward", backward)
    x = torch.randn(2, 3, 8, requires_grad=True)
    logp, entropy, best, places = lm.token_log_probs(x, t, 1.5, top=2)
    assert logp.shape == entropy.shape == (2, 3) and best.shape == places.shape == (2, 3, 2)
    assert not best.requires_grad
    logp.sum().backward()
    assert (x.grad == 7).all() and seen[-1][1] is None and (seen[-1][0] == 1).all()
    lm.token_log_probs(x, t)[1].sum().backward()
    assert seen[-1][0] is None


def test_the_optimizer_groups_its_tensors(dyt, monkeypatch):  # noqa: F811
    """A call for each step count and width of the states."""
    from bwd_dyt_forward_amd import _lm
    calls = []
    monkeypatch.setattr(_lm, "dyt_adamw_step", lambda ps, gs, ms, vs, **kw: calls.append((ps, ms, kw)))
    p = [torch.nn.Parameter(torch.zeros(n, dtype=dt)) for n, dt in ((10, torch.float32), (600, torch.bfloat16), (700, torch.float32))]
    opt = dyt.AdamW([{"params": p[:2]}, {"params": p[2:], "lr": 0.5}], state_bits=8, min_8bit=512, master=True, seed=3)
    for x in p:
        x.grad = torch.ones_like(x)
    opt.step()
    assert [len(c[0]) for c in calls] == [1, 1, 1]
    small, large, other = calls
    assert small[1][0].dtype == torch.float32 and "seed" not in small[2] and small[2]["masters"] == [None]
    assert large[1][0].dtype == torch.int8 and large[2]["masters"][0].dtype == torch.float32
    assert large[2]["avg_scales"][0].shape == (5,) and other[2]["seed"] != large[2]["seed"] and other[2]["lr"] == 0.5
    assert all(c[2]["step"] == 1 for c in calls)
    p[1].grad = None
    opt.step()
    p[1].grad = torch.ones_like(p[1])
    opt.step()
    assert [c[2]["step"] for c in calls[3:]] == [2, 2, 3, 2, 3]
    sd = opt.state_dict()
    opt2 = dyt.AdamW([{"params": p[:2]}, {"params": p[2:]}], state_bits=8, min_8bit=512, master=True)
    opt2.load_state_dict(sd)
    for x in p:
        for k, v in opt.state[x].items():
            w = opt2.state[x][k]
            assert (v.dtype == w.dtype and torch.equal(v, w) and v is not w) if isinstance(v, torch.Tensor) else v == w
