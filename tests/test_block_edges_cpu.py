"""Block operators without a GPU: rules of the sources, refusals at the edges
of the ranges, the cache's and the autograd functions' bookkeeping. Pointers
are made up; every call comes back before it would use them."""
import glob
import os
import random
import re
import shutil
import subprocess
import sys

import pytest
import torch

from test_block_cpu import AT, CSRC, ROOT, bwd, codes, desc, dyt, fwd  # noqa: F401


def test_every_asm_statement_that_writes_m0_names_it():
    """The compiler keeps values of its own in m0."""
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.h*")):
        for asm in re.findall(r"asm(?: volatile)?\s*\((.*?)\);", open(path).read(), flags=re.S):
            if re.search(r"s_mov_b32 m0", asm):
                found += 1
                assert '"m0"' in asm.rsplit(":", 1)[1], (path, asm)
    assert found == 2


def places(base, size, stride):
    """Elements of a [B, S, H, D] tensor by their address."""
    B, S, H, D = size
    return {base + b * stride[0] + s * stride[1] + h * stride[2] + x
            for b in range(B) for s in range(S) for h in range(H) for x in range(D)}


def overlap_status(dyt, at, sizes, strides):
    """The backward's answer for outputs at these element offsets, without a
    workspace: DYT_ERR_WORKSPACE_TOO_SMALL where they pass."""
    (B, Sq, Hq, D), (_, Sk, Hkv, _) = sizes[:2]
    d = desc(B=B, Sq=Sq, Sk=Sk, Hq=Hq, Hkv=Hkv, D=D, **dict(zip(("dq", "dk", "dv"), strides)))
    base = 1 << 40
    return bwd(dyt, d, n=0, ws=None, **{t: base + 2 * x for t, x in zip(("dq", "dk", "dv"), at)})


def test_gradients_that_share_elements_are_refused(dyt, codes):  # noqa: F811
    bad, ok = codes["DYT_ERR_INVALID_ARG"], codes["DYT_ERR_WORKSPACE_TOO_SMALL"]
    B, S, Hq, Hkv, D = 2, 33, 4, 2, 64
    q, k = (B, S, Hq, D), (B, S, Hkv, D)
    n = Hq + 2 * Hkv
    fused = (S * n * D, n * D, D)
    own = lambda s: (s[1] * s[2] * s[3], s[2] * s[3], s[3])
    far = 1 << 24
    # slices of one projection, each after the other and with one head too far
    assert overlap_status(dyt, (0, Hq * D, (Hq + Hkv) * D), (q, k, k), (fused,) * 3) == ok
    assert overlap_status(dyt, (0, (Hq - 1) * D, (Hq + Hkv) * D), (q, k, k), (fused,) * 3) == bad
    assert overlap_status(dyt, (0, Hq * D, (Hq + Hkv - 1) * D), (q, k, k), (fused,) * 3) == bad
    assert overlap_status(dyt, (0, Hq * D + 1, (Hq + Hkv) * D), (q, k, k), (fused,) * 3) == bad
    # [B, n, S, D]
    heads = (n * S * D, D, S * D)
    assert overlap_status(dyt, (0, Hq * S * D, (Hq + Hkv) * S * D), (q, k, k), (heads,) * 3) == ok
    assert overlap_status(dyt, (0, Hq * S * D - 1, (Hq + Hkv) * S * D), (q, k, k), (heads,) * 3) == bad
    # tensors of their own, one behind the other and one element over it
    m = B * S * Hkv * D
    assert overlap_status(dyt, (far, 0, m), (q, k, k), (own(q), own(k), own(k))) == ok
    assert overlap_status(dyt, (far, 0, m - 1), (q, k, k), (own(q), own(k), own(k))) == bad
    assert overlap_status(dyt, (far, 0, 64), (q, k, k), (own(q), own(k), own(k))) == bad
    assert overlap_status(dyt, (0, B * S * Hq * D - 1, far), (q, k, k), (own(q), own(k), own(k))) == bad
    # batch entries in turn
    assert overlap_status(dyt, (far, 0, S * Hkv * D), (q, k, k), (own(q), (2 * S * Hkv * D, Hkv * D, D), (2 * S * Hkv * D, Hkv * D, D))) == ok


def test_shared_elements_of_random_layouts(dyt, codes):  # noqa: F811
    """Against sets of addresses."""
    bad, ok = codes["DYT_ERR_INVALID_ARG"], codes["DYT_ERR_WORKSPACE_TOO_SMALL"]
    rng = random.Random(11)
    met = 0

    def layout(size):
        order, at, stride = rng.sample(range(3), 3), size[3] + rng.choice([0, 0, 1, 8]), [0, 0, 0]
        for i in order:
            stride[i] = at * rng.choice([1, 1, 2, 3])
            at = stride[i] * size[i]
        return tuple(stride)

    for _ in range(400):
        B, Sq, Sk, Hkv, D = (rng.randint(1, n) for n in (3, 5, 5, 3, 9))
        q, k = (B, Sq, Hkv * rng.randint(1, 2), D), (B, Sk, Hkv, D)
        strides = [layout(q), layout(k), layout(k)]
        if rng.random() < 0.5:
            strides[2] = strides[1]
        at = [rng.randint(0, rng.choice([60, 600])) for _ in range(3)]
        sets = [places(a, s, st) for a, s, st in zip(at, (q, k, k), strides)]
        want = bad if sets[0] & sets[1] or sets[0] & sets[2] or sets[1] & sets[2] else ok
        met += want == bad
        assert overlap_status(dyt, at, (q, k, k), strides) == want, (q, k, strides, at)
    assert 50 < met < 350


def test_problems_that_one_launch_cannot_hold(dyt, codes):  # noqa: F811
    """A launch has fewer than 2^32 threads: refused before anything is
    enqueued, not by a launch in the middle."""
    bad = codes["DYT_ERR_INVALID_ARG"]
    at = {t: (i + 1) << 48 for i, t in enumerate(AT)}
    table = dict(table=1 << 60, buckets=128, distance=1024)
    sizes = dyt.block_lib
    for kw in (dict(B=1, Hq=64, Hkv=64, Sq=1 << 28, Sk=16, D=1), dict(B=64, Hq=64, Hkv=64, Sq=1 << 22, Sk=16, D=1),
               dict(table, B=1, Hq=1 << 20, Hkv=1 << 20, Sq=1 << 11, Sk=4, D=1)):
        d = desc(**kw)
        assert fwd(dyt, d, n=1 << 60, **at) == bad, kw
        assert bwd(dyt, d, n=1 << 60, **at) == bad, kw
        assert sizes.dyt_attn_forward_workspace_size(d) == 0
        assert sizes.dyt_attn_backward_workspace_size(d) == 0
    # many keys, and many heads' buckets: the backward alone
    for kw in (dict(B=1, Hq=64, Hkv=64, Sq=16, Sk=1 << 28, D=1), dict(table, B=1, Hq=1 << 16, Hkv=1 << 16, Sq=4, Sk=4, D=1)):
        d = desc(**kw)
        assert bwd(dyt, d, n=1 << 60, **at) == bad, kw
        assert sizes.dyt_attn_backward_workspace_size(d) == 0
    # no query head, and more key heads than a problem may have
    d = desc(B=4, Hq=0, Hkv=1 << 62, k=(0, 0, 0), v=(0, 0, 0), dk=(0, 0, 0), dv=(0, 0, 0))
    assert fwd(dyt, d, **at) == bad and bwd(dyt, d, **at) == bad
    assert sizes.dyt_attn_backward_workspace_size(desc(B=1, Hq=64, Hkv=64, Sq=1 << 20, Sk=1 << 20, D=128)) > 0


def test_every_dkv_instance_of_four_row_groups_can_be_picked(dyt):  # noqa: F811
    """Two slices above a padded head dimension of 64 in the 16-bit types, and
    there one only with the bias, where a wide table's sums leave no room."""
    names = subprocess.run(["nm", "-C", dyt.BLOCK_LIB_FILE], capture_output=True, text=True, check=True).stdout
    found = {(t, int(dp), int(sl), b == "true") for t, dp, sl, b in re.findall(
        r"attn_dkv_kernel<(?:dyt::)?(\w+), (\d+), 4, (\d), (true|false), true>\(", names)}
    want = {("float", dp, 1, b) for dp in (32, 64, 96, 128) for b in (True, False)}
    for t in ("bf16_t", "f16_t"):
        want |= {(t, dp, 1, b) for dp in (32, 64) for b in (True, False)}
        want |= {(t, dp, 2, b) for dp in (96, 128) for b in (True, False)} | {(t, dp, 1, True) for dp in (96, 128)}
    assert found == want


@pytest.mark.parametrize("state", ["missing", "other sources"])
def test_the_package_without_the_block_library(dyt, tmp_path, state):  # noqa: F811
    """DyT needs its own library only; the block operators' names fail loudly."""
    package = "bwd_dyt_forward_amd"
    os.mkdir(tmp_path / package)
    for name in os.listdir(os.path.join(ROOT, package)):
        if name.endswith((".py", ".so", ".json")) and name != "libdyt_block.so" or name == "csrc":
            os.symlink(os.path.join(ROOT, package, name), tmp_path / package / name)
    # build.py finds the sources next to itself
    os.remove(tmp_path / package / "build.py")
    shutil.copy(os.path.join(ROOT, package, "build.py"), tmp_path / package / "build.py")
    os.symlink(os.path.join(ROOT, "include"), tmp_path / "include")
    if state == "other sources":
        lib = open(dyt.BLOCK_LIB_FILE, "rb").read()
        mark = lib.index(b"DYT_BUILD_ID=") + 13
        open(tmp_path / package / "libdyt_block.so", "wb").write(lib[:mark] + b"0" * 16 + lib[mark + 16:])
    word = "not found" if state == "missing" else "other sources"
    code = f"""
import sys
sys.path.insert(0, {str(tmp_path)!r})
import {package} as m
from {package} import *
assert m.__file__.startswith({str(tmp_path)!r}) and m.dyt_abi_version() and DyT(8).num_features == 8
for name in ("Attention", "layer_norm", "block_lib"):
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


def test_a_build_at_the_default_path_brings_the_block_library(monkeypatch):
    from bwd_dyt_forward_amd import build
    for stream_ref in (True, False):
        made = []
        monkeypatch.setattr(build, "_compile", lambda out, *a, **kw: made.append(out))
        build.build(with_stream_ref=stream_ref)
        assert build.BLOCK_LIB_PATH in made and (build.STREAM_REF_PATH in made) == stream_ref
        made.clear()
        build.build(out="/elsewhere.so", with_stream_ref=stream_ref)
        assert made == ["/elsewhere.so"]


@pytest.mark.parametrize("name", ["seqlens_k", "q_start"])
def test_lists_that_change_before_the_backward_are_an_error(dyt, monkeypatch, name):  # noqa: F811
    """The kernels replaced by plain operations on CPU tensors."""
    from bwd_dyt_forward_amd import _block, block
    seen = []

    def backward(q, k, v, o, do, stats, *, table, seqlens_k, q_start, **kw):
        seen.append((seqlens_k, q_start))
        return (do, k, v) if table is None else (do, k, v, table)

    monkeypatch.setattr(_block, "dyt_attn_forward", lambda q, k, v, **kw: (q * 2, q[..., 0]))
    monkeypatch.setattr(_block, "dyt_attn_backward", backward)
    q, k, v = (torch.randn(2, 3, 2, 4, requires_grad=True) for _ in range(3))
    table = torch.randn(8, 2, requires_grad=True)
    for t in (None, table):
        lists = {name: torch.tensor([1, 2], dtype=torch.int32)}
        block.attention(q, k, v, table=t, **lists).sum().backward()
        got = dict(zip(("seqlens_k", "q_start"), seen[-1]))
        assert got.pop(name).tolist() == [1, 2] and list(got.values()) == [None]
        o = block.attention(q, k, v, table=t, **lists)
        lists[name] += 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            o.sum().backward()
    assert len(seen) == 2 and table.grad is not None


def test_an_append_that_fails_takes_no_room(dyt):  # noqa: F811
    c = dyt.KVCache(2, 5, 1, 4, torch.float32, "cpu")
    x = torch.ones(2, 3, 1, 4)
    for k, v in ((x.double(), x), (x, x.double()), (x[..., :3], x), (x, x[:, :2]), (torch.ones(3, 3, 1, 4), x)):
        with pytest.raises((RuntimeError, IndexError)):
            c.append(k, v)
        assert c.length.tolist() == [0, 0]
    assert c.append(x, x).tolist() == [0, 0] and c.append(x[:, :2], x[:, :2]).tolist() == [3, 3]
    with pytest.raises(ValueError, match="no room"):
        c.append(x[:, :1], x[:, :1])


def test_a_batch_that_is_not_the_caches_changes_nothing(dyt):  # noqa: F811
    m = dyt.Attention(8, 2, 2, device="cpu")
    c = dyt.KVCache(3, 5, 2, 4, torch.float32, "cpu")
    with pytest.raises(ValueError, match="sequences"):
        m(torch.ones(1, 2, 8), cache=c)
    assert c.length.tolist() == [0, 0, 0] and (c.k == 0).all()


def test_appends_behind_the_end_write_nothing_out_of_range(dyt):  # noqa: F811
    """What a captured append's replays do once the cache is full: the host's
    check does not run again."""
    c = dyt.KVCache(3, 4, 1, 2, torch.float32, "cpu")
    c.length.copy_(torch.tensor([1, 3, 4]))
    x = torch.arange(1.0, 13).view(3, 2, 1, 2)
    starts = [c.append(x, -x).tolist()]
    for _ in range(2):
        c._used = 0
        starts.append(c.append(x + 100, x + 100).tolist())
    assert starts == [[1, 3, 4], [3, 4, 4], [4, 4, 4]] and c.length.tolist() == [4, 4, 4]
    assert c.k.shape == (3, 4, 1, 2)
    want = torch.zeros(3, 4, 1, 2)
    want[0, 1:3], want[0, 3], want[1, 3] = x[0], x[0, 0] + 100, x[1, 0]
    assert torch.equal(c.k, want)


def test_a_cache_holds_values_and_no_graph(dyt):  # noqa: F811
    c = dyt.KVCache(2, 6, 1, 4, torch.float32, "cpu")
    k, v = (torch.randn(2, 2, 1, 4, requires_grad=True) for _ in range(2))
    for n in (0, 2):
        start = c.append(k, v)
        assert not c.k.requires_grad and not c.v.requires_grad and not c.length.requires_grad
        all_k, all_v = c.with_gradient(k, v, start)
        assert torch.equal(all_k, c.k) and torch.equal(all_v, c.v) and all_k.shape == c.k.shape
        k.grad = v.grad = None
        (all_k * 2 + all_v * 3).sum().backward()
        assert (k.grad == 2).all() and (v.grad == 3).all()
    with torch.no_grad():
        start = c.append(k, v)
        assert all(a is b for a, b in zip(c.with_gradient(k, v, start), (c.k, c.v)))
    assert c.with_gradient(k.detach(), v.detach(), start)[0] is c.k
