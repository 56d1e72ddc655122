"""Attention's gradients where a masked place could leak into a sum: padding
rows of the last tile under a large bias, against the formulas in float64
(tests/block_ref.py) and against the same problem with whole tiles."""
import math

import pytest
import torch

from block_ref import Attention
from test_gpu_block_attn import DTYPES, dyt, make, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu

# row tiles of 32 and 64 that end before the tile does, one wave and four to
# a workgroup, slices, splits, each padded head dimension
SIZES = [(2, 33, 70, 2, 1, 32), (1, 70, 40, 2, 2, 64), (1, 96, 96, 1, 1, 24), (2, 129, 129, 2, 2, 80),
         (1, 700, 40, 1, 1, 64), (16, 160, 130, 16, 16, 64), (16, 100, 130, 16, 16, 128), (1, 37, 50, 2, 1, 33)]


def table_problem(dt, causal, size, shift, every):
    t, do, kw = make(41, DTYPES[dt], *size, buckets=16, distance=40, causal=causal, bidirectional=not causal,
                     table_dt=torch.float32)
    kw["table"][::every] += shift
    return t, do, kw


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("entry", [12.0, 30.0])
def test_entries_whose_exponential_passes_float16(dyt, entry, causal, size):  # noqa: F811
    """exp(11.09) is float16's largest value."""
    run_and_check(dyt, *table_problem("f16", causal, size, entry, 3))


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt,shift", [("f16", 30.0), ("bf16", 100.0), ("f32", 100.0)])
def test_an_offset_of_the_whole_table(dyt, dt, shift, causal, size):  # noqa: F811
    """The softmax takes it out again; exp(88.72) is float32's largest value."""
    run_and_check(dyt, *table_problem(dt, causal, size, shift, 1))


@pytest.mark.parametrize("size", [s for s in SIZES if s[1] % 32], ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt,entry", [("f16", 12.0), ("f16", 30.0), ("bf16", 90.0), ("f32", 100.0)])
def test_rows_of_zero_gradient_change_no_bit(dyt, dt, entry, causal, size):  # noqa: F811
    """The rows that complete a block of 32 (so every launch stays the same)
    have do = 0: they add exact zeros."""
    B, Sq, Sk, Hq, Hkv, D = size
    full = (B, (Sq + 31) // 32 * 32, Sk, Hq, Hkv, D)
    t, do, kw = table_problem(dt, causal, full, entry, 3)
    kw["q_start"] = torch.full((B,), Sk - Sq, dtype=torch.int32, device="cuda")
    do[:, Sq:] = 0
    o, stats = dyt.dyt_attn_forward(t["q"], t["k"], t["v"], **kw)
    want = dyt.dyt_attn_backward(t["q"], t["k"], t["v"], o, do, stats, **kw)
    q, o, do = (x[:, :Sq].contiguous() for x in (t["q"], o, do))
    got = dyt.dyt_attn_backward(q, t["k"], t["v"], o, do, stats[:, :, :Sq].contiguous(), **kw)
    for name, a, b in zip(("dq", "dk", "dv", "dtable"), got, (want[0][:, :Sq], *want[1:])):
        assert torch.isfinite(a).all() and torch.equal(a, b), name
