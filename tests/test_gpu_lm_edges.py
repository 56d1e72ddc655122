"""Calls of the decoder operators that the documentation allows at the edges of
their ranges, on the GPU against float64."""
import math

import numpy as np
import pytest
import torch
from torch import nn

from block_ref import HALF, U, check, d
from lm_ref import EXP2, LogProb, avg_values

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dyt():
    import bwd_dyt_forward_amd as m
    return m


# ---------------------------------------------------- root-mean-square norm
@pytest.mark.parametrize("M,N", [(64, 8192), (700, 96), (5, 70001)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_codes_are_the_rounded_quotients(dyt, M, N, group):
    """q is y / scale, a float32 quotient, rounded to e4m3. Elements of 8 bits
    make many quotients lie next to the middle between two codes."""
    g = torch.Generator().manual_seed(N)
    x = (torch.randn(M, N, generator=g) * 1.5).bfloat16().float().cuda()
    gamma = (torch.randn(N, generator=g) * 0.1 + 1).bfloat16().float().cuda()
    x[:, ::61] *= 8
    y, _ = dyt.dyt_rms_forward(x, gamma)
    q, scales = dyt.dyt_rms_forward_q8(x, gamma, group=group)
    s = scales.cpu().repeat_interleave(group or N, 1)[:, :N]
    want = (y.cpu() / s).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))
