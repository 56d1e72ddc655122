"""Host side of the decoder operators at their edges, without a GPU: as in
test_lm_cpu.py the pointers are made up, and every call must come back before it
would use them."""
import pytest
import torch

from test_block_cpu import codes, dyt  # noqa: F401
from test_lm_cpu import BF16, OK, P


def lp_fwd_norm(lib, **kw):
    a = dict(x=P, ld=0, t=2 * P, logp=3 * P, ent=4 * P, lse=5 * P, norm=9 * P, top_logp=6 * P, top_tokens=7 * P, ws=8 * P,
             n=1 << 24, T=50, V=100, scale=1.0, top=3, dt=BF16, bits=64)
    a.update(kw)
    return lib.dyt_logprob_forward_norm(*a.values(), None)


def lp_bwd_norm(lib, **kw):
    a = dict(x=P, ld=0, t=2 * P, ent=3 * P, norm=4 * P, dlogp=5 * P, dent=6 * P, dx=7 * P, ldd=0, T=50, V=100, scale=1.0,
             dt=BF16, bits=64)
    a.update(kw)
    return lib.dyt_logprob_backward_norm(*a.values(), None)


def test_refusals_of_the_sums_in_two_numbers(dyt, codes):  # noqa: F811
    lib = dyt.lm_lib
    bad, mis = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED"))
    for kw in (dict(norm=None), dict(norm=3 * P + 196), dict(norm=P + 64), dict(logp=9 * P + 396), dict(norm=7 * P),
               dict(lse=None), dict(top=0)):
        assert lp_fwd_norm(lib, **kw) == bad, kw
    for kw in (dict(norm=None), dict(dx=4 * P + 396), dict(ent=None), dict(dx=P + 2)):
        assert lp_bwd_norm(lib, **kw) == bad, kw
    assert lp_fwd_norm(lib, norm=9 * P + 2) == mis and lp_bwd_norm(lib, norm=4 * P + 2) == mis
    assert lp_fwd_norm(lib, T=0, norm=None) == OK and lp_bwd_norm(lib, T=0, norm=None) == OK


def test_a_library_without_an_entry_is_an_import_error(dyt):  # noqa: F811
    from bwd_dyt_forward_amd import _lm
    with pytest.raises(ImportError, match="rebuild"):
        _lm._load(dyt.BLOCK_LIB_FILE)
