"""Host side of the decoder operators at their edges, without a GPU: as in
test_lm_cpu.py the pointers are made up, and every call must come back before it
would use them."""
import pytest
import torch

from test_block_cpu import codes, dyt  # noqa: F401
from test_lm_cpu import BF16, OK, P, options, tensor


def lp_fwd_norm(lib, **kw):
    a = dict(x=P, ld=0, t=2 * P, logp=3 * P, ent=4 * P, lse=5 * P, norm=9 * P, top_logp=6 * P, top_tokens=7 * P, ws=8 * P,
             n=1 << 24, T=50, V=100, scale=1.0, top=3, dt=BF16, bits=64)
    a.update(kw)
    return lib.dyt_logprob_forward_norm(*a.values(), None)


def lp_bwd_norm(lib, **kw):
    a = dict(x=P, ld=0, t=2 * P, norm=4 * P, dlogp=5 * P, dent=6 * P, dx=7 * P, ldd=0, T=50, V=100, scale=1.0,
             dt=BF16, bits=64)
    a.update(kw)
    return lib.dyt_logprob_backward_norm(*a.values(), None)


def test_refusals_of_the_sums_in_two_numbers(dyt, codes):  # noqa: F811
    lib = dyt.lm_lib
    bad, mis = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED"))
    for kw in (dict(norm=None), dict(norm=3 * P + 196), dict(norm=P + 64), dict(logp=9 * P + 596), dict(norm=7 * P),
               dict(lse=None), dict(top=0)):
        assert lp_fwd_norm(lib, **kw) == bad, kw
    for kw in (dict(norm=None), dict(dx=4 * P + 596), dict(dx=P + 2)):
        assert lp_bwd_norm(lib, **kw) == bad, kw
    assert lp_fwd_norm(lib, norm=9 * P + 2) == mis and lp_bwd_norm(lib, norm=4 * P + 2) == mis
    assert lp_fwd_norm(lib, T=0, norm=None) == OK and lp_bwd_norm(lib, T=0, norm=None) == OK


def test_a_library_without_an_entry_is_an_import_error(dyt):  # noqa: F811
    from bwd_dyt_forward_amd import _lm
    with pytest.raises(ImportError, match="rebuild"):
        _lm._load(dyt.BLOCK_LIB_FILE)


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_does_not_count(dyt, capturable):  # noqa: F811
    """Parameters on the host are refused."""
    p = torch.nn.Parameter(torch.zeros(8))
    p.grad = torch.ones(8)
    opt = dyt.AdamW([p], capturable=capturable)
    for _ in range(2):
        with pytest.raises(ValueError, match="device"):
            opt.step()
        assert int(opt.state[p]["step"]) == 0


def test_a_shared_counter_needs_equal_counts(dyt, monkeypatch):  # noqa: F811
    from bwd_dyt_forward_amd import _lm
    calls = []
    monkeypatch.setattr(_lm, "dyt_adamw_step", lambda ps, gs, ms, vs, **kw: calls.append(int(kw["step"])))
    p = [torch.nn.Parameter(torch.zeros(8)) for _ in range(2)]
    for x in p:
        x.grad = torch.ones(8)
    first = dyt.AdamW(p)
    first.step()
    # equal counts, of whatever kind, become one counter
    opt = dyt.AdamW(p, capturable=True)
    sd = first.state_dict()
    sd["param_groups"][0]["capturable"] = True
    opt.load_state_dict(sd)
    opt.step()
    assert calls[-1] == 2 and opt.state[p[0]]["step"] is opt.state[p[1]]["step"]
    again = dyt.AdamW(p, capturable=True)
    again.load_state_dict(opt.state_dict())
    again.step()
    assert calls[-1] == 3 and again.state[p[0]]["step"] is again.state[p[1]]["step"]
    # different ones are refused, and nothing moves on
    p[1].grad = None
    first.step()
    sd = first.state_dict()
    sd["param_groups"][0]["capturable"] = True
    opt = dyt.AdamW(p, capturable=True)
    opt.load_state_dict(sd)
    p[1].grad = torch.ones(8)
    count = len(calls)
    with pytest.raises(ValueError, match="numbers of steps"):
        opt.step()
    assert len(calls) == count and [int(opt.state[x]["step"]) for x in p] == [2, 1]


def test_a_step_can_be_checked_alone(dyt, codes):  # noqa: F811
    check = dyt.lm_lib.dyt_adamw_check
    bad, mis = (codes[f"DYT_ERR_{n}"] for n in ("INVALID_ARG", "MISALIGNED"))
    at = 16 * P
    assert check(tensor(1) + tensor(2), 2, options()) == OK and check(None, 0, options()) == OK
    assert check(tensor(1) + tensor(1), 2, options()) == bad and check(tensor(1), 1, options(lr=-1.0)) == bad
    assert check(tensor(1, m=at), 1, options()) == bad and check(tensor(1, p=at + 1), 1, options()) == mis
    assert check(tensor(), 1, None) == bad
