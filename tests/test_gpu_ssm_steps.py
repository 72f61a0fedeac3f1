"""Selective scan: raw steps at the ends of fp32's range inside a sequence.

-inf and the lowest values switch a token off: softplus and its slope are zero
there, the state passes through and the token's own input enters nowhere but
through D. The highest values empty the state: the decay is zero, and with x and B
zero at such a token nothing enters either. Every call against the fp64 oracle,
within the bounds of the ordinary steps."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import held
from oracle import mixer as M
from test_gpu_ssm import (K, adjoints, check_backward, check_forward, check_l2,
                          inputs, ref_args)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LOW, HIGH = torch.finfo(F32).min, torch.finfo(F32).max
OFF = [float("-inf"), LOW, -2.4e38, -1e30, -200.0]
# the first and last tokens, both sides of blocks of 16 and chunks of 32 and 64
AT = (0, 1, 15, 16, 31, 32, 47, 63, 64, 100, 128, 149)


def switched_off(T, dt, seed):
    a, k = inputs(2, 4, 2, T, 64, 32, dt, seed=seed)
    for i, t in enumerate(AT):
        if t < T:
            a["dt"][:, :, t] = OFF[i % len(OFF)]
            a["dt"][1, :, t] = OFF[(i + 2) % len(OFF)]
    a["dt"][:, 0, T // 2:] = LOW          # a head that stops half way
    return a, k


def emptied(T, dt, high, seed):
    a, k = inputs(2, 4, 2, T, 64, 32, dt, seed=seed)
    for t in (5, 16, 63, 64, 130):
        if t < T:
            a["dt"][:, :, t] = high
            a["x"][:, :, t] = 0
            a["B"][:, :, t] = 0
    return a, k


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 20, 150, 600])
def test_tokens_switched_off(T, dt):
    a, k = switched_off(T, dt, T)
    check_forward(a, k, osdn.ssm_forward(**a, **k))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("high", [HIGH, 2.4e38, 1e30])
@pytest.mark.parametrize("T", [20, 150, 600])
def test_state_emptied(T, high, dt):
    a, k = emptied(T, dt, high, T)
    check_forward(a, k, osdn.ssm_forward(**a, **k))


def decoded(a, k):
    k = dict(k)
    S0 = k.pop("S0")
    k.pop("lengths")
    S = torch.empty_like(S0)
    y = osdn.ssm_decode(**a, S=S0, S_out=S, **k)
    k.update(S0=S0, lengths=None)
    r, q, ab, qb = ref_args(a, k)
    ry, rS = M.ssm_ref(**r, **q)
    my, mS = M.ssm_ref(**ab, **qb)
    held(y, ry, my, K, what="y")
    held(S, rS, mS, K, what="S")


@pytest.mark.parametrize("dt", [BF, F32])
def test_single_tokens(dt):
    decoded(*switched_off(20, dt, 3))
    for high in (HIGH, 2.4e38, 1e30):
        decoded(*emptied(20, dt, high, 4))
    # one token, switched off: the state's bits stay, y = S C + D x
    a, k = switched_off(1, dt, 5)
    S = k["S0"].clone()
    osdn.ssm_decode(**a, S=S, D=k["D"], dt_bias=k["dt_bias"])
    assert torch.equal(S, k["S0"])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("high", [None, HIGH, 2.4e38, 1e30])
@pytest.mark.parametrize("T", [20, 150, 900])
def test_gradients(T, high, dt):
    a, k = switched_off(T, dt, T + 1) if high is None else emptied(T, dt, high, T + 1)
    dy, dS = adjoints(a, k)
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    ref = check_backward(a, k, dy, dS, got)
    check_l2(got, ref, ("dt", "A", "D", "dt_bias", "S0"), 1e-5)
    if high is None:
        off = torch.isneginf(a["dt"]) | (a["dt"] < -1e29)
        assert off.any() and not got["dt"][off].any()
        assert np.all(ref["dt"][off.cpu().numpy()] == 0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_step_that_is_no_number_stays_none(dt):
    """NaN in dt reaches its own head's later tokens, and no others."""
    a, k = inputs(1, 4, 2, 150, 64, 32, dt, seed=6)
    y0, S0 = osdn.ssm_forward(**a, **k)
    a["dt"][0, 1, 70] = float("nan")
    y, S = osdn.ssm_forward(**a, **k)
    assert torch.isnan(y[0, 1, 70:]).all() and torch.isnan(S[0, 1]).all()
    for h in (0, 2, 3):
        assert torch.equal(y[0, h], y0[0, h]) and torch.equal(S[0, h], S0[0, h])
    one = {n: (t if n == "A" else t[:, :, 70:71].contiguous()) for n, t in a.items()}
    st = k["S0"].clone()
    y = osdn.ssm_decode(**one, S=st, D=k["D"], dt_bias=k["dt_bias"])
    assert torch.isnan(y[0, 1]).all() and torch.isnan(st[0, 1]).all()
    assert torch.isfinite(y[0, 0]).all() and torch.isfinite(st[0, 2:]).all()
