"""Selective scan: errors of whole outputs. y in bf16 is the exact result rounded
once, and little else: rounding the 64-bit result itself is e0 (relative L2);
operands in two bf16 parts leave 2^-16 of terms up to some thirty times their sums,
2^-11. fp32 results: at most 320 roundings of terms ten times their sums,
sqrt(320) 2^-24 10 = 1.1e-5."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import f64
from oracle import mixer as M
from test_gpu_ssm import CASES, IDS, inputs, ref_args

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rel(got, ref):
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)


@pytest.mark.parametrize("state", [1.0, 10.0])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_error(case, state):
    """``state`` scales S0: at 10 the states that came in make up most of y."""
    print("case:", case, state, flush=True)
    B, H, G, T, P, N, dt, lens = case
    a, k = inputs(B, H, G, T, P, N, dt, lens=lens, seed=12)
    k["S0"] *= state
    y, S = osdn.ssm_forward(**a, **k)
    r, q, _, _ = ref_args(a, k)
    ry, rS = M.ssm_ref(**r, **q)
    e0 = rel(torch.from_numpy(ry).to(dt).double().numpy(), ry) if dt is BF else 0.0
    bound = e0 + 2.0 ** -11 if dt is BF else 1.1e-5
    print("y: %.3e (rounding alone %.3e), S_T: %.3e" % (rel(f64(y), ry), e0, rel(f64(S), rS)),
          flush=True)
    assert rel(f64(y), ry) <= bound
    assert rel(f64(S), rS) <= 1.1e-5
