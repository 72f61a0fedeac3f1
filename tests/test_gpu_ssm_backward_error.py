"""Selective scan's backward: errors of whole gradients in bf16. dx, dB and dC are the
exact gradients rounded once, and little else: rounding the 64-bit gradient itself is
e0 (relative L2); operands in two bf16 parts leave 2^-16 of terms up to some thirty
times their sums, 2^-11, which is independent of it: the squares add. ``left`` scales the adjoint dS_T, ``came`` the state S0: at 10
they make up most of the gradients, of dx where D is not there."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import f64
from oracle import mixer as M
from test_gpu_ssm import CASES, IDS, adjoints, inputs, ref_args

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BF_CASES = [(c, i) for c, i in zip(CASES, IDS) if c[6] is BF]
# heads of a group in turn: 128 x 128 in one part, and in two
BF_CASES += [((128, 6, 2, 5, 128, 128, BF, None), "heads-128x128"),
             ((64, 4, 1, 66, 128, 64, BF, None), "heads-128x64")]


def rel(got, ref):
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)


@pytest.mark.parametrize("left,came,D", [(1.0, 1.0, True), (10.0, 1.0, True),
                                         (1.0, 10.0, True), (1.0, 1.0, False),
                                         (10.0, 1.0, False)])
@pytest.mark.parametrize("case", [c for c, _ in BF_CASES], ids=[i for _, i in BF_CASES])
def test_gradient_error(case, left, came, D):
    print("case:", case, left, came, D, flush=True)
    B, H, G, T, P, N, dt, lens = case
    a, k = inputs(B, H, G, T, P, N, dt, lens=lens, seed=13)
    k["S0"] *= came
    if not D:
        k["D"] = None
    dy, dS = adjoints(a, k)
    dS *= left
    got = osdn.ssm_backward(**a, dy=dy, dS_T=dS, **k)
    r, q, _, _ = ref_args(a, k)
    ref = M.ssm_backward_ref(**r, dy=f64(dy), dS_T=f64(dS), **q)
    for n in ("x", "B", "C"):
        e0 = rel(torch.from_numpy(ref[n]).to(dt).double().numpy(), ref[n])
        e = rel(f64(got[n]), ref[n])
        print("d%s: %.3e (rounding alone %.3e)" % (n, e, e0), flush=True)
        assert e <= np.hypot(e0, 2.0 ** -11), n
