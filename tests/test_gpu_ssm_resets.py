"""Selective scan: the decay between two tokens behind strong ones of their block of
16. Steps that empty the state many times over leave log sums of up to 1.5e5, whose
fp32 steps are 2^-6; the factor between two mild tokens behind them is still exact to
a few roundings. One key column, one value channel: y_i = exp(-(d_{j+1} + .. + d_i))
d_j x_j, a single product, off by at most 16 roundings (products, exponential, its
argument's parts)."""
import math

import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("strong", [300.7, 1234.5, 4999.9, 9999.37, 1e6])
@pytest.mark.parametrize("T", [16, 64, 150])
def test_mild_tokens_behind_strong_ones(T, strong):
    B, H, P, N = 1, 8, 32, 32
    g = torch.Generator().manual_seed(T)
    dt = strong * (1 + 0.01 * torch.rand((B, H, T), generator=g))
    for c in range(0, T, 16):
        for t in (13, 14, 15):
            if c + t < T:
                dt[:, :, c + t] = torch.rand((B, H), generator=g)
    x, Bm = torch.zeros(B, H, T, P), torch.zeros(B, 1, T, N)
    x[..., 0] = 1 + torch.rand((B, H, T), generator=g)
    for c in range(0, T, 16):
        if c + 13 < T:
            Bm[:, :, c + 13, 0] = 1.0          # only this token of the block enters
    Cm = torch.zeros(B, 1, T, N)
    Cm[..., 0] = 1.0
    A = -torch.ones(H)
    y, _ = osdn.ssm_forward(x.to(DEV), dt.to(DEV), A.to(DEV), Bm.to(DEV), Cm.to(DEV),
                            softplus=False)
    y = y.cpu().double()
    for c in range(0, T - 15, 16):
        j = c + 13
        want = dt[:, :, j].double() * x[:, :, j, 0].double()
        for i in (j, j + 1, j + 2):
            if i > j:
                want = want * torch.exp(-dt[:, :, i].double())
            err = float(((y[:, :, i, 0] - want) / want).abs().max())
            print("tokens %d to %d: %.2e" % (j, i, err), flush=True)
            assert err <= 16 * 2.0 ** -24, (j, i)
    assert math.isfinite(float(y.abs().max()))
