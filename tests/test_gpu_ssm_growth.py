"""Selective scan: factors past fp32's range."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from test_gpu_ssm import inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [BF, F32])
def test_growth_past_the_range_is_infinite(dt):
    """A factor past fp32's range is inf, as in the single-token form: the state
    keeps its signs."""
    a, k = inputs(1, 2, 1, 40, 64, 64, dt, seed=5)
    a["A"].fill_(1.0)
    a["dt"].zero_()
    a["x"][:, :, 0] = 0
    k.update(D=None, dt_bias=None)
    for grow in torch.linspace(89.0, 300.0, 40).tolist() + [9e3, 1e5, 3e38]:
        a["dt"][:, :, 0] = grow
        _, S = osdn.ssm_forward(**a, **k, softplus=False)
        want = torch.empty_like(S)
        osdn.ssm_decode(**a, S=k["S0"], S_out=want, softplus=False)
        assert torch.isinf(want).all()
        assert torch.equal(S, want)
