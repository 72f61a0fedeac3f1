"""Single tokens of the recurrence on rows whose offsets pass 32 bits: every batch entry,
every token and the state that is left give the bits of rows side by side."""
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32
from test_gpu_layer_far import apart, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [64, 63])
def test_decode_rows_far_apart(C, dt):
    """Tokens 2^22 elements apart, the limit, and entries 1200 of them (20 GB in fp32)."""
    B, T = 2, 4
    x, r, i = (rand(B, T, C, seed=s, dt=dt) for s in range(3))
    A, h = -torch.rand(C, device=DEV), torch.randn(B, C, device=DEV)
    row = 1 << 22
    buf = torch.empty(1200 * row + T * row, dtype=dt, device=DEV)
    fx = buf.as_strided((B, T, C), (1200 * row, row, 1))
    fx.copy_(x)
    assert fx.stride(0) * (B - 1) > 1 << 32
    want, got = h.clone(), h.clone()
    y = osdn.glr_decode(x, r, A, want, i=i)
    for a, b, c in ((fx, r, i), (x, apart(r, row), i), (x, r, apart(i, row))):
        got.copy_(h)
        assert torch.equal(osdn.glr_decode(a, b, A, got, i=c), y) and torch.equal(got, want)
    # one token: the entries alone lie far apart
    want, got = h.clone(), h.clone()
    y = osdn.glr_decode(x[:, -1:], r[:, -1:], A, want)
    assert torch.equal(osdn.glr_decode(fx[:, -1:], r[:, -1:], A, got), y)
    assert torch.equal(got, want)
