"""Gradients of the recurrence's gates far from their middle, against the fp64 oracle.
Both carry a factor 1 - sigmoid, which is far below one at an open gate and has to keep
its digits there: as exp(-z) sigmoid(z) it is off by 2 units of 2^-24 for the exponential
and 1.3 |z| for its rounded argument (half a step, and log2(e) as rounded)."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32, f64, held
from oracle import layer as Y

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("C", [70, 71])
@pytest.mark.parametrize("low,high", [(8.0, 20.0), (20.0, 80.0), (-20.0, -8.0), (-2.0, 2.0)])
def test_gate_gradients(low, high, C, normalize, dt):
    B, T = 2, 40
    g = torch.Generator().manual_seed(int(low) + C)
    n = lambda *s: torch.randn(s, generator=g)
    z = lambda: (low + (high - low) * torch.rand((B, T, C), generator=g)).to(dt).to(DEV)
    x, r, i, dy = n(B, T, C).to(dt).to(DEV), z(), z(), n(B, T, C).to(dt).to(DEV)
    A = -torch.exp(n(C) - 2).to(DEV)
    h0, dh = n(B, C).to(DEV), n(B, C).to(DEV)
    d = osdn.glr_backward(x, r, A, dy, i=i, h0=h0, dh_T=dh, normalize=normalize)
    torch.cuda.synchronize()
    ref, mag = Y.glr_backward_ref(f64(x), f64(r), f64(A), f64(dy), i=f64(i), h0=f64(h0),
                                  dh_T=f64(dh), normalize=normalize)
    wide = 112 + T / 8
    for name, z in (("r", r), ("i", i)):
        assert np.all(ref[name] != 0)
        held(d[name], ref[name], (wide + 1.3 * np.abs(f64(z)), mag[name]), what="d" + name)
    for name in ("x", "A", "h0"):
        held(d[name], ref[name], (wide, mag[name]), what="d" + name)
