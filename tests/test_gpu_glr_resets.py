"""The recurrence behind gates that forget: what is left of a state, and what came in
after it, keep their digits however large the state was before. Every bound is relative
to the terms that are left."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32, f64, held
from oracle import layer as Y

pytestmark = pytest.mark.gpu


def inputs(B, T, C, dt, scale, fade, seed):
    """Weak inputs, states and adjoints of `scale`, decays from none to exp(-fade) a token."""
    g = torch.Generator().manual_seed(seed + T + C)
    n = lambda *s: torch.randn(s, generator=g)
    x, dy = (1e-3 * n(B, T, C)).to(dt).to(DEV), (1e-3 * n(B, T, C)).to(dt).to(DEV)
    r = (2 * n(B, T, C)).to(dt).to(DEV)
    A = -fade * torch.rand(C, generator=g).to(DEV)
    return x, r, A, dy, scale * n(B, C).to(DEV), scale * n(B, C).to(DEV)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 1e4, 1e15])
@pytest.mark.parametrize("fade", [1.0, 8.0, 60.0])
@pytest.mark.parametrize("B,T,C", [(2, 16, 66), (2, 130, 65), (1, 600, 64), (2, 1300, 34)])
def test_states_behind_resets(B, T, C, fade, scale, dt):
    x, r, A, dy, h0, dh = inputs(B, T, C, dt, scale, fade, 20)
    y, h_T, states = osdn.glr_forward(x, r, A, h0=h0, save=True)
    d = osdn.glr_backward(x, r, A, dy, h0=h0, dh_T=dh, states=states)
    torch.cuda.synchronize()
    a = [f64(t) for t in (x, r, A)]
    ry, rh, rb = Y.glr_ref(*a, h0=f64(h0))
    my, mh, mb = Y.glr_ref(np.abs(a[0]), a[1], a[2], h0=np.abs(f64(h0)))
    # a logarithm summed over the memory scales its roundings by itself: exp(-L) is off by
    # 6 L units, and L passes 80 before exp(-L) times the largest state is below the rest
    u = 48 + T / 16 + 6 * 80
    held(y, ry, (u, my), what="y")
    held(h_T, rh, (u, mh), what="h_T")
    held(states, rb[:, ::16], (u, mb[:, ::16]), what="states")
    g, mag = Y.glr_backward_ref(*a, f64(dy), h0=f64(h0), dh_T=f64(dh))
    for n in ("x", "r", "A", "h0"):
        held(d[n], g[n], (2 * u + 16, mag[n]), what="d" + n)


@pytest.mark.parametrize("T", [16, 128, 129, 4096])
def test_a_total_reset_leaves_the_new_terms(T):
    """A decay of zero: the state is the last input, whatever it was before."""
    B, C = 1, 64
    x = torch.randn((B, T, C), generator=torch.Generator().manual_seed(21)).to(DEV)
    r = torch.full_like(x, 30.0)
    A = torch.full((C,), -1e4, device=DEV)
    h0 = torch.full((B, C), 1e30, device=DEV)
    y, h_T, states = osdn.glr_forward(x, r, A, h0=h0, save=True)
    assert torch.equal(y, x) and torch.equal(h_T, x[:, -1])
    assert torch.equal(states[:, 0], h0) and torch.equal(states[:, 1:], x[:, 15:T - 1:16])
    d = osdn.glr_backward(x, r, A, x, h0=h0, dh_T=h0)
    # (y is x: its gradient is dy, and dh_T comes in at the last token)
    want = x.clone()
    want[:, -1] += h0
    assert torch.equal(d["x"], want) and not d["h0"].any()


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,C", [(2, 40, 66), (1, 300, 65), (2, 1300, 34)])
def test_growth(B, T, C, dt):
    """Without the input factor a positive A is a state that grows."""
    x, r, A, dy, h0, dh = inputs(B, T, C, dt, 1.0, 1.0, 22)
    A = -A * min(1.0, 60.0 / T)
    k = dict(h0=h0, normalize=False)
    y, h_T, states = osdn.glr_forward(x, r, A, save=True, **k)
    d = osdn.glr_backward(x, r, A, dy, dh_T=dh, states=states, **k)
    torch.cuda.synchronize()
    a, k = [f64(t) for t in (x, r, A)], dict(h0=f64(h0), normalize=False)
    ry, rh, rb = Y.glr_ref(*a, **k)
    my, mh, mb = Y.glr_ref(np.abs(a[0]), a[1], a[2], h0=np.abs(k["h0"]), normalize=False)
    # (no memory ends: every token's decay is off by 8 units, every join's by 6 L)
    u = 48 + 8 * T + 6 * 80
    held(y, ry, (u, my), what="y")
    held(h_T, rh, (u, mh), what="h_T")
    held(states, rb[:, ::16], (u, mb[:, ::16]), what="states")
    g, mag = Y.glr_backward_ref(*a, f64(dy), dh_T=f64(dh), **k)
    for n in ("x", "r", "A", "h0"):
        held(d[n], g[n], (2 * u + 16, mag[n]), what="d" + n)
