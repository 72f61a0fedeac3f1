"""GPU parity of the gated head norm and the residual norm against the fp64
oracle."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from mixer_checks import DEV, f64, held, rows
from oracle import mixer as M

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# B, H, T, D, dtype, extra channels of z's rows (None: no gate), weight per head
GATED = [
    (2, 3, 37, 64, BF, 64, False),
    (1, 1, 1, 128, F32, 0, True),
    (2, 5, 19, 32, BF, 3, True),        # z off 16 bytes
    (3, 16, 130, 128, BF, 0, False),
    (1, 7, 65, 32, F32, 1, False),
    (2, 4, 33, 64, F32, None, True),
    (1, 20, 300, 32, BF, 0, True),
]


def _gated(case, seed=0):
    B, H, T, D, dt, extra, ph = case
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, H, T, D), generator=g) * 0.5).to(dt).to(DEV)
    z = None if extra is None else rows((B, T, H * D), dt, g, extra)
    w = (1 + 0.1 * torch.randn((H, D) if ph else D, generator=g)).to(DEV)
    dy = torch.randn((B, T, H * D), generator=g).to(dt).to(DEV)
    return x, z, w, dy


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("case", GATED, ids=lambda c: "-".join(map(str, c)))
def test_gated_norm(case, gate_first):
    B, H, T, D, dt, extra, ph = case
    print("case:", case, gate_first, flush=True)
    x, z, w, dy = _gated(case)
    y = osdn.gated_norm_forward(x, z, w, gate_first=gate_first)
    got = osdn.gated_norm_backward(x, z, w, dy, gate_first=gate_first)
    torch.cuda.synchronize()
    rx, rz, rw, rdy = f64(x), f64(z), f64(w), f64(dy)
    ref = M.gated_norm_ref(rx, rz, rw, gate_first=gate_first)
    az = np.zeros((B, T, H * D)) if z is None else np.abs(rz)
    # every factor is positive or a product: relative, with silu's through |z|
    held(y, ref, ref * (1 + az), D + 32, what="y")
    gr = M.gated_norm_backward_ref(rx, rz, rw, rdy, gate_first=gate_first)
    heads = lambda t: t.reshape(B, T, H, D)
    xt, zt = rx.transpose(0, 2, 1, 3), (None if z is None else heads(rz))
    gate = np.ones_like(xt) if z is None else np.abs(M.silu(zt))
    v = np.abs(xt) * gate if gate_first else np.abs(xt)
    r = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-6)
    up = np.abs(heads(rdy)) * (1 if gate_first else gate)
    dn = up * np.abs(rw)
    dv = r * dn + v * (v * dn).mean(-1, keepdims=True) * r ** 3
    f = 1 + heads(az)
    k = 2 * D + 64
    held(got["x"], gr["x"], (dv * (gate if gate_first else 1) * f).transpose(0, 2, 1, 3),
         k, what="dx")
    mw = up * v * r * f
    held(got["weight"], gr["weight"], mw.sum((0, 1)) if ph else mw.sum((0, 1, 2)),
         k + 64, what="dweight")
    if z is None:
        assert got["z"] is None
    else:
        dg = dv * np.abs(xt) if gate_first else np.abs(heads(rdy)) * v * r * np.abs(rw)
        slope = M.sigmoid(zt) * (1 + np.abs(zt))
        held(got["z"], gr["z"], (dg * slope * f).reshape(B, T, H * D), k, what="dz")


def test_gated_norm_extremes():
    x, z, w, dy = _gated((1, 2, 9, 64, BF, 0, False))
    # a zero row and gates whose exponential leaves the range
    x[0, 0, 0] = 0
    z[0, 1, :64], z[0, 1, 64:] = -300.0, 300.0
    for first in (False, True):
        y = osdn.gated_norm_forward(x, z, w, gate_first=first)
        d = osdn.gated_norm_backward(x, z, w, dy, gate_first=first)
        assert torch.isfinite(y).all() and not y[0, 0, :64].any()
        assert not y[0, 1, :64].any()
        assert all(bool(torch.isfinite(t).all()) for t in d.values())
    # no tokens, no batch
    for B, T in ((0, 4), (2, 0)):
        x0 = torch.empty((B, 2, T, 64), dtype=BF, device=DEV)
        z0 = torch.empty((B, T, 128), dtype=BF, device=DEV)
        assert osdn.gated_norm_forward(x0, z0, w).shape == (B, T, 128)
        d = osdn.gated_norm_backward(x0, z0, w, z0)
        assert not d["weight"].any()


# rows, width, dtype, residual dtype (None: no residual), scale
RES = [
    (37, 2048, BF, F32, 1.0),
    (5, 1021, BF, BF, 0.5),
    (1, 1, F32, F32, 1.0),
    (3, 8, BF, BF, 2.0),
    (9, 63, F32, None, 0.25),
    (11, 520, BF, F32, 0.1),
    (2, 4104, BF, F32, 1.0),           # four waves a row
    (3, 16384, BF, BF, 1.0),
    (2, 16383, F32, F32, 1.0),         # sixteen waves, element by element
    (1100, 260, BF, BF, 1.0),
    (2100, 129, F32, F32, 1.0),        # more rows than one pass of the backward
    (6, 4000, F32, None, 1.0),
    (1030, 1300, BF, F32, 0.5),        # three vectors a lane of one wave
    (7, 1537, F32, F32, 1.0),          # the first width of four waves
    (600, 2500, BF, BF, 1.0),
    (3, 6001, BF, F32, 0.3),
    (3, 8193, F32, None, 1.0),
]


@pytest.mark.parametrize("case", RES, ids=lambda c: "-".join(map(str, c)))
def test_residual_norm(case):
    R, C, dt, rt, scale = case
    print("case:", case, flush=True)
    g = torch.Generator().manual_seed(R)
    x = torch.randn((R, C), generator=g).to(dt).to(DEV)
    res = None if rt is None else torch.randn((R, C), generator=g).to(rt).to(DEV)
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(DEV)
    y, h = osdn.residual_norm_forward(x, w, res, scale=scale)
    torch.cuda.synchronize()
    ry, rh = M.residual_norm_ref(f64(x), f64(w), f64(res), scale)
    ah = np.abs(scale * f64(x)) + (0 if res is None else np.abs(f64(res)))
    root = 1 / np.sqrt((rh * rh).mean(-1, keepdims=True) + 1e-6)
    # an error of h moves its own element and the root of the row
    rel = np.sqrt((ah * ah).mean(-1, keepdims=True)) * root
    k = C / 64 + 32
    held(h, rh, ah, 2, what="h")
    held(y, ry, ah * root * np.abs(f64(w)) + np.abs(ry) * (1 + rel), k, what="y")

    dy = torch.randn((R, C), generator=g).to(dt).to(DEV)
    dh = torch.randn((R, C), generator=g).to(h.dtype).to(DEV)
    for adj in (dh, None):
        got = osdn.residual_norm_backward(dy, h, w, adj, scale=scale)
        torch.cuda.synchronize()
        hh, dd, ww = f64(h), f64(dy), f64(w)
        gr = M.residual_norm_backward_ref(dd, hh, ww, f64(adj), scale)
        ar = 1 / np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-6)
        dn = np.abs(dd * ww)
        m = ar * dn + np.abs(hh) * (np.abs(hh) * dn).mean(-1, keepdims=True) * ar ** 3
        m = m + (0 if adj is None else np.abs(f64(adj)))
        held(got["residual"], gr["residual"], m, k + 32, what="dh")
        held(got["x"], gr["x"], abs(scale) * m, k + 32, what="dx")
        held(got["weight"], gr["weight"], (np.abs(dd * hh) * ar).sum(0),
             k + R / 64 + 96, what="dweight")


def test_residual_norm_in_place_and_empty():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((4, 7, 256), generator=g).to(BF).to(DEV)
    res = torch.randn((4, 7, 256), generator=g).to(DEV)
    w = torch.ones(256, device=DEV)
    y, h = osdn.residual_norm_forward(x, w, res)
    r2 = res.clone()
    y2, h2 = osdn.residual_norm_forward(x, w, r2, out=(torch.empty_like(x), r2))
    assert h2 is r2 and torch.equal(h2, h) and torch.equal(y2, y)
    y3, h3 = osdn.residual_norm_forward(x, w, res, out=(torch.empty_like(x), None))
    assert h3 is None and torch.equal(y3, y)
    z = torch.zeros_like(x)
    y, h = osdn.residual_norm_forward(z, w)
    assert not y.any() and not h.any()
    e = torch.empty((0, 256), dtype=BF, device=DEV)
    y, h = osdn.residual_norm_forward(e, w)
    assert y.shape == (0, 256)
    d = osdn.residual_norm_backward(e, e, w)
    assert not d["weight"].any()


@pytest.mark.gpu
def test_gated_norm_backward_without_heads():
    """No heads: a shared weight's gradient is zeros."""
    x, z, dy = (torch.zeros(s, device=DEV) for s in ((2, 0, 3, 64), (2, 3, 0), (2, 3, 0)))
    for weight in (torch.ones(64, device=DEV), torch.ones(0, 64, device=DEV)):
        g = osdn.gated_norm_backward(x, z, weight, dy)
        assert g["weight"].shape == weight.shape and not g["weight"].any()
    assert osdn.gated_norm_forward(x, z, torch.ones(64, device=DEV)).shape == (2, 3, 0)
