"""Gated feed-forward product (forward and backward) against the fp64 oracle, element
by element: few rows and many, odd sizes and strides, every tile shape and split."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
from layer_checks import BF, DEV, F32, U, UNIT, f64, held
from oracle import layer as Y

pytestmark = pytest.mark.gpu


def inputs(R, C, F, dt, extra=0, seed=0):
    g = torch.Generator().manual_seed(seed + R + 3 * C + 5 * F)
    n = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(dt).to(DEV)
    x = n(R, C + extra)[:, :C]
    return x, n(F, C, scale=max(C, 1) ** -0.5), n(F, C, scale=max(C, 1) ** -0.5), n(R, F)


def check_forward(R, C, F, dt, act="silu", **kw):
    print("forward", R, C, F, dt, act, kw, flush=True)
    x, wg, wu, _ = inputs(R, C, F, dt, **kw)
    h, g, u = osdn.gated_ffn_forward(x, wg, wu, activation=act, save=True)
    alone = osdn.gated_ffn_forward(x, wg, wu, activation=act)
    torch.cuda.synchronize()
    assert torch.equal(alone[0], h) and alone[1] is None
    rx, rg, ru = f64(x), f64(wg), f64(wu)
    rh, gg, uu = Y.gated_ffn_ref(rx, rg, ru, act)
    mg, mu = np.abs(rx) @ np.abs(rg).T, np.abs(rx) @ np.abs(ru).T
    held(g, gg, (C, mg), what="gate")
    held(u, uu, (C, mu), what="up")
    f = np.abs(Y.activation(gg, act)[0])
    # the slope of every activation is under 1.13
    held(h, rh, (C, 1.13 * mg * np.abs(uu) + f * mu),
         (24, np.abs(gg * uu) * (1 + np.abs(gg))), what="h")


def check_backward(R, C, F, dt, act="silu", **kw):
    print("backward", R, C, F, dt, act, kw, flush=True)
    x, wg, wu, dh = inputs(R, C, F, dt, **kw)
    _, g, u = osdn.gated_ffn_forward(x, wg, wu, activation=act, save=True)
    d = osdn.gated_ffn_backward(x, wg, wu, g, u, dh, activation=act)
    torch.cuda.synchronize()
    rx, rg, ru, rd = f64(x), f64(wg), f64(wu), f64(dh)
    ref, dg, du = Y.gated_ffn_backward_ref(rx, rg, ru, f64(g), f64(u), rd, act)
    # dg and du enter rounded to the operands' type (U), from 24 units of their terms
    one = U[BF] / UNIT if dt is BF else 0.0
    gg = np.abs(f64(g))
    tg = one * np.abs(dg) + 24 * np.abs(rd * f64(u)) * (1 + gg) * 1.13
    tu = one * np.abs(du) + 24 * np.abs(rd) * gg * (1 + gg)
    ax, ag, au, adg, adu = (np.abs(t) for t in (rx, rg, ru, dg, du))
    held(d["x"], ref["x"], (1, tg @ ag + tu @ au), (2 * F, adg @ ag + adu @ au), what="dx")
    held(d["w_gate"], ref["w_gate"], (1, tg.T @ ax), (R, adg.T @ ax), what="dw_gate")
    held(d["w_up"], ref["w_up"], (1, tu.T @ ax), (R, adu.T @ ax), what="dw_up")


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 2, 8, 15, 16, 17, 32, 33, 64, 65, 100])
def test_rows(R, dt):
    check_forward(R, 128, 96, dt)
    check_backward(R, 128, 96, dt)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("C,F", [(1, 1), (7, 5), (31, 17), (64, 16), (72, 40), (200, 130),
                                 (509, 33), (136, 264)])
@pytest.mark.parametrize("R", [3, 70, 130])
def test_widths(R, C, F, dt):
    check_forward(R, C, F, dt, seed=1)
    check_backward(R, C, F, dt, seed=1)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations(act, dt):
    check_forward(5, 64, 48, dt, act, seed=2)
    check_forward(90, 64, 48, dt, act, seed=2)
    check_backward(90, 64, 48, dt, act, seed=2)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("extra", [1, 8, 64])
def test_row_strides(extra, dt):
    check_forward(9, 128, 64, dt, extra=extra, seed=3)
    check_forward(80, 128, 64, dt, extra=extra, seed=3)
    check_backward(80, 128, 64, dt, extra=extra, seed=3)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_rows_off_16_bytes(dt):
    """x that starts off 16 bytes with rows of whole eights; weights there are refused,
    and taken where C is none."""
    for R in (20, 90):
        x, wg, wu, dh = inputs(R, 72, 40, dt, seed=10)
        flat = torch.zeros(8192, dtype=dt, device=DEV)
        y = flat[1:1 + x.numel()].view(R, 72)
        y.copy_(x)
        h, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
        assert torch.equal(osdn.gated_ffn_forward(y, wg, wu)[0], h)
        a, b = (osdn.gated_ffn_backward(t, wg, wu, g, u, dh) for t in (x, y))
        assert all(torch.equal(a[n], b[n]) for n in a)
        w = flat[1:1 + wg.numel()].view(40, 72)
        with pytest.raises(osdn.OsdnError) as e:
            osdn.gated_ffn_forward(x, w, wu)
        assert e.value.status == 7
        with pytest.raises(osdn.OsdnError):
            osdn.gated_ffn_backward(x, wg, w, g, u, dh)
    check_backward(90, 71, 40, dt, seed=11)
    both = torch.randn(80, 71, device=DEV).to(dt)       # one tensor's halves
    x = torch.randn(90, 71, device=DEV).to(dt)
    want = osdn.gated_ffn_forward(x, both[:40].clone(), both[40:].clone())[0]
    assert torch.equal(osdn.gated_ffn_forward(x, both[:40], both[40:])[0], want)


@pytest.mark.parametrize("dt,R,C,F", [
    (BF, 8192, 64, 2048),        # large tiles, one of k
    (BF, 4100, 264, 1050),       # their ends
    (BF, 2048, 1024, 1024),
    (BF, 700, 512, 1400),
    (BF, 130, 2048, 512),        # parts of k
    (BF, 130, 512, 2048),
    (BF, 96, 4096, 128),
    (BF, 2111, 320, 200),
    (F32, 1030, 132, 520),
    (F32, 300, 1000, 257),
    (F32, 4096, 64, 512)])
def test_shapes(dt, R, C, F):
    check_forward(R, C, F, dt, seed=4)
    check_backward(R, C, F, dt, seed=4)


def test_parts_are_used():
    """The sizes above reach the split products: their workspace holds more than dg, du
    and copies of x and the weights."""
    up = lambda n: (n + 255) // 256 * 256
    need = osdn.gated_ffn_forward_workspace_bytes
    assert need(96, 4096, 128, BF) > up(96 * 4096 * 2)
    assert need(8192, 64, 2048, BF) == up(8192 * 64 * 2)
    assert need(64, 4096, 128, BF) == 0
    assert need(4100, 263, 64, BF) >= up(4100 * 264 * 2) + 2 * up(64 * 264 * 2)
    assert (osdn.gated_ffn_backward_workspace_bytes(130, 512, 2048, BF)
            > 2 * up(130 * 2048 * 2) + up(130 * 512 * 2))


def test_leading_dimensions():
    x, wg, wu, dh = inputs(24, 64, 32, BF, seed=5)
    h, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
    d = osdn.gated_ffn_backward(x, wg, wu, g, u, dh)
    y = x.view(2, 3, 4, 64)
    h2, g2, u2 = osdn.gated_ffn_forward(y, wg, wu, save=True)
    assert h2.shape == (2, 3, 4, 32) and torch.equal(h2.view(24, 32), h)
    d2 = osdn.gated_ffn_backward(y, wg, wu, g2, u2, dh.view(2, 3, 4, 32))
    assert d2["x"].shape == y.shape and torch.equal(d2["x"].view(24, 64), d["x"])
    assert torch.equal(d2["w_up"], d["w_up"])
    one = osdn.gated_ffn_forward(x[0], wg, wu)[0]
    assert one.shape == (32,) and torch.equal(one, osdn.gated_ffn_forward(x[:1], wg, wu)[0][0])


def test_extremes():
    """Values at the ends of the activation: no NaN where the result is finite, and an
    inf or NaN of a row stays in that row."""
    x, wg, wu, _ = inputs(70, 64, 32, F32, seed=6)
    for act in ("silu", "gelu", "gelu_tanh"):
        big = x * 1e4
        h, g, u = osdn.gated_ffn_forward(big, wg, wu, activation=act, save=True)
        assert torch.isfinite(h).all()
        d = osdn.gated_ffn_backward(big, wg, wu, g, u, torch.ones_like(h), activation=act)
        assert all(torch.isfinite(t).all() for t in d.values())
        for rows in (slice(0, 70), slice(0, 20)):
            bad = x[rows].clone()
            bad[3, 7] = float("nan")
            bad[5, 1] = float("inf")
            keep = torch.ones(bad.shape[0], dtype=torch.bool, device=DEV)
            keep[3] = keep[5] = False
            a = osdn.gated_ffn_forward(bad, wg, wu, activation=act)[0]
            b = osdn.gated_ffn_forward(x[rows].contiguous(), wg, wu, activation=act)[0]
            assert torch.equal(a[keep], b[keep]) and torch.isnan(a[3]).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_huge_gates(act):
    """Far out every activation is its argument or zero, with a slope of one or zero,
    up to gates whose square or cube is past the type."""
    for s in (20.0, 1e4, 1e20, 1e38):
        g = torch.tensor([s, -s] * 16, device=DEV).repeat(2, 1)
        z = lambda *n: torch.zeros(n, device=DEV)
        x, w, one = z(2, 32), torch.eye(32, device=DEV), torch.ones_like(g)
        # with the identity as the gate's weights dx is dg
        d = osdn.gated_ffn_backward(x, w, z(32, 32), g, one, one, activation=act)
        # (slope of silu at -20: -20 exp(-20))
        assert torch.allclose(d["x"], (g > 0).float(), rtol=0, atol=5e-8), (s, d["x"])
        h = osdn.gated_ffn_forward(g, w, w, activation=act)[0]
        assert h[:, 0].isinf().all() if s == 1e38 else torch.allclose(h[:, 0], g[:, 0] ** 2)


@pytest.mark.parametrize("R,C,F", [(0, 8, 8), (3, 0, 8), (3, 8, 0), (100, 0, 8)])
def test_empty(R, C, F):
    x, wg, wu, dh = inputs(R, C, F, F32)
    h, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
    assert h.shape == (R, F) and not h.any()
    d = osdn.gated_ffn_backward(x, wg, wu, g, u, dh)
    torch.cuda.synchronize()
    assert not d["x"].any() and not d["w_gate"].any() and not d["w_up"].any()


def test_the_same_bits_again():
    x, wg, wu, dh = inputs(300, 509, 130, F32, seed=7)
    _, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
    one = osdn.gated_ffn_backward(x, wg, wu, g, u, dh)
    for _ in range(3):
        two = osdn.gated_ffn_backward(x, wg, wu, g, u, dh)
        assert all(torch.equal(one[n], two[n]) for n in one)


def test_gradient_against_differences():
    x, wg, wu, dh = inputs(40, 48, 36, F32, seed=8)
    h, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
    d = osdn.gated_ffn_backward(x, wg, wu, g, u, dh)
    gen = torch.Generator().manual_seed(9)
    for n, t in dict(x=x, w_gate=wg, w_up=wu).items():
        v = torch.randn(t.shape, generator=gen).to(DEV) * t.abs().mean()
        e = 2e-3

        def loss(s):
            m = dict(x=x, w_gate=wg, w_up=wu)
            m[n] = (t + s * v).contiguous()
            return float((osdn.gated_ffn_forward(**m)[0].double() * dh.double()).sum())
        num, want = (loss(e) - loss(-e)) / (2 * e), float((d[n].double() * v.double()).sum())
        # e^2 of the third derivative; 64 units of 1440 terms at random over 2 e
        scale = float((d[n].double() * v.double()).norm()) + 64 * UNIT * 40 / e
        print(n, num, want, scale, flush=True)
        assert abs(num - want) <= 2e-2 * scale
