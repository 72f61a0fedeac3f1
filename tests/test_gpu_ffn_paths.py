"""Every way in which the planner cuts the feed-forward products, against the same
products in 64 bits: each tile shape alone and in the joined launch, whole rounds, split
rounds and both in one product, the five operand buffers more than once in turn, ragged
ends of every dimension. A size names the path that it is there for, and the planner is
asked for it.

Bounds. An element is a sum of n products of independent inputs of random sign, with
sigma^2 the sum of their squares. Roundings of the factors (a half step U of a stored type
each) are independent errors of at most U times a product: with probability 1 - 3e-14 an
element's are under 8 U sigma together (Hoeffding: 2 exp(-8^2 / 2)). A partial sum of the
products stays under 8 sigma likewise, every addition rounds it once: 2^-24 8 sigma,
n times, 64 sqrt(n) 2^-24 sigma together. So a missing tile of k, which leaves out a
root of its share of sigma, is 5 bounds away at the sizes here."""
import numpy as np
import pytest
import torch

import delta_rule_recurrent_scan_amd as osdn
import ffn_plans as P
from ffn_plans import LARGE, MIDDLE, SMALL
from layer_checks import BF, DEV, F32, U, UNIT

pytestmark = pytest.mark.gpu


def within(got, ref, sigma, n, relative, what):
    """relative: the rounding of the factors of a product, over all of them."""
    g = got.double()
    assert got.shape == ref.shape and torch.isfinite(g).all(), what
    bound = U[got.dtype] * ref.abs() + (8 * relative + 64 * n ** 0.5 * UNIT) * sigma + 1e-30
    worst = float(((g - ref).abs() / bound).max())
    print("%s: worst error %.3f of its bound" % (what, worst), flush=True)
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


def root(a, b):
    """sigma of a @ b."""
    return ((a * a) @ (b * b)).sqrt()


def inputs(R, C, F, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s, scale=1.0: (torch.randn(s, generator=g, device=DEV) * scale).to(dt)
    return n(R, C), n(F, C, scale=C ** -0.5), n(F, C, scale=C ** -0.5), n(R, F)


def silu(v):
    s = torch.sigmoid(v)
    return v * s, s * (1 + v * (1 - s))


F_, T_ = False, True


# type, R, C, F, (shape, split, whole rounds), tiles of k at least
FORWARDS = [
    (BF, 3001, 712, 1366, (LARGE, F_, F_), 11),
    (BF, 4001, 712, 2001, (LARGE, F_, T_), 11),
    (BF, 6001, 1021, 1366, (LARGE, T_, T_), 16),
    (BF, 4100, 1500, 1366, (LARGE, F_, F_), 23),
    (BF, 1500, 264, 1366, (MIDDLE, F_, F_), 4),
    (BF, 6001, 264, 1366, (MIDDLE, F_, T_), 4),
    (BF, 65, 264, 130, (SMALL, F_, F_), 4),
    (BF, 1000, 264, 2001, (SMALL, F_, T_), 4),
    (BF, 65, 1500, 130, (SMALL, T_, F_), 23),
    (BF, 1500, 2100, 1366, (SMALL, T_, T_), 32),
    (F32, 4001, 264, 777, (MIDDLE, F_, F_), 8),
    (F32, 4001, 264, 2001, (MIDDLE, F_, T_), 8),
    (F32, 6001, 1500, 130, (MIDDLE, T_, F_), 46),
    (F32, 6001, 2100, 777, (MIDDLE, T_, T_), 65),
    (F32, 65, 264, 130, (SMALL, F_, F_), 8),
    (F32, 1000, 264, 2001, (SMALL, F_, T_), 8),
    (F32, 65, 509, 130, (SMALL, T_, F_), 15),
    (F32, 1500, 509, 1366, (SMALL, T_, T_), 15)]


@pytest.mark.parametrize("dt,R,C,F,path,tiles", FORWARDS)
def test_forward(dt, R, C, F, path, tiles):
    p = P.forward(R, C, F, dt is BF)
    assert (p.shape, p.splits > 1, p.whole > 0) == path and p.nt >= tiles
    x, wg, wu, _ = inputs(R, C, F, dt, R + C)
    osdn.kernel_timing(True)
    h, g, u = osdn.gated_ffn_forward(x, wg, wu, save=True)
    names = set(osdn.kernel_times())
    osdn.kernel_timing(False)
    assert ("ffn_join" in names) == path[1] and "ffn" in names
    x, wg, wu = x.double(), wg.double(), wu.double()
    rg, ru, sg, su = x @ wg.t(), x @ wu.t(), root(x, wg.t()), root(x, wu.t())
    within(g, rg, sg, C, 0, "gate")
    within(u, ru, su, C, 0, "up")
    f = silu(rg)[0]
    # (the slope of SiLU is under 1.1; 24 units and the argument's for its own roundings)
    own = 24 * UNIT * (rg * ru).abs() * (1 + rg.abs()) / (64 * C ** 0.5 * UNIT)
    within(h, f * ru, 1.1 * sg * ru.abs() + f.abs() * su + own, C, 0, "h")


# type, R, C, F, dx's path, the weights' path (None: both in one launch of the first's
# shape, with the splits of each)
BACKWARDS = [
    (BF, 4100, 2100, 521, (LARGE, F_, F_), (SMALL, F_, F_)),
    (BF, 8191, 1500, 1050, (LARGE, F_, F_), (LARGE, T_, F_)),
    (BF, 777, 2100, 3000, (SMALL, F_, F_), (LARGE, F_, F_)),
    (BF, 2050, 2100, 3000, (LARGE, T_, F_), (LARGE, F_, F_)),
    (BF, 8191, 2100, 777, (LARGE, T_, T_), (MIDDLE, F_, F_)),
    (BF, 4100, 2100, 777, (LARGE, F_, F_), (MIDDLE, F_, F_)),
    (BF, 8191, 2100, 257, (MIDDLE, F_, T_), (MIDDLE, T_, F_)),
    (BF, 6001, 2100, 2001, (LARGE, F_, F_), (MIDDLE, T_, T_)),
    (BF, 4001, 1500, 130, (MIDDLE, F_, F_), (SMALL, T_, F_)),
    (BF, 333, 2100, 3000, (MIDDLE, T_, F_), (LARGE, F_, F_)),
    (BF, 4001, 2100, 3000, (MIDDLE, T_, T_), (LARGE, F_, F_)),
    (BF, 65, 2100, 2001, (SMALL, T_, F_), (SMALL, F_, T_)),
    (F32, 200, 2100, 3000, (MIDDLE, T_, F_), (MIDDLE, F_, T_)),
    (F32, 3001, 1500, 521, (SMALL, T_, T_), (MIDDLE, T_, F_)),
    (F32, 513, 2100, 2001, (MIDDLE, T_, F_), (MIDDLE, T_, T_)),
    (F32, 65, 712, 3000, (SMALL, T_, F_), (SMALL, F_, T_)),
    (F32, 6001, 777, 130, (SMALL, F_, T_), (SMALL, T_, F_)),
    (F32, 2050, 2100, 1050, (SMALL, T_, T_), (SMALL, T_, T_)),
    (F32, 4100, 1500, 130, (MIDDLE, F_, F_), (SMALL, T_, F_)),
    (F32, 8191, 1021, 130, (MIDDLE, F_, T_), (SMALL, T_, F_)),
    (F32, 4001, 2100, 257, (MIDDLE, T_, T_), (SMALL, T_, F_)),
    (F32, 777, 2100, 1366, (SMALL, F_, F_), (SMALL, F_, T_)),
    (BF, 2050, 2100, 777, (LARGE, F_, F_), None),
    (BF, 4001, 2100, 130, (LARGE, F_, T_), None),
    (BF, 200, 2100, 2001, (LARGE, T_, F_), None),
    (BF, 1500, 2100, 257, (MIDDLE, F_, F_), None),
    (BF, 4001, 1021, 130, (MIDDLE, F_, T_), None),
    (BF, 65, 1021, 2001, (MIDDLE, T_, F_), None),
    (BF, 1500, 264, 130, (SMALL, F_, T_), None),
    (BF, 65, 264, 777, (SMALL, T_, F_), None),
    (F32, 1000, 2100, 521, (MIDDLE, F_, F_), None),
    (F32, 2050, 1500, 130, (MIDDLE, F_, T_), None),
    (F32, 65, 2100, 777, (MIDDLE, T_, F_), None),
    (F32, 1000, 333, 2001, (MIDDLE, T_, T_), None),
    (F32, 513, 264, 130, (SMALL, T_, T_), None)]


@pytest.mark.parametrize("dt,R,C,F,dx,dw", BACKWARDS)
def test_backward(dt, R, C, F, dx, dw):
    p, q, pair = P.backward(R, C, F, dt is BF)
    if dw is None:
        assert pair and p.shape == q.shape
        assert (p.shape, p.splits > 1, q.splits > 1) == dx
        launches = {"ffn_dxdw"} | ({"ffn_dxdw_join"} if dx[1] or dx[2] else set())
    else:
        assert not pair
        assert (p.shape, p.splits > 1, p.whole > 0) == dx
        assert (q.shape, q.splits > 1, q.whole > 0) == dw
        launches = ({"ffn_dx", "ffn_dw"} | ({"ffn_dx_join"} if dx[1] else set()) |
                    ({"ffn_dw_join"} if dw[1] else set()))
    x, wg, wu, dh = inputs(R, C, F, dt, R + F)
    gen = torch.Generator(device=DEV).manual_seed(F)
    gate, up = (torch.randn((R, F), generator=gen, device=DEV).to(dt) for _ in range(2))
    osdn.kernel_timing(True)
    d = osdn.gated_ffn_backward(x, wg, wu, gate, up, dh)
    names = set(osdn.kernel_times())
    osdn.kernel_timing(False)
    assert names == launches | {"ffn_grad"}
    x, wg, wu, dh, gate, up = (t.double() for t in (x, wg, wu, dh, gate, up))
    f, slope = silu(gate)
    # dg and du enter rounded to bf16, or off by 24 units and the argument's: |g| < 6
    dg, du = dh * up * slope, dh * f
    one = U[BF] if dt is BF else 0.0
    wide = 24 * 7 * 1.1 * UNIT
    tg, tu = (dh * up).abs(), dh.abs() * gate.abs()
    part = lambda a, t, b, a2, t2, b2: (one ** 2 * ((a * a) @ (b * b) + (a2 * a2) @ (b2 * b2)) +
                                        wide ** 2 * ((t * t) @ (b * b) + (t2 * t2) @ (b2 * b2))
                                        ).sqrt()
    z = lambda t: t[:, :0]
    for name, ref, sigma, err, n in (
            ("x", dg @ wg + du @ wu, (root(dg, wg) ** 2 + root(du, wu) ** 2).sqrt(),
             part(dg, tg, wg, du, tu, wu), 2 * F),
            ("w_gate", dg.t() @ x, root(dg.t(), x),
             part(dg.t(), tg.t(), x, z(dg.t()), z(dg.t()), x[:0]), R),
            ("w_up", du.t() @ x, root(du.t(), x),
             part(du.t(), tu.t(), x, z(du.t()), z(du.t()), x[:0]), R)):
        within(d[name], ref, sigma + 8 * err / (64 * n ** 0.5 * UNIT), n, 0, "d" + name)


def test_every_path_is_here():
    """Each shape whole and split, alone and joined, appears above."""
    for dt in (BF, F32):
        for s in (LARGE, MIDDLE, SMALL)[dt is F32:]:
            assert {c[4][1:] for c in FORWARDS if c[0] is dt and c[4][0] == s} >= {
                (F_, F_), (F_, T_)}
            for k in (4, 5):
                cuts = {c[k][1:] for c in BACKWARDS if c[0] is dt and c[5] and c[k][0] == s}
                assert len(cuts) >= 2, (dt, s, k, cuts)
            assert [c for c in BACKWARDS if c[0] is dt and not c[5] and c[4][0] == s]
